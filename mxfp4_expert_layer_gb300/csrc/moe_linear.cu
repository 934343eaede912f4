// The gradient of a projection's epilogue, out = act(pre) + residual with pre = x W^T + b:
//   dp = dout act'(pre)       rounded to 16 bits, the next products' operand type
//   db = sum_t dp             of the unrounded dp, in f32
// One pass over dout and pre; bound by memory.
#include "moe_dense.cuh"
#include "sm100_ptx.cuh"

namespace moe {

namespace {

// A block takes 256 columns (8 a lane) of a run of rows, a row to a warp in turn; its warps'
// sums are added in order, and the blocks along T leave a row of partial sums each.
template <typename X, typename O>
__global__ void __launch_bounds__(256) linear_grad_kernel(const __grid_constant__ LinearGradParams p) {
  __shared__ float sums[8][32][9];
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int col = (blockIdx.x * 32 + lane) * 8;
  const int t0 = (int)((long long)blockIdx.y * p.T / p.splits), t1 = (int)((long long)(blockIdx.y + 1) * p.T / p.splits);
  float sum[8] = {};
  if (col < p.N)
    for (int t = t0 + warp; t < t1; t += 8) {
      const size_t at = ((size_t)t * p.N + col) / 8;
      Vec8<O> d;
      float f[8];
      d.load(p.d_out, at);
      if (p.pre) {
        Vec8<float> v;
        float g[8];
        v.load(p.pre, at);
        v.get(g);
        d.get(f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float slope;
          if (p.act == kActSilu)
            act_f<kActSilu>(g[i], slope);
          else
            act_f<kActGelu>(g[i], slope);
          f[i] *= slope;
        }
      } else {
        d.get(f);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[i] += f[i];
      if (p.dp) {
        Vec8<X> o;
        o.set(f);
        o.store(p.dp, at);
      }
    }
  if (!p.d_bias) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) sums[warp][lane][i] = sum[i];
  __syncthreads();
  const int c = threadIdx.x, at = blockIdx.x * 256 + c;
  float v = sums[0][c >> 3][c & 7];
#pragma unroll
  for (int w = 1; w < 8; ++w) v += sums[w][c >> 3][c & 7];
  if (at < p.N) (p.splits > 1 ? p.partial + (size_t)blockIdx.y * p.N : p.d_bias)[at] = v;
}

__global__ void __launch_bounds__(256) linear_bias_kernel(const float* partial, int splits, int N, float* d_bias) {
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= N) return;
  float v = 0.f;
  for (int s = 0; s < splits; ++s) v += __ldcg(partial + (size_t)s * N + c);
  d_bias[c] = v;
}

template <typename X, typename O>
cudaError_t grad_t(const LinearGradParams& p, cudaStream_t stream) {
  const cudaError_t e = launch_pdl(linear_grad_kernel<X, O>, dim3(ceil_div(p.N, 256), p.splits), dim3(256), 0, stream, p);
  if (e != cudaSuccess || !p.d_bias || p.splits == 1) return e;
  return launch_pdl(linear_bias_kernel, dim3(ceil_div(p.N, 256)), dim3(256), 0, stream, (const float*)p.partial, p.splits, p.N,
                    p.d_bias);
}

}  // namespace

// Blocks along T: enough to fill the GPU, with eight rows each at least.
int linear_grad_splits(int T, int N) {
  const int cols = ceil_div(N, 256), want = ceil_div(8 * kMaxCtas, cols), most = ceil_div(T, 8);
  const int s = want < most ? want : most;
  return s > 256 ? 256 : s;
}

cudaError_t launch_linear_grad(const LinearGradParams& p, int dtype, int out_dtype, cudaStream_t stream) {
  if (dtype == kDtypeBf16)
    return out_dtype == kDtypeF32 ? grad_t<__nv_bfloat16, float>(p, stream) : grad_t<__nv_bfloat16, __nv_bfloat16>(p, stream);
  return out_dtype == kDtypeF32 ? grad_t<__half, float>(p, stream) : grad_t<__half, __half>(p, stream);
}

}  // namespace moe
