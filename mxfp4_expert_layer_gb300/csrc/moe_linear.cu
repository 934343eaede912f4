// The gradient of a projection's epilogue, out = act(pre) + residual with pre = x W^T + b:
//   dp = dout act'(pre)       rounded to 16 bits, the next products' operand type
//   db = sum_t dp             of the unrounded dp, in f32
// One pass over dout and pre; bound by memory.
#include <algorithm>

#include "moe_dense.cuh"
#include "sm100_ptx.cuh"

namespace moe {

namespace {

// A block takes 256 columns (8 a lane) of a run of rows, two rows to a warp in turn; its warps'
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
  auto load = [&](int t, Vec8<O>& d, Vec8<float>& v) {
    const size_t at = ((size_t)t * p.N + col) / 8;
    d.load(p.d_out, at);
    if (p.pre) v.load(p.pre, at);
  };
  auto use = [&](int t, const Vec8<O>& d, const Vec8<float>& v) {
    float f[8];
    d.get(f);
    if (p.pre) {
      float g[8];
      v.get(g);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float slope;
        if (p.act == kActSilu)
          act_f<kActSilu>(g[i], slope);
        else
          act_f<kActGelu>(g[i], slope);
        f[i] *= slope;
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[i] += f[i];
    if (p.dp) {
      Vec8<X> o;
      o.set(f);
      o.store(p.dp, ((size_t)t * p.N + col) / 8);
    }
  };
  if (col < p.N)
    for (int t = t0 + warp; t < t1; t += 16) {
      Vec8<O> d0, d1;
      Vec8<float> v0, v1;
      load(t, d0, v0);
      if (t + 8 < t1) load(t + 8, d1, v1);
      use(t, d0, v0);
      if (t + 8 < t1) use(t + 8, d1, v1);
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

// The sums of the partial rows: eight threads take those of one column in turn, then add in
// order.  Every load of a thread at once, up to eight: one after the other each is a memory round trip.
constexpr int kMaxSplits = 64;
__global__ void __launch_bounds__(256) linear_bias_kernel(const float* partial, int splits, int N, float* d_bias) {
  __shared__ float buf[8][33];
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5, c = blockIdx.x * 32 + tx;
  float part[kMaxSplits / 8], v = 0.f;
#pragma unroll
  for (int i = 0; i < kMaxSplits / 8; ++i) {
    const int s = ty + 8 * i;
    part[i] = s < splits && c < N ? __ldcg(partial + (size_t)s * N + c) : 0.f;
  }
#pragma unroll
  for (int i = 0; i < kMaxSplits / 8; ++i) v += part[i];
  buf[ty][tx] = v;
  __syncthreads();
  if (ty == 0 && c < N) {
#pragma unroll
    for (int i = 1; i < 8; ++i) v += buf[i][tx];
    d_bias[c] = v;
  }
}

template <typename X, typename O>
cudaError_t grad_t(const LinearGradParams& p, cudaStream_t stream) {
  const cudaError_t e = launch_pdl(linear_grad_kernel<X, O>, dim3(ceil_div(p.N, 256), p.splits), dim3(256), 0, stream, p);
  if (e != cudaSuccess || !p.d_bias || p.splits == 1) return e;
  return launch_pdl(linear_bias_kernel, dim3(ceil_div(p.N, 32)), dim3(256), 0, stream, (const float*)p.partial, p.splits, p.N,
                    p.d_bias);
}

}  // namespace

// Blocks along T: four to an SM altogether, with sixteen rows each at least.
int linear_grad_splits(int T, int N) {
  const int cols = ceil_div(N, 256), want = ceil_div(4 * kMaxCtas, cols), most = ceil_div(T, 16);
  return std::min(std::min(want, most), kMaxSplits);
}

cudaError_t launch_linear_grad(const LinearGradParams& p, int dtype, int out_dtype, cudaStream_t stream) {
  if (dtype == kDtypeBf16)
    return out_dtype == kDtypeF32 ? grad_t<__nv_bfloat16, float>(p, stream) : grad_t<__nv_bfloat16, __nv_bfloat16>(p, stream);
  return out_dtype == kDtypeF32 ? grad_t<__half, float>(p, stream) : grad_t<__half, __half>(p, stream);
}

}  // namespace moe
