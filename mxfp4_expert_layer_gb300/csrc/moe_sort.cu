// Tokens sorted by expert and back, for experts of the caller's own, with the gradients of
// both moves and of the top-k weights.
//
// With N = T k assignments a = t k + j of keys e_a (the expert, or E for an index outside
// [0, E), an assignment that is dropped):
//   place(a) = #{b : (e_b, b) < (e_a, a)}          a stable counting sort
//   rows[place(a)] = x[t]                          0 where dropped
//   out[t] = sum_j w[t, j] y[place(t, j)]          and its gradients
//   dy[place(t, j)] = w[t, j] dout[t],  dw[t, j] = <dout[t], y[place(t, j)]>
// Everything but the dot products and the sums over j is movement: bound by memory.
#include "moe_dense.cuh"
#include "sm100_ptx.cuh"

namespace moe {

namespace {

constexpr int kOrderThreads = 1024, kOrderWarps = kOrderThreads / 32;
constexpr int kKeys = kMaxExperts + 1;  // the experts, and what is dropped

__device__ __forceinline__ int key_of(int e, int E) { return e >= 0 && e < E ? e : E; }

// The order of a routing by one block: each warp counts the keys of a contiguous run of
// assignments, the counts become the warps' first places, and each warp places its run.
__global__ void __launch_bounds__(kOrderThreads) order_kernel(const __grid_constant__ SortParams p) {
  __shared__ int count[kOrderWarps][kKeys + 2];
  __shared__ int first[kKeys];
  __shared__ int warp_total[kOrderWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, keys = p.E + 1;
  for (int i = tid; i < kOrderWarps * (kKeys + 2); i += kOrderThreads) (&count[0][0])[i] = 0;
  __syncthreads();
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  const int n = p.T * p.k, run = ceil_div(ceil_div(n, kOrderWarps), 32) * 32;
  const int begin = min(n, warp * run), end = min(n, begin + run);
  for (int a = begin + lane; a < end; a += 32) atomicAdd(&count[warp][key_of(__ldcg(p.idx + a), p.E)], 1);
  __syncthreads();
  // the places of key e begin behind the lower keys; those of a warp behind the lower warps
  int total = 0;
  if (tid < keys)
    for (int w = 0; w < kOrderWarps; ++w) {
      const int c = count[w][tid];
      count[w][tid] = total;
      total += c;
    }
  int scan = total;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, scan, d);
    if (lane >= d) scan += o;
  }
  if (lane == 31) warp_total[warp] = scan;
  __syncthreads();
  if (tid < keys) {
    int before = scan - total;
    for (int w = 0; w < warp; ++w) before += warp_total[w];
    first[tid] = before;
    p.offsets[tid] = before;
  }
  __syncthreads();
  for (int a0 = begin; a0 < end; a0 += 32) {
    const int a = a0 + lane;
    const bool on = a < end;
    const int key = on ? key_of(__ldcg(p.idx + a), p.E) : -1;
    const unsigned same = __match_any_sync(0xffffffffu, key);
    const int rank = __popc(same & ((1u << lane) - 1));
    if (on) {
      const int place = first[key] + count[warp][key] + rank;
      const bool kept = key < p.E;
      p.perm[place] = kept ? a : -1 - a;
      p.inv_perm[a] = kept ? place : -1 - place;
    }
    __syncwarp();
    if (on && rank == 0) count[warp][key] += __popc(same);
    __syncwarp();
  }
}

// One row of scales of `bytes` bytes to another place, or zeros, by a warp.
template <typename U>
__device__ __forceinline__ void move_units(void* dst, const void* src, size_t to, size_t from, int units, bool kept) {
  for (int i = threadIdx.x & 31; i < units; i += 32)
    reinterpret_cast<U*>(dst)[to * units + i] = kept ? __ldcg(reinterpret_cast<const U*>(src) + from * units + i) : U(0);
}
__device__ __forceinline__ void move_scales(const SortParams& p, size_t to, size_t from, bool kept) {
  if ((p.scale_bytes & 3) == 0)
    move_units<unsigned>(p.row_scales, p.scales, to, from, p.scale_bytes >> 2, kept);
  else if ((p.scale_bytes & 1) == 0)
    move_units<unsigned short>(p.row_scales, p.scales, to, from, p.scale_bytes >> 1, kept);
  else
    move_units<unsigned char>(p.row_scales, p.scales, to, from, p.scale_bytes, kept);
}

// One block per token: its row is read once and written to its k places.
__global__ void __launch_bounds__(256) gather_kernel(const __grid_constant__ SortParams p) {
  __shared__ int place[kMaxTopK];
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  const size_t t = blockIdx.x;
  if (threadIdx.x < p.k) place[threadIdx.x] = __ldcg(p.inv_perm + t * p.k + threadIdx.x);
  __syncthreads();
  const int vecs = p.row_bytes / 16;
  uint4* rows = reinterpret_cast<uint4*>(p.rows);
  for (int v = threadIdx.x; v < vecs; v += blockDim.x) {
    const uint4 r = __ldcg(reinterpret_cast<const uint4*>(p.x) + t * vecs + v);
    for (int j = 0; j < p.k; ++j) {
      const int at = place[j];
      if (at >= 0)
        rows[(size_t)at * vecs + v] = r;
      else
        rows[(size_t)(-1 - at) * vecs + v] = make_uint4(0, 0, 0, 0);
    }
  }
  if (p.scale_bytes)
    for (int j = threadIdx.x >> 5; j < p.k; j += blockDim.x >> 5) {
      const int at = place[j];
      move_scales(p, at >= 0 ? at : -1 - at, t, at >= 0);
    }
}

// Row of assignment (t, j) that takes part, or -1; where it was dropped `zero` is its row.
__device__ __forceinline__ int row_of(int at, int n) { return at >= 0 && at < n ? at : -1; }

// out[t] = sum_j w[t, j] y[place(t, j)], eight columns a thread.
template <typename A>
__global__ void __launch_bounds__(256) unsort_kernel(const __grid_constant__ UnsortParams p) {
  __shared__ int row[kMaxTopK];
  __shared__ float weight[kMaxTopK];
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  const size_t t = blockIdx.x;
  if (threadIdx.x < p.k) {
    row[threadIdx.x] = row_of(__ldcg(p.inv_perm + t * p.k + threadIdx.x), p.T * p.k);
    weight[threadIdx.x] = p.w ? __ldcg(p.w + t * p.k + threadIdx.x) : 1.f;
  }
  __syncthreads();
  const int vecs = p.H / 8;
  for (int v = threadIdx.x; v < vecs; v += blockDim.x) {
    float sum[8] = {};
    for (int j = 0; j < p.k; ++j) {
      if (row[j] < 0) continue;
      Vec8<A> r;
      float f[8];
      r.load(p.y, (size_t)row[j] * vecs + v);
      r.get(f);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[i] = fmaf(weight[j], f[i], sum[i]);
    }
    Vec8<A> o;
    o.set(sum);
    o.store(p.out, t * vecs + v);
  }
}

// dy[place(t, j)] = w[t, j] dout[t] and dw[t, j] = <dout[t], y[place(t, j)]>: one block per token.
template <typename A>
__global__ void __launch_bounds__(256) unsort_backward_kernel(const __grid_constant__ UnsortBackwardParams q) {
  __shared__ float part[8];
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  const UnsortParams& p = q.f;
  const size_t t = blockIdx.x;
  const int vecs = p.H / 8, n = p.T * p.k, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int j = 0; j < p.k; ++j) {
    const int at = __ldcg(p.inv_perm + t * p.k + j), row = row_of(at, n), to = row_of(at >= 0 ? at : -1 - at, n);
    const float w = row < 0 ? 0.f : p.w ? __ldcg(p.w + t * p.k + j) : 1.f;
    float dot = 0.f;
    for (int v = threadIdx.x; v < vecs; v += blockDim.x) {
      Vec8<A> r;
      float d[8], f[8];
      r.load(q.d_out, t * vecs + v);
      r.get(d);
      if (q.d_w && row >= 0) {
        r.load(p.y, (size_t)row * vecs + v);
        r.get(f);
#pragma unroll
        for (int i = 0; i < 8; ++i) dot = fmaf(d[i], f[i], dot);
      }
      if (q.d_y && to >= 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] = row < 0 ? 0.f : w * d[i];
        r.set(d);
        r.store(q.d_y, (size_t)to * vecs + v);
      }
    }
    if (!q.d_w) continue;
#pragma unroll
    for (int s = 16; s >= 1; s >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, s);
    if (lane == 0) part[warp] = dot;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int i = 1; i < (int)blockDim.x / 32; ++i) dot += part[i];
      q.d_w[t * p.k + j] = dot;
    }
    __syncthreads();
  }
}

// The gradient of the top-k weights into the logits, a warp per token.  With S = sum_i w_i g_i:
//   softmax over the k selected   dl_j = w_j (g_j - S)
//   sigmoids over their sum       dl_j = w_j (1 - sigmoid(l_j)) (g_j - S)
//   softmax over all E            dl_e = p_e (g_e - S), g_e = 0 where e was not selected
// added where an expert was selected twice, in the order of j; 0 elsewhere.
__global__ void __launch_bounds__(256) route_backward_kernel(const __grid_constant__ RouteBackwardParams p) {
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const size_t t = (size_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (t >= (size_t)p.T) return;
  int e = -1;
  float g = 0.f, w = 0.f;
  if (lane < p.k) {
    e = __ldcg(p.idx + t * p.k + lane);
    if (e >= p.E) e = -1;
    g = __ldcg(p.d_w + t * p.k + lane);
    w = __ldcg(p.w + t * p.k + lane);
  }
  float s = w * g;
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
  const float* logits = p.logits + t * p.E;
  float* out = p.d_logits + t * p.E;
  const bool all = p.gating == kGatingSoftmaxAll;
  float part = all ? g : w * (g - s);
  if (p.gating == kGatingSigmoid && e >= 0) part *= 1.f / (1.f + expf(__ldcg(logits + e)));
  float top = -INFINITY, sum = 0.f, l[kMaxExperts / 32];
  if (all) {
#pragma unroll
    for (int i = 0; i < kMaxExperts / 32; ++i) {
      l[i] = lane + 32 * i < p.E ? __ldcg(logits + lane + 32 * i) : -INFINITY;
      top = fmaxf(top, l[i]);
    }
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
#pragma unroll
    for (int i = 0; i < kMaxExperts / 32; ++i) {
      l[i] = lane + 32 * i < p.E ? expf(l[i] - top) : 0.f;
      sum += l[i];
    }
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  }
#pragma unroll
  for (int i = 0; i < kMaxExperts / 32; ++i) {
    if (32 * i >= p.E) break;
    const int c = lane + 32 * i;
    float v = 0.f;
    for (int j = 0; j < p.k; ++j) {
      const float add = __shfl_sync(0xffffffffu, part, j);
      if (__shfl_sync(0xffffffffu, e, j) == c) v += add;
    }
    if (all) v = l[i] / sum * (v - s);
    if (c < p.E) out[c] = v;
  }
}

template <typename A>
cudaError_t unsort_t(const UnsortParams& p, cudaStream_t stream) {
  return launch_pdl(unsort_kernel<A>, dim3(p.T), dim3(256), 0, stream, p);
}
template <typename A>
cudaError_t unsort_backward_t(const UnsortBackwardParams& q, cudaStream_t stream) {
  return launch_pdl(unsort_backward_kernel<A>, dim3(q.f.T), dim3(256), 0, stream, q);
}

}  // namespace

cudaError_t launch_sort(const SortParams& p, cudaStream_t stream) {
  const cudaError_t e = launch_pdl(order_kernel, dim3(1), dim3(kOrderThreads), 0, stream, p);
  return e != cudaSuccess ? e : launch_pdl(gather_kernel, dim3(p.T), dim3(256), 0, stream, p);
}

cudaError_t launch_unsort(const UnsortParams& p, int dtype, cudaStream_t stream) {
  return dtype == kDtypeBf16  ? unsort_t<__nv_bfloat16>(p, stream)
         : dtype == kDtypeF16 ? unsort_t<__half>(p, stream)
                              : unsort_t<float>(p, stream);
}

cudaError_t launch_unsort_backward(const UnsortBackwardParams& q, int dtype, cudaStream_t stream) {
  return dtype == kDtypeBf16  ? unsort_backward_t<__nv_bfloat16>(q, stream)
         : dtype == kDtypeF16 ? unsort_backward_t<__half>(q, stream)
                              : unsort_backward_t<float>(q, stream);
}

cudaError_t launch_route_backward(const RouteBackwardParams& p, cudaStream_t stream) {
  return launch_pdl(route_backward_kernel, dim3(ceil_div(p.T, 8)), dim3(256), 0, stream, p);
}

}  // namespace moe
