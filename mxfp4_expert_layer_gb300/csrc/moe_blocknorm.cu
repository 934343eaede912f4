// The norms before and after a block, fused with the block's gate and the residual
// scale, forward and backward.
//
// With z the block's output, r the residual stream, w the post-norm's weight, v the
// next pre-norm's weight and g the gate (per feature, per token, or full):
//   n = z / rms(z) * w              (n = z without a post-norm)
//   s = round(a r + g n)            the stream, rounded to its stored type
//   y = s / rms(s) * v              of the stored s, as the layer's own norm step does
// Backward, given ds' (into s from downstream) and dy:
//   ds = ds' + rs (v dy - s rs mean(v dy s rs))    rs = 1 / rms(s)
//   dr = a ds,  p = g ds,  dg = ds n,  dw = sum_t p z rz,  dv = sum_t dy s rs
//   dz = rz (w p - z rz mean(w p z rz))            rz = 1 / rms(z)
// Both are bound by memory: one block holds a row in registers, so every element is
// read once and written once, and the row's sums are the only exchange.
#include "moe_dense.cuh"
#include "sm100_ptx.cuh"

namespace moe {

namespace {

// Sums of N values over the block, the same bits in every thread (fixed order: lanes by
// butterfly, then warps ascending).  `buf` holds N * 32 floats; successive calls take
// two buffers in turn, so one barrier per call is enough: whoever writes a buffer again
// has passed the barrier of the call between, which every reader of it reached later.
template <int N>
__device__ __forceinline__ void block_sums(float (&v)[N], float* buf) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_sum_butterfly(v[i]);
  if (nw == 1) return;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) buf[i * 32 + warp] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_sum_butterfly(lane < nw ? buf[i * 32 + lane] : 0.f);
}

template <typename A, typename S, int VPT>
__global__ void __launch_bounds__(1024) block_norm_kernel(BlockNormParams p) {
  __shared__ float buf[2][32];
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  const int nvec = p.H / 8;
  const size_t row = blockIdx.x;
  const size_t base = row * nvec;
  Vec8<A> zr[VPT];
  Vec8<S> rr[VPT];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int v = threadIdx.x + j * blockDim.x;
    zr[j].zero();
    rr[j].zero();
    if (v < nvec) {
      zr[j].load(p.block, base + v);
      if (p.residual) rr[j].load(p.residual, base + v);
    }
  }
  float rz = 1.f;
  if (p.norm_w) {
    float ss[1] = {0.f};
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      float f[8];
      zr[j].get(f);
#pragma unroll
      for (int i = 0; i < 8; ++i) ss[0] = fmaf(f[i], f[i], ss[0]);
    }
    block_sums(ss, buf[0]);
    rz = rsqrtf(ss[0] / (float)p.H + p.eps);
  }
  if (p.gate_kind == kGateToken) rz *= reinterpret_cast<const float*>(p.gate)[row];
  Vec8<S> sr[VPT];
  float ss[1] = {0.f};
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int v = threadIdx.x + j * blockDim.x;
    sr[j].zero();
    if (v >= nvec) continue;
    float z[8], r[8], w[8];
    zr[j].get(z);
    rr[j].get(r);
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] *= rz;
    Vec8<A> t;
    if (p.norm_w) {
      t.load_weight(p.norm_w, v);
      t.get(w);
#pragma unroll
      for (int i = 0; i < 8; ++i) z[i] *= w[i];
    }
    if (p.gate_kind == kGateFeature || p.gate_kind == kGateFull) {
      t.load(p.gate, (p.gate_kind == kGateFull ? base : 0) + v);
      t.get(w);
#pragma unroll
      for (int i = 0; i < 8; ++i) z[i] *= w[i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = fmaf(p.scale, r[i], z[i]);
    sr[j].set(z);
    if (p.residual_out) sr[j].store(p.residual_out, base + v);
    sr[j].get(z);  // the stored values
#pragma unroll
    for (int i = 0; i < 8; ++i) ss[0] = fmaf(z[i], z[i], ss[0]);
  }
  if (!p.next_w) return;
  block_sums(ss, buf[1]);
  const float rs = rsqrtf(ss[0] / (float)p.H + p.eps);
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int v = threadIdx.x + j * blockDim.x;
    if (v >= nvec) continue;
    float s[8], w[8];
    sr[j].get(s);
    Vec8<A> t;
    t.load_weight(p.next_w, v);
    t.get(w);
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] = s[i] * rs * w[i];
    t.set(s);
    t.store(p.out, base + v);
  }
}

template <typename A, typename S, int VPT>
__global__ void __launch_bounds__(VPT == 1 ? 1024 : 512) block_norm_backward_kernel(BlockNormBackwardParams q) {
  __shared__ float buf[2][3 * 32];
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  const BlockNormParams& p = q.f;
  const int nvec = p.H / 8;
  const float inv_h = 1.f / (float)p.H;
  int turn = 0;
  // this thread's columns of the weight gradients, over the block's rows in order
  float acc_next[VPT][8] = {}, acc_norm[VPT][8] = {}, acc_gate[VPT][8] = {};
  for (size_t row = blockIdx.x; row < (size_t)p.T; row += gridDim.x) {
    const size_t base = row * nvec;
    Vec8<A> zr[VPT], yr[VPT];
    Vec8<S> sr[VPT], gr[VPT];
    float sum[3] = {0.f, 0.f, 0.f};  // z^2, s^2, (dy v) s
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v = threadIdx.x + j * blockDim.x;
      zr[j].zero();
      yr[j].zero();
      sr[j].zero();
      gr[j].zero();
      if (v < nvec) {
        zr[j].load(p.block, base + v);
        if (p.next_w) {
          sr[j].load(p.residual_out, base + v);
          yr[j].load(q.d_out, base + v);
        }
        if (q.d_residual_out) gr[j].load(q.d_residual_out, base + v);
      }
    }
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v = threadIdx.x + j * blockDim.x;
      if (v >= nvec) continue;
      float z[8];
      zr[j].get(z);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[0] = fmaf(z[i], z[i], sum[0]);
      if (p.next_w) {
        float s[8], dy[8], w[8];
        sr[j].get(s);
        yr[j].get(dy);
        Vec8<A> t;
        t.load_weight(p.next_w, v);
        t.get(w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          sum[1] = fmaf(s[i], s[i], sum[1]);
          sum[2] = fmaf(dy[i] * w[i], s[i], sum[2]);
        }
      }
    }
    block_sums(sum, buf[turn ^= 1]);
    const float rz = p.norm_w ? rsqrtf(sum[0] * inv_h + p.eps) : 1.f;
    const float rs = p.next_w ? rsqrtf(sum[1] * inv_h + p.eps) : 0.f;
    const float ms = rs * sum[2] * inv_h;  // mean(dy v s / rms(s))
    const float gt = p.gate_kind == kGateToken ? reinterpret_cast<const float*>(p.gate)[row] : 1.f;
    // pass 2: ds (written scaled as dr), the weight gradients, and sum of ds w z (times
    // the gate where it varies along the row); (ds, and w p for dz, are kept)
    float wp[VPT][8];
    float dot[1] = {0.f};
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v = threadIdx.x + j * blockDim.x;
      if (v >= nvec) continue;
      float z[8], ds[8], w[8];
      zr[j].get(z);
      gr[j].get(ds);
      Vec8<A> t;
      if (p.next_w) {
        float s[8], dy[8];
        sr[j].get(s);
        yr[j].get(dy);
        t.load_weight(p.next_w, v);
        t.get(w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float sn = s[i] * rs;  // no power of rs above the first: rs^3 leaves f32 for large rows
          ds[i] += rs * (dy[i] * w[i] - ms * sn);
          acc_next[j][i] = fmaf(dy[i], sn, acc_next[j][i]);
        }
      }
      if (q.d_residual) {
        float dr[8];
        Vec8<S> o;
#pragma unroll
        for (int i = 0; i < 8; ++i) dr[i] = p.scale * ds[i];
        o.set(dr);
        o.store(q.d_residual, base + v);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = 1.f;
      if (p.norm_w) {
        t.load_weight(p.norm_w, v);
        t.get(w);
      }
      if (p.gate_kind == kGateFeature || p.gate_kind == kGateFull) {
        float g[8], dg[8];
        t.load(p.gate, (p.gate_kind == kGateFull ? base : 0) + v);
        t.get(g);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          dg[i] = ds[i] * (z[i] * rz * w[i]);
          ds[i] *= g[i];
        }
        if (p.gate_kind == kGateFeature) {
#pragma unroll
          for (int i = 0; i < 8; ++i) acc_gate[j][i] += dg[i];
        } else if (q.d_gate) {
          t.set(dg);
          t.store(q.d_gate, base + v);
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        acc_norm[j][i] = fmaf(gt * ds[i], z[i] * rz, acc_norm[j][i]);
        wp[j][i] = ds[i] * w[i];
        dot[0] = fmaf(wp[j][i], z[i], dot[0]);
      }
    }
    if (p.norm_w || p.gate_kind == kGateToken) block_sums(dot, buf[turn ^= 1]);
    if (p.gate_kind == kGateToken && q.d_gate && threadIdx.x == 0)
      reinterpret_cast<float*>(q.d_gate)[row] = rz * dot[0];
    const float mz = p.norm_w ? rz * (gt * dot[0]) * inv_h : 0.f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v = threadIdx.x + j * blockDim.x;
      if (v >= nvec) continue;
      float z[8], dz[8];
      zr[j].get(z);
#pragma unroll
      for (int i = 0; i < 8; ++i) dz[i] = rz * (gt * wp[j][i] - mz * (z[i] * rz));
      Vec8<A> t;
      t.set(dz);
      t.store(q.d_block, base + v);
    }
  }
  float* part = q.partial + (size_t)blockIdx.x * 3 * p.H;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int v = threadIdx.x + j * blockDim.x;
    if (v >= nvec) continue;
    Vec8<float> t;
    if (q.d_next_w) { t.set(acc_next[j]); t.store(part, v); }
    if (q.d_norm_w) { t.set(acc_norm[j]); t.store(part + p.H, v); }
    if (p.gate_kind == kGateFeature && q.d_gate) { t.set(acc_gate[j]); t.store(part + 2 * p.H, v); }
  }
}

// Column sums of the blocks' partial weight gradients, in a fixed order: eight threads
// take the rows of one column in turn, then add in order.
__global__ void __launch_bounds__(256) block_norm_reduce_kernel(const float* partial, int rows, int H, float* d_next,
                                                                 float* d_norm, float* d_gate) {
  __shared__ float buf[8][33];
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  float* const outs[3] = {d_next, d_norm, d_gate};
  float* out = outs[blockIdx.y];
  if (!out) return;
  const int c = blockIdx.x * 32 + tx;
  float v = 0.f;
  if (c < H)
    for (int r = ty; r < rows; r += 8) v += __ldcg(partial + ((size_t)r * 3 + blockIdx.y) * H + c);
  buf[ty][tx] = v;
  __syncthreads();
  if (ty == 0 && c < H) {
#pragma unroll
    for (int i = 1; i < 8; ++i) v += buf[i][tx];
    out[c] = v;
  }
}

template <typename A, typename S>
cudaError_t forward_t(const BlockNormParams& p, cudaStream_t stream) {
  const int nvec = p.H / 8;
  const int threads = (nvec + 31) / 32 * 32;
  return launch_pdl(block_norm_kernel<A, S, 1>, dim3(p.T), dim3(threads), 0, stream, p);
}

template <typename A, typename S>
cudaError_t backward_t(const BlockNormBackwardParams& q, cudaStream_t stream) {
  const int nvec = q.f.H / 8;
  const int threads = (nvec + 31) / 32 * 32;
  cudaError_t e = launch_pdl(block_norm_backward_kernel<A, S, 1>, dim3(q.blocks), dim3(threads), 0, stream, q);
  if (e != cudaSuccess) return e;
  float* d_gate = q.f.gate_kind == kGateFeature ? reinterpret_cast<float*>(q.d_gate) : nullptr;
  if (!q.d_next_w && !q.d_norm_w && !d_gate) return cudaSuccess;
  return launch_pdl(block_norm_reduce_kernel, dim3((q.f.H + 31) / 32, 3), dim3(256), 0, stream, (const float*)q.partial,
                    q.blocks, q.f.H, q.d_next_w, q.d_norm_w, d_gate);
}

}  // namespace

int block_norm_backward_blocks(int T, int) { return T < kNormMaxPartials ? T : kNormMaxPartials; }

cudaError_t launch_block_norm(const BlockNormParams& p, int dtype, int stream_dtype, cudaStream_t stream) {
  if (dtype == kDtypeBf16)
    return stream_dtype == kDtypeF32 ? forward_t<__nv_bfloat16, float>(p, stream)
                                     : forward_t<__nv_bfloat16, __nv_bfloat16>(p, stream);
  return stream_dtype == kDtypeF32 ? forward_t<__half, float>(p, stream) : forward_t<__half, __half>(p, stream);
}

cudaError_t launch_block_norm_backward(const BlockNormBackwardParams& q, int dtype, int stream_dtype,
                                       cudaStream_t stream) {
  if (dtype == kDtypeBf16)
    return stream_dtype == kDtypeF32 ? backward_t<__nv_bfloat16, float>(q, stream)
                                     : backward_t<__nv_bfloat16, __nv_bfloat16>(q, stream);
  return stream_dtype == kDtypeF32 ? backward_t<__half, float>(q, stream) : backward_t<__half, __half>(q, stream);
}

}  // namespace moe
