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
#include <type_traits>

#include "moe_dense.cuh"
#include "sm100_ptx.cuh"

namespace moe {

namespace {

constexpr int kNormSmem = 224 * 1024;  // shared memory that the rows in flight may take

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

// ---- pairs of floats: one instruction per two products (the backward is otherwise bound
// by instructions before memory)
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 make2(float a, float b) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 split2(f32x2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ f32x2 both(float a) { return make2(a, a); }
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
template <typename V>
__device__ __forceinline__ void get2(const V& v, f32x2 (&f)[4]) {
  float t[8];
  v.get(t);
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = make2(t[2 * i], t[2 * i + 1]);
}
template <typename V>
__device__ __forceinline__ void set2(V& v, const f32x2 (&f)[4]) {
  float t[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 q = split2(f[i]);
    t[2 * i] = q.x;
    t[2 * i + 1] = q.y;
  }
  v.set(t);
}

// GATE of a kernel: the gate kind (none and token are one) of a call that has every other
// argument, or kAnyGate, which tests for what is absent.
constexpr int kAnyGate = -1;

// One block per row, eight values a thread: for few rows, where latency is all (one row of
// 2880 bf16 values: 1.9 us a call in a graph).
template <typename A, typename S, int GATE>
__global__ void __launch_bounds__(1024) block_norm_kernel(const __grid_constant__ BlockNormParams p) {
  __shared__ float buf[2][32];
  constexpr bool ANY = GATE == kAnyGate;
  const bool has_norm = !ANY || p.norm_w, has_next = !ANY || p.next_w, has_residual = !ANY || p.residual;
  const bool has_out = !ANY || p.residual_out;
  const bool feature = ANY ? p.gate_kind == kGateFeature : GATE == kGateFeature;
  const bool full = ANY ? p.gate_kind == kGateFull : GATE == kGateFull;
  const bool token = (ANY || GATE == kGateNone) && p.gate_kind == kGateToken;
  const int nvec = p.H / 8, v = threadIdx.x;
  const bool on = v < nvec;
  const size_t row = blockIdx.x, at = row * nvec + v;
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  // everything the row needs, in flight at once
  Vec8<A> zr, wz, wg, wn;
  Vec8<S> rr;
  float gt = 1.f;
  zr.zero();
  rr.zero();
  if (on) {
    zr.load(p.block, at);
    if (has_residual) rr.load(p.residual, at);
    if (has_norm) wz.load_weight(p.norm_w, v);
    if (feature) wg.load_weight(p.gate, v);
    if (full) wg.load(p.gate, at);
    if (has_next) wn.load_weight(p.next_w, v);
  }
  if (token) gt = __ldcg(reinterpret_cast<const float*>(p.gate) + row);
  f32x2 z[4], w[4];
  get2(zr, z);
  float rz = 1.f;
  if (has_norm) {
    f32x2 sq = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) sq = fma2(z[k], z[k], sq);
    const float2 f = split2(sq);
    float ss[1] = {f.x + f.y};
    block_sums(ss, buf[0]);
    rz = rsqrtf(ss[0] / (float)p.H + p.eps);
  }
  const f32x2 g2 = both(rz * gt), a2 = both(p.scale);
#pragma unroll
  for (int k = 0; k < 4; ++k) z[k] = mul2(z[k], g2);
  if (on) {
    if (has_norm) {
      get2(wz, w);
#pragma unroll
      for (int k = 0; k < 4; ++k) z[k] = mul2(z[k], w[k]);
    }
    if (feature || full) {
      get2(wg, w);
#pragma unroll
      for (int k = 0; k < 4; ++k) z[k] = mul2(z[k], w[k]);
    }
    if (has_residual) {
      get2(rr, w);
#pragma unroll
      for (int k = 0; k < 4; ++k) z[k] = fma2(a2, w[k], z[k]);
    }
  }
  Vec8<S> sr;
  set2(sr, z);
  if (on && has_out) sr.store(p.residual_out, at);
  if (!has_next) return;
  get2(sr, z);  // the stored values
  f32x2 sq = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) sq = fma2(z[k], z[k], sq);
  const float2 f = split2(sq);
  float ss[1] = {f.x + f.y};
  block_sums(ss, buf[1]);
  if (!on) return;
  const f32x2 rs = both(rsqrtf(ss[0] / (float)p.H + p.eps));
  get2(wn, w);
#pragma unroll
  for (int k = 0; k < 4; ++k) z[k] = mul2(mul2(z[k], rs), w[k]);
  zr.raw = make_uint4(0, 0, 0, 0);
  set2(zr, z);
  zr.store(p.out, at);
}

// The rows that a block reads in turn, brought to shared memory by bulk copies a few rows
// ahead: row i of the block is in stage i % stages.  A register-only form of the backward
// had the next row's loads wait for the row before it to be finished (8192 x 4096, f32
// stream: 221 us); bulk copies keep the memory busy through the row's two reductions.
struct RowCopies {
  static constexpr int kMax = 5;
  const uint8_t* src[kMax];
  int bytes[kMax];   // of one row; 0: absent
  int offset[kMax];  // in a stage
  int total, stages;
  int threads;       // of one row
};

constexpr uint64_t kRowWaitNs = 1000000000ull;  // a wait may take 1 s
__device__ uint32_t g_norm_status;              // bits as in the layer's status word

__device__ __forceinline__ void issue_row(const RowCopies& c, uint8_t* stage, uint64_t* bar, size_t row) {
  ptx::mbar_arrive_expect_tx(bar, c.total);
#pragma unroll
  for (int i = 0; i < RowCopies::kMax; ++i)
    if (c.bytes[i]) ptx::bulk_load(stage + c.offset[i], c.src[i] + row * c.bytes[i], c.bytes[i], bar);
}

// A copy waited for in vain may still land: report, and stay until it surely has.
__device__ __forceinline__ void leave_late() {
  report_status(&g_norm_status, kStatusTimeoutMain);
  const uint64_t t0 = ptx::globaltimer_ns();
  while (ptx::globaltimer_ns() - t0 < kRowWaitNs / 50) __nanosleep(1000);
}

// Sum of each of eight values over the warp: the lanes halve the values they carry at each
// of the first three butterfly steps (9 exchanges for all eight).  Lane l returns the sum
// of value l / 4.
__device__ __forceinline__ float warp_sums8(float (&v)[8]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int n = 4, bit = 16; n >= 1; n >>= 1, bit >>= 1) {
    const bool up = lane & bit;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float keep = up ? v[i + n] : v[i], send = up ? v[i] : v[i + n];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, send, bit);
    }
  }
  float t = v[0];
  t += __shfl_xor_sync(0xffffffffu, t, 2);
  t += __shfl_xor_sync(0xffffffffu, t, 1);
  return t;
}

// One group of threads per row (8 values a thread), several groups per block where rows
// are narrow.  All six sums of a row are taken in one pass, so that one reduction serves
// it: with G = g w, the sum of ds G z is
//   sum ds' G z + rs (sum u G z - ms rs sum s G z),    u = v dy,  ms = rs mean(u s).
// Rows of up to 4096 values keep the row and the weights in registers (VPT 1); wider ones
// take 16 values a thread and read both twice.  GATE as above: the tests for absent
// arguments alone would be a third of a row's instructions.  Bound by HBM over many rows
// (8192 x 4096 bf16, f32 stream, with the reduction below: 101 us, 6.0 TB/s of a copy's 6.7),
// by the latency of two launches and of a block's rows in turn over few (333 x 2880 f16,
// full gate: 8.7 us).
template <typename A, typename S, int VPT, int GATE>
__global__ void __launch_bounds__(512)
    block_norm_backward_kernel(const __grid_constant__ BlockNormBackwardParams q, const __grid_constant__ RowCopies rows) {
  extern __shared__ __align__(128) uint8_t norm_smem[];
  __shared__ float sums[2][16 * 8];
  __shared__ uint64_t full_bar[kNormMaxGroups][3];
  constexpr bool HOLD = VPT == 1, ANY = GATE == kAnyGate;
  const BlockNormParams& p = q.f;
  const bool has_next = !ANY || p.next_w, has_norm = !ANY || p.norm_w, has_ds = !ANY || q.d_residual_out;
  const bool has_dr = !ANY || q.d_residual;
  const bool feature = ANY ? p.gate_kind == kGateFeature : GATE == kGateFeature;
  const bool full = ANY ? p.gate_kind == kGateFull : GATE == kGateFull;
  const bool token = (ANY || GATE == kGateNone) && p.gate_kind == kGateToken;
  const int nvec = p.H / 8, per = rows.threads, group = threadIdx.x / per, v0 = threadIdx.x - group * per;
  const int groups = blockDim.x / per, warps = per >> 5, warp = v0 >> 5, lane = threadIdx.x & 31;
  const bool leader = v0 == 0;
  const float inv_h = 1.f / (float)p.H;
  uint8_t* const ring = norm_smem + group * rows.stages * rows.total;
  auto barrier = [&]() {
    if (warps > 1)
      asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(per) : "memory");
    else
      __syncwarp();
  };
  if (leader) {
    for (int i = 0; i < rows.stages; ++i) ptx::mbar_init(&full_bar[group][i], 1);
    ptx::fence_mbar_init();
  }
  __syncthreads();
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  const int row0 = blockIdx.x * groups + group, row_step = gridDim.x * groups;
  if (leader)
    for (int i = 0; i < rows.stages; ++i)
      if (row0 + i * row_step < p.T) issue_row(rows, ring + i * rows.total, &full_bar[group][i], row0 + i * row_step);
  const f32x2 zero = 0, one = both(1.f);
  f32x2 wn[4] = {zero, zero, zero, zero}, wz[4] = {one, one, one, one}, wg[4] = {one, one, one, one};
  auto load_weights = [&](int v) {
    Vec8<A> t;
    if (has_next) {
      t.load_weight(p.next_w, v);
      get2(t, wn);
    }
    if (has_norm) {
      t.load_weight(p.norm_w, v);
      get2(t, wz);
    }
    if (feature) {
      t.load_weight(p.gate, v);
      get2(t, wg);
    }
  };
  if (HOLD && v0 < nvec) load_weights(v0);
  f32x2 acc_next[VPT][4] = {}, acc_norm[VPT][4] = {}, acc_gate[VPT][4] = {};  // this thread's columns of the weight gradients
  int stage = 0;
  uint32_t phase = 0;
  int turn = 0;
  bool ok = true;
  for (int row = row0; row < p.T; row += row_step) {
    const uint8_t* st = ring + stage * rows.total;
    if (ok && !ptx::mbar_wait_bounded(&full_bar[group][stage], phase, kRowWaitNs)) ok = false;
    f32x2 z[4] = {}, s[4] = {}, dy[4] = {}, ds[4] = {}, fg[4] = {one, one, one, one};
    auto load_row = [&](int v) {
      Vec8<A> t;
      Vec8<S> o;
      t.load_shared(st + rows.offset[0], v);
      get2(t, z);
      if (has_next) {
        t.load_shared(st + rows.offset[1], v);
        get2(t, dy);
        o.load_shared(st + rows.offset[2], v);
        get2(o, s);
      }
      if (has_ds) {
        o.load_shared(st + rows.offset[3], v);
        get2(o, ds);
      }
      if (full) {
        t.load_shared(st + rows.offset[4], v);
        get2(t, fg);
      }
    };
    f32x2 sum[6] = {};
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v = v0 + j * per;
      if (v >= nvec) break;
      if (!HOLD) load_weights(v);
      load_row(v);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const f32x2 u = mul2(dy[k], wn[k]);
        f32x2 gz = mul2(wz[k], z[k]);
        if (full) gz = mul2(gz, fg[k]);
        if (feature) gz = mul2(gz, wg[k]);
        sum[0] = fma2(z[k], z[k], sum[0]);
        sum[1] = fma2(s[k], s[k], sum[1]);
        sum[2] = fma2(u, s[k], sum[2]);
        sum[3] = fma2(ds[k], gz, sum[3]);
        sum[4] = fma2(u, gz, sum[4]);
        sum[5] = fma2(s[k], gz, sum[5]);
      }
    }
    __syncwarp();
    float tot[8] = {};
#pragma unroll
    for (int k = 0; k < 6; ++k) {
      const float2 f = split2(sum[k]);
      tot[k] = f.x + f.y;
    }
    // the warps' sums, added in a fixed order (lane l: value l % 8)
    float* buf = sums[turn];
    turn ^= 1;  // two buffers in turn, as in block_sums
    const float mine = warp_sums8(tot);
    if ((lane & 3) == 0) buf[(group * warps + warp) * 8 + (lane >> 2)] = mine;
    barrier();
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < 16; w += 4)
      if (w + (lane >> 3) < warps) t += buf[(group * warps + w + (lane >> 3)) * 8 + (lane & 7)];
    t += __shfl_xor_sync(0xffffffffu, t, 8);
    t += __shfl_xor_sync(0xffffffffu, t, 16);
#pragma unroll
    for (int k = 0; k < 6; ++k) tot[k] = __shfl_sync(0xffffffffu, t, k);
    auto refill = [&]() {
      if (leader && ok && row + rows.stages * row_step < p.T)
        issue_row(rows, ring + stage * rows.total, &full_bar[group][stage], row + rows.stages * row_step);
    };
    if (HOLD) refill();  // the whole group is past the barrier, and so past reading the stage
    const float rz = has_norm ? rsqrtf(tot[0] * inv_h + p.eps) : 1.f;
    const float rs = has_next ? rsqrtf(tot[1] * inv_h + p.eps) : 0.f;
    const float ms = rs * tot[2] * inv_h;  // mean(u s / rms(s)): no power of rs above the first leaves f32's range
    const float dot = tot[3] + rs * (tot[4] - ms * (rs * tot[5]));
    const float gt = token ? __ldcg(reinterpret_cast<const float*>(p.gate) + row) : 1.f;
    if (token && q.d_gate && leader) reinterpret_cast<float*>(q.d_gate)[row] = rz * dot;
    const float mz = has_norm ? rz * (gt * dot) * inv_h : 0.f;
    const f32x2 rs2 = both(rs), rz2 = both(rz), nms = both(-ms), nmz = both(-mz), a2 = both(p.scale), gt2 = both(gt);
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v = v0 + j * per;
      if (v >= nvec) break;
      const size_t at = (size_t)row * nvec + v;
      if (!HOLD) {
        load_weights(v);
        load_row(v);
      }
      f32x2 dr[4], dg[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const f32x2 sn = mul2(s[k], rs2), zn = mul2(z[k], rz2);
        const f32x2 d = fma2(rs2, fma2(nms, sn, mul2(dy[k], wn[k])), ds[k]);
        acc_next[j][k] = fma2(dy[k], sn, acc_next[j][k]);
        dr[k] = mul2(a2, d);
        f32x2 dp = mul2(d, gt2);  // one of the gates, the others being 1
        if (feature || full) {
          const f32x2 n = mul2(zn, wz[k]);
          dg[k] = mul2(d, n);
          if (feature) acc_gate[j][k] = fma2(d, n, acc_gate[j][k]);
          dp = mul2(d, full ? fg[k] : wg[k]);
        }
        acc_norm[j][k] = fma2(dp, zn, acc_norm[j][k]);
        z[k] = mul2(rz2, fma2(nmz, zn, mul2(dp, wz[k])));  // dz
      }
      Vec8<A> o;
      Vec8<S> os;
      set2(o, z);
      o.store(q.d_block, at);
      if (has_dr) {
        set2(os, dr);
        os.store(q.d_residual, at);
      }
      if (full && q.d_gate) {
        set2(o, dg);
        o.store(q.d_gate, at);
      }
    }
    if (!HOLD) {
      barrier();  // the whole group has left the stage
      refill();
    }
    if (++stage == rows.stages) {
      stage = 0;
      phase ^= 1;
    }
  }
  if (!ok) leave_late();
  // the groups' sums in order, in shared memory; one row of partial sums per block
  __syncthreads();
  float* red = reinterpret_cast<float*>(norm_smem);
  float* part = q.partial + (size_t)blockIdx.x * 3 * p.H;
  for (int k = 0; k < groups; ++k) {
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v = v0 + j * per;
      if (group != k || v >= nvec) break;
      auto add = [&](int which, f32x2 (&acc)[4]) {
        Vec8<float> t;
        if (k > 0) {
          f32x2 f[4];
          t.load_shared(red + which * p.H, v);
          get2(t, f);
#pragma unroll
          for (int c = 0; c < 4; ++c) acc[c] = fma2(one, f[c], acc[c]);
        }
        set2(t, acc);
        t.store(k + 1 < groups ? red + which * p.H : part + which * p.H, v);
      };
      if (q.d_next_w) add(0, acc_next[j]);
      if (q.d_norm_w) add(1, acc_norm[j]);
      if (feature && q.d_gate) add(2, acc_gate[j]);
    }
    __syncthreads();
  }
}

// The forward over many rows: persistent blocks, groups of threads and row copies as in
// the backward; the weights stay in registers as they were loaded.  Two reductions a row
// (the second is of the rounded stream), each a barrier of the group's own.  Bound by HBM,
// past the first rows' latency: 4096 x 2880 bf16 17.4 us, 5.4 TB/s (a copy: 6.7).
template <typename A, typename S, int GATE>
__global__ void __launch_bounds__(512, 2)
    block_norm_rows_kernel(const __grid_constant__ BlockNormParams p, const __grid_constant__ RowCopies rows) {
  extern __shared__ __align__(128) uint8_t norm_smem[];
  __shared__ float sums[2][16];
  __shared__ uint64_t full_bar[kNormMaxGroups][3];
  const bool token = GATE == kGateNone && p.gate_kind == kGateToken;
  const int nvec = p.H / 8, per = rows.threads, group = threadIdx.x / per, v = threadIdx.x - group * per;
  const int groups = blockDim.x / per, warps = per >> 5, warp = v >> 5, lane = threadIdx.x & 31;
  const bool on = v < nvec, leader = v == 0;
  const float inv_h = 1.f / (float)p.H;
  uint8_t* const ring = norm_smem + group * rows.stages * rows.total;
  auto group_sum = [&](f32x2 sq, float* buf) {
    const float2 f = split2(sq);
    float t = warp_sum_butterfly(f.x + f.y);
    if (warps == 1) return t;
    if (lane == 0) buf[group * warps + warp] = t;
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(per) : "memory");
    return warp_sum_butterfly(lane < warps ? buf[group * warps + lane] : 0.f);
  };
  if (leader) {
    for (int i = 0; i < rows.stages; ++i) ptx::mbar_init(&full_bar[group][i], 1);
    ptx::fence_mbar_init();
  }
  __syncthreads();
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  const int row0 = blockIdx.x * groups + group, row_step = gridDim.x * groups;
  if (leader)
    for (int i = 0; i < rows.stages; ++i)
      if (row0 + i * row_step < p.T) issue_row(rows, ring + i * rows.total, &full_bar[group][i], row0 + i * row_step);
  Vec8<A> wz, wg, wn;
  wz.zero();
  wg.zero();
  wn.zero();
  if (on) {
    wz.load_weight(p.norm_w, v);
    wn.load_weight(p.next_w, v);
    if (GATE == kGateFeature) wg.load_weight(p.gate, v);
  }
  int stage = 0;
  uint32_t phase = 0;
  bool ok = true;
  for (int row = row0; row < p.T; row += row_step) {
    const uint8_t* st = ring + stage * rows.total;
    if (ok && !ptx::mbar_wait_bounded(&full_bar[group][stage], phase, kRowWaitNs)) ok = false;
    Vec8<A> t;
    Vec8<S> r;
    t.zero();
    r.zero();
    if (on) {
      t.load_shared(st + rows.offset[0], v);
      r.load_shared(st + rows.offset[1], v);
      if (GATE == kGateFull) wg.load_shared(st + rows.offset[2], v);
    }
    f32x2 z[4], w[4], sq = 0;
    get2(t, z);
#pragma unroll
    for (int k = 0; k < 4; ++k) sq = fma2(z[k], z[k], sq);
    const float gt = token ? __ldcg(reinterpret_cast<const float*>(p.gate) + row) : 1.f;
    __syncwarp();
    const f32x2 g2 = both(rsqrtf(group_sum(sq, sums[0]) * inv_h + p.eps) * gt), a2 = both(p.scale);
    // (for one warp, the sum's exchanges come after every lane's reads)
    if (leader && ok && row + rows.stages * row_step < p.T)
      issue_row(rows, ring + stage * rows.total, &full_bar[group][stage], row + rows.stages * row_step);
    get2(wz, w);
#pragma unroll
    for (int k = 0; k < 4; ++k) z[k] = mul2(mul2(z[k], g2), w[k]);
    if (GATE == kGateFeature || GATE == kGateFull) {
      get2(wg, w);
#pragma unroll
      for (int k = 0; k < 4; ++k) z[k] = mul2(z[k], w[k]);
    }
    get2(r, w);
#pragma unroll
    for (int k = 0; k < 4; ++k) z[k] = fma2(a2, w[k], z[k]);
    set2(r, z);
    const size_t at = (size_t)row * nvec + v;
    if (on) r.store(p.residual_out, at);
    get2(r, z);  // the stored values
    sq = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) sq = fma2(z[k], z[k], sq);
    const f32x2 rs = both(rsqrtf(group_sum(sq, sums[1]) * inv_h + p.eps));
    get2(wn, w);
#pragma unroll
    for (int k = 0; k < 4; ++k) z[k] = mul2(mul2(z[k], rs), w[k]);
    set2(t, z);
    if (on) t.store(p.out, at);
    if (++stage == rows.stages) {
      stage = 0;
      phase ^= 1;
    }
  }
  if (!ok) leave_late();
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
  // every load at once: a few in turn would each wait for L2
  constexpr int kEach = (kNormBlocks + 7) / 8;
  float part[kEach], v = 0.f;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int r = ty + 8 * i;
    part[i] = r < rows && c < H ? __ldcg(partial + ((size_t)r * 3 + blockIdx.y) * H + c) : 0.f;
  }
#pragma unroll
  for (int i = 0; i < kEach; ++i) v += part[i];
  buf[ty][tx] = v;
  __syncthreads();
  if (ty == 0 && c < H) {
#pragma unroll
    for (int i = 1; i < 8; ++i) v += buf[i][tx];
    out[c] = v;
  }
}

// Threads of one row of the persistent kernels: 8 values each, 16 past 4096 values.
int block_norm_row_threads(int H) { return ((H <= 4096 ? H / 8 : (H / 8 + 1) / 2) + 31) / 32 * 32; }

RowCopies make_rows(int H, int n, const void* const* src, const int* size) {
  RowCopies r{};
  for (int i = 0; i < n; ++i) {
    r.src[i] = static_cast<const uint8_t*>(src[i]);
    r.bytes[i] = src[i] ? H * size[i] : 0;
    r.offset[i] = r.total;
    r.total += r.bytes[i];
  }
  r.threads = block_norm_row_threads(H);
  return r;
}

template <typename A, typename S>
cudaError_t forward_t(const BlockNormParams& p, cudaStream_t stream) {
  const bool every = p.norm_w && p.next_w && p.residual && p.residual_out;
  const int gate = !every ? kAnyGate : p.gate_kind == kGateToken ? kGateNone : p.gate_kind;
  const int row_threads = (p.H / 8 + 31) / 32 * 32, groups = min(512 / row_threads, kNormMaxGroups);
  // many rows: persistent blocks, as many per SM as 56 registers a thread allow, which f16
  // takes at most and bf16 without a feature or full gate does (fewer rows are done sooner by a
  // block each).  With such a gate bf16 takes 58 to 64: at some widths (2880 is one) one block
  // per SM fewer is resident than this asks for, and the last ones run in a second round.
  // Rows of calls without every argument, and of more than 4096 values, have a block each.
  const int per_sm = groups > 0 ? 1152 / (groups * row_threads) : 0, blocks = per_sm * device_sms();
  if (every && groups > 0 && p.T >= 4 * groups * blocks) {
    const void* src[3] = {p.block, p.residual, gate == kGateFull ? p.gate : nullptr};
    const int size[3] = {2, (int)sizeof(S), 2};
    RowCopies r = make_rows(p.H, 3, src, size);
    r.threads = row_threads;
    r.stages = min(3, kNormSmem / per_sm / (groups * r.total));
    static SmemOptIn o[3];
    auto launch = [&](auto kern, SmemOptIn& opt_in) {
      const cudaError_t e = opt_in.ensure(kern, kNormSmem);
      return e != cudaSuccess ? e
                              : launch_pdl(kern, dim3(blocks), dim3(groups * r.threads), groups * r.stages * r.total, stream, p, r);
    };
    if (gate == kGateFeature) return launch(block_norm_rows_kernel<A, S, kGateFeature>, o[0]);
    if (gate == kGateFull) return launch(block_norm_rows_kernel<A, S, kGateFull>, o[1]);
    return launch(block_norm_rows_kernel<A, S, kGateNone>, o[2]);
  }
  auto launch = [&](auto kern) { return launch_pdl(kern, dim3(p.T), dim3(row_threads), 0, stream, p); };
  if (gate == kAnyGate) return launch(block_norm_kernel<A, S, kAnyGate>);
  if (gate == kGateFeature) return launch(block_norm_kernel<A, S, kGateFeature>);
  if (gate == kGateFull) return launch(block_norm_kernel<A, S, kGateFull>);
  return launch(block_norm_kernel<A, S, kGateNone>);
}

template <typename A, typename S>
cudaError_t backward_t(const BlockNormBackwardParams& q, cudaStream_t stream) {
  const void* src[RowCopies::kMax] = {q.f.block, q.f.next_w ? q.d_out : nullptr, q.f.next_w ? q.f.residual_out : nullptr,
                                      q.d_residual_out, q.f.gate_kind == kGateFull ? q.f.gate : nullptr};
  const int size[RowCopies::kMax] = {2, 2, (int)sizeof(S), (int)sizeof(S), 2};
  RowCopies r = make_rows(q.f.H, RowCopies::kMax, src, size);
  const int threads = r.threads;
  const int groups = block_norm_backward_groups(q.f.H);
  // up to three rows in flight per group; and the groups' sums are joined in the same memory
  r.stages = kNormSmem / (groups * r.total);
  if (r.stages > 3) r.stages = 3;
  if (r.stages < 1) return cudaErrorInvalidValue;
  int smem = groups * r.stages * r.total;
  if (groups > 1 && smem < 3 * q.f.H * 4) smem = 3 * q.f.H * 4;
  auto launch = [&](auto kern, SmemOptIn& opt_in) {
    const cudaError_t o = opt_in.ensure(kern, kNormSmem);
    return o != cudaSuccess ? o : launch_pdl(kern, dim3(q.blocks), dim3(groups * threads), smem, stream, q, r);
  };
  static SmemOptIn o[8];
  const bool every = q.f.next_w && q.f.norm_w && q.d_residual_out && q.d_residual;
  const int gate = !every ? kAnyGate : q.f.gate_kind == kGateToken ? kGateNone : q.f.gate_kind;
  auto pick = [&](auto vpt, int at) {
    constexpr int V = decltype(vpt)::value;
    if (gate == kAnyGate) return launch(block_norm_backward_kernel<A, S, V, kAnyGate>, o[at]);
    if (gate == kGateFeature) return launch(block_norm_backward_kernel<A, S, V, kGateFeature>, o[at + 1]);
    if (gate == kGateFull) return launch(block_norm_backward_kernel<A, S, V, kGateFull>, o[at + 2]);
    return launch(block_norm_backward_kernel<A, S, V, kGateNone>, o[at + 3]);
  };
  const cudaError_t e = q.f.H <= 4096 ? pick(std::integral_constant<int, 1>{}, 0) : pick(std::integral_constant<int, 2>{}, 4);
  if (e != cudaSuccess) return e;
  float* d_gate = q.f.gate_kind == kGateFeature ? reinterpret_cast<float*>(q.d_gate) : nullptr;
  if (!q.d_next_w && !q.d_norm_w && !d_gate) return cudaSuccess;
  return launch_pdl(block_norm_reduce_kernel, dim3((q.f.H + 31) / 32, 3), dim3(256), 0, stream, (const float*)q.partial,
                    q.blocks, q.f.H, q.d_next_w, q.d_norm_w, d_gate);
}

}  // namespace

uint32_t* norm_status_word() {
  void* p = nullptr;
  return cudaGetSymbolAddress(&p, g_norm_status) == cudaSuccess ? static_cast<uint32_t*>(p) : nullptr;
}

// Rows that a block takes side by side, and the blocks: one per SM.
int block_norm_backward_groups(int H) {
  const int g = 512 / block_norm_row_threads(H);
  return g > kNormMaxGroups ? kNormMaxGroups : g;
}
int block_norm_backward_blocks(int T, int H) {
  const int need = ceil_div(T, block_norm_backward_groups(H));
  return need < kNormBlocks ? need : kNormBlocks;
}

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
