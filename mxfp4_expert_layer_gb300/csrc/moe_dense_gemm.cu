// Dense GEMMs of the gated feed-forward block and of projections on the 5th-generation tensor cores:
//   forward   gu = x Wgu^T, h = act(g) u (one kernel);  out = h Wd^T
//   backward  dh = dout Wd, with dg = dh u act'(g), du = dh act(g) and h again in its
//             epilogue;  dx = dgu Wgu;  dWgu = dgu^T x;  dWd = dout^T h
// and of projections:  out = act(x W^T + b) + r;  dx = dp W;  dW = dp^T x.
// All are C[m, n] = sum_k A[m, k] B[n, k].  The operands are used as they are stored: a
// matrix whose rows run along K is a K-major operand, one whose rows run along M or N
// an MN-major one (both are forms of the same swizzled shared-memory tile), so nothing
// is transposed in memory.
//
// One persistent block per SM.  Warps 0 and 10 issue the TMA loads of A and of B into a
// ring of stages, warp 1 the MMAs into one of two accumulators in tensor memory, warps
// 2-9 run the epilogue of one tile while the next one's MMAs proceed.  Large products run
// on pairs of SMs (cta_group::2): the pair computes a tile of 256 rows, each SM loading its
// own 128 rows of A and half of B, so the bytes an SM must bring in per MMA are halved
// against a 128-row tile of one SM; the first block of the pair issues the MMAs for both.
// What bounds a large product is the MMAs: 540 cycles a K group of 64 of a 256 x 256 tile
// against their 512 (2048 tokens, 4096 x 14336, forward: 367 us, 1.97 PFLOP/s).
// Sums are f32; g and u are saved in f32 so that the backward's derivatives carry no
// rounding but their own; h, dg and du are rounded to 16 bits because the next
// product's tensor-core operands have that type.
#include <cmath>
#include <utility>
#include "moe_dense.cuh"
#include "sm100_ptx.cuh"

namespace moe {

using namespace ptx;

namespace {

// 16-column steps that the derivative epilogue's g, u come in ahead (forward and backward of
// 2048 tokens x 2880 x 2880: 250 us with one, 242 with two, 276 with three)
constexpr int kAhead = 2;
// kParts epilogue warps per tensor-memory lane quarter (three and four measured no faster:
// what bounds an epilogue is its rows' separate sectors, not its instructions)
constexpr int kEpiWarps = 8, kParts = kEpiWarps / 4;
constexpr int kDenseThreads = 96 + 32 * kEpiWarps;
constexpr uint64_t kDrainLimit = 1000000000ull;  // ns for MMAs already issued (1 s)
constexpr uint64_t kLandingNs = 20000000ull;     // ns after a time-out in which every issued copy has landed (20 ms)

__device__ uint32_t g_dense_status;  // bits as in the layer's status word

// ------------------------------------------------------------------ PTX of CTA pairs
template <bool PAIR>
__device__ __forceinline__ void tmem_alloc_g(uint32_t* dst, uint32_t ncols) {
  if constexpr (PAIR) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(ncols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  } else {
    tmem_alloc(dst, ncols);
    tmem_relinquish();
  }
}
template <bool PAIR>
__device__ __forceinline__ void tmem_dealloc_g(uint32_t taddr, uint32_t ncols) {
  if constexpr (PAIR)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
  else
    tmem_dealloc(taddr, ncols);
}
// Forms that a warp runs in step with one elected lane issuing.  The election is inside
// each: with the loop in one lane's branch, or a predicate of the lane's number, a stage's
// instructions took longer to issue than its MMAs to run (a K group of a 256 x 256 pair
// tile, one warp for all loads: 700 and 640 cycles; elected 560).
#define MOE_ELECTED "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\t@p "
// 2-D tiled load; in a pair the barrier may be the peer's (a cluster address).
template <bool PAIR>
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const void* tmap, uint32_t bar, int32_t c0, int32_t c1) {
  if constexpr (PAIR)
    asm volatile(MOE_ELECTED
                 "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, "
                 "%4}], [%2];\n\t}" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(c0), "r"(c1)
                 : "memory");
  else
    asm volatile(MOE_ELECTED
                 "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], "
                 "[%2];\n\t}" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(c0), "r"(c1)
                 : "memory");
}
template <bool PAIR>
__device__ __forceinline__ void mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  if constexpr (PAIR)
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 q, %4, 0;\n\telect.sync _|p, 0xffffffff;\n\t"
        "@p tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, q;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 q, %4, 0;\n\telect.sync _|p, 0xffffffff;\n\t"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, q;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Arrive on `bar` -- in a pair on both blocks' barrier of that offset -- when the MMAs
// issued so far are done.
template <bool PAIR>
__device__ __forceinline__ void commit(uint64_t* bar) {
  if constexpr (PAIR)
    asm volatile(MOE_ELECTED
                 "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(
                     smem_u32(bar)),
                 "h"((uint16_t)3)
                 : "memory");
  else
    asm volatile(MOE_ELECTED "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
                     smem_u32(bar))
                 : "memory");
}
// The same on this block's barrier alone.
template <bool PAIR>
__device__ __forceinline__ void commit_own(uint64_t* bar) {
  if constexpr (PAIR)
    asm volatile(MOE_ELECTED "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
                     smem_u32(bar))
                 : "memory");
  else
    commit<false>(bar);
}
#undef MOE_ELECTED
// A bounded wait of a whole warp, in step; the answer is the same in every lane.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, uint64_t limit_ns) {
  const bool ok = mbar_wait_bounded(bar, parity, limit_ns);
  return __all_sync(0xffffffffu, ok);
}
// A wait gave up: in the status word, and for this launch in the block's own flag.
__device__ __forceinline__ void give_up(volatile uint32_t* late, uint32_t bits) {
  if ((threadIdx.x & 31) == 0) {
    report_status(&g_dense_status, bits);
    *late = 1;
  }
}
__device__ __forceinline__ void st_cluster_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// The values of a tensor-memory load, once it has been waited for: the registers pass through
// an empty statement behind the wait, so that no use of them can move ahead of it.
__device__ __forceinline__ void landed(uint32_t (&r)[16], float (&f)[16]) {
  asm volatile("" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                    "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]));
#pragma unroll
  for (int i = 0; i < 16; ++i) f[i] = __uint_as_float(r[i]);
}

// A whole 32-byte sector per thread: with 16-byte accesses of a thread per row, every
// sector would be asked for twice.
struct Sector {
  uint32_t w[8];
};
__device__ __forceinline__ void store_sector(void* p, const Sector& s) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(s.w[0]), "r"(s.w[1]), "r"(s.w[2]),
               "r"(s.w[3]), "r"(s.w[4]), "r"(s.w[5]), "r"(s.w[6]), "r"(s.w[7])
               : "memory");
}
__device__ __forceinline__ void load_sector(float* f, const float* p) {
  asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3]), "=f"(f[4]), "=f"(f[5]), "=f"(f[6]), "=f"(f[7])
               : "l"(p));
}
// 16 (or, at the end of a row, 8) values of a row, rounded to 16 bits.
template <typename X>
__device__ __forceinline__ void store16(X* p, const float* v, int n) {
  Sector s;
#pragma unroll
  for (int i = 0; i < 8; ++i) s.w[i] = pack2<X>(v[2 * i], v[2 * i + 1]);
  if (n >= 16 && (reinterpret_cast<uintptr_t>(p) & 31) == 0) {
    store_sector(p, s);
  } else {
    reinterpret_cast<uint4*>(p)[0] = make_uint4(s.w[0], s.w[1], s.w[2], s.w[3]);
    if (n >= 16) reinterpret_cast<uint4*>(p)[1] = make_uint4(s.w[4], s.w[5], s.w[6], s.w[7]);
  }
}
// 8 values in 32 bits (f32 rows of a multiple of 8 values: sectors are aligned where the
// array is).
__device__ __forceinline__ void store8(float* p, const float* v) {
  if ((reinterpret_cast<uintptr_t>(p) & 31) == 0) {
    Sector s;
#pragma unroll
    for (int i = 0; i < 8; ++i) s.w[i] = __float_as_uint(v[i]);
    store_sector(p, s);
  } else {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}
__device__ __forceinline__ void load8(float* f, const float* p) {
  if ((reinterpret_cast<uintptr_t>(p) & 31) == 0) {
    load_sector(f, p);
  } else {
    Vec8<float> t;
    t.load(p, 0);
    float v[8];
    t.get(v);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = v[i];
  }
}

// ------------------------------------------------------------------ configuration
template <int BN, bool PAIR>
struct DenseCfg {
  static constexpr int kCtas = PAIR ? 2 : 1;
  static constexpr int kTileM = 128 * kCtas;
  static constexpr int kABytes = 128 * 128, kBBytes = BN / kCtas * 128;  // of B in this block's shared memory
  static constexpr int kGroupBytes = kABytes + kBBytes;  // of one K group (64 values)
  // K groups per stage: a stage's waits and commits cost 440 cycles, more than the MMAs of a
  // small tile's group (2048 tokens in 64-column tiles: 1215 us by one, 921 by two); a pair's
  // tiles need the finer ring more (1001 tokens x 2880 x 2880: 44.0 us by one, 47.5 by two)
  static constexpr int kGroups = PAIR ? 1 : 2;
  static constexpr int kStages = 196608 / (kGroups * kGroupBytes);
  static constexpr int kSmemBytes = kStages * kGroups * kGroupBytes + 1024;
  static constexpr int kTmemCols = 2 * BN < 32 ? 32 : 2 * BN;
  static_assert(kTmemCols <= 512 && (kTmemCols & (kTmemCols - 1)) == 0, "tensor memory columns");
};

// Work units: the first `full` tiles whole, each tile after them in `splits` K slices (the
// last round of tiles, when it would leave most SMs idle).  Tiles in groups of kRasterM
// row tiles, the row tile running fastest inside a group, so the tiles in flight at one
// time share both operands through L2.
constexpr int kRasterM = 8;
struct Unit {
  int g, m, n, slot, k0, k1;  // product; slot: place of the slice's partial sums, or -1
};
__device__ __forceinline__ void map_tile(const DenseProblem& g, int u, Unit& r) {
  const int first = u / (kRasterM * g.tiles_n) * kRasterM;
  const int rows = min(kRasterM, g.tiles_m - first);
  const int within = u - first * g.tiles_n;
  r.n = within / rows;
  r.m = first + within - r.n * rows;
}
__device__ __forceinline__ Unit map_unit(const DenseGemmParams& p, int u) {
  Unit r;
  r.g = 0;
  r.slot = u - p.full;
  r.k0 = 0;
  r.k1 = p.g[0].kgroups;
  if (r.slot < 0) {
    r.slot = -1;
  } else if (p.splits > 1) {
    const int split = r.slot % p.splits;
    u = p.full + r.slot / p.splits;
    r.k0 = (int)((long long)split * p.g[0].kgroups / p.splits);
    r.k1 = (int)((long long)(split + 1) * p.g[0].kgroups / p.splits);
  }
  map_tile(p.g[0], u, r);
  return r;
}

// The units of one worker (a block, or a pair): every `workers`-th.  Several products: the
// tiles of the long class (the larger K) in turn; then, while the workers that got one more
// of those are still at it, each of the others takes `lead` tiles of the short class; then
// all take the rest of it in turn, the earlier ones first.  So the products end together,
// where each by itself would leave part of its last round's SMs idle.
template <bool GROUP>
struct Units {
  const DenseGemmParams& p;
  const int worker, workers;
  int u, end, step, phase;
  int n_long, n_short, more, head;  // tiles of the classes; workers with one more long tile; tiles taken in the lead
  __device__ __forceinline__ Units(const DenseGemmParams& q, int w, int ws) : p(q), worker(w), workers(ws), phase(0) {
    u = worker;
    step = workers;
    if constexpr (GROUP) {
      n_long = n_short = 0;
      for (int i = 0; i < p.group; ++i) (i < p.long_n ? n_long : n_short) += p.g[i].tiles_m * p.g[i].tiles_n;
      more = n_long % workers;
      head = more > 0 ? min(n_short, (workers - more) * p.lead) : 0;
      end = n_long;
      settle();
    } else {
      end = p.full + (p.g[0].tiles_m * p.g[0].tiles_n - p.full) * p.splits;
    }
  }
  __device__ __forceinline__ void settle() {
    while (u >= end && phase < 2) {
      if (++phase == 1) {
        u = worker >= more ? worker - more : head;
        end = head;
        step = workers - more;
      } else if (n_short > 0) {
        const bool late_first = (long long)p.lead * p.g[p.long_n].kgroups > p.g[0].kgroups;
        u = head + (late_first || more == 0 ? worker : worker >= more ? worker - more : worker + workers - more);
        end = n_short;
        step = workers;
      }
    }
  }
  __device__ __forceinline__ bool on() const { return u < end; }
  __device__ __forceinline__ void next() {
    u += step;
    if constexpr (GROUP) settle();
  }
  __device__ __forceinline__ Unit get() const {
    if constexpr (GROUP) {
      Unit r;
      int at = u;
      r.g = phase == 0 ? 0 : p.long_n;
      for (; at >= p.g[r.g].tiles_m * p.g[r.g].tiles_n; ++r.g) at -= p.g[r.g].tiles_m * p.g[r.g].tiles_n;
      r.slot = -1;
      r.k0 = 0;
      r.k1 = p.g[r.g].kgroups;
      map_tile(p.g[r.g], at, r);
      return r;
    } else {
      return map_unit(p, u);
    }
  }
};

// g and u of W columns of a row.
template <int W>
__device__ __forceinline__ void load_gateup(const DenseGemmParams& p, const DenseProblem& c, int m, int n, int left,
                                            float (&g)[W], float (&u)[W]) {
  const float* gu = p.gateup + (size_t)m * 2 * c.N + n;
#pragma unroll
  for (int j = 0; j < W; j += 8)
    if (j < left) {
      load8(&g[j], gu + j);
      load8(&u[j], gu + c.N + j);
    }
}
// dh, g, u -> dg, du, h.
template <typename X, int W>
__device__ __forceinline__ void epilogue_grad(const DenseGemmParams& p, const DenseProblem& c, int m, int n, int left,
                                              float (&v)[W], float (&g)[W], float (&u)[W]) {
  X* dg = reinterpret_cast<X*>(c.out) + (size_t)m * 2 * c.N + n;
  X* hh = reinterpret_cast<X*>(p.out_h) + (size_t)m * c.N + n;
  auto grad = [&](auto tag) {
#pragma unroll
    for (int j = 0; j < W; ++j) {
      float slope;
      const float gj = g[j], uj = u[j], a = act_f<decltype(tag)::value>(gj, slope);
      g[j] = v[j] * uj * slope;
      u[j] = v[j] * a;
      v[j] = a * uj;
    }
  };
  if (p.act == kActSilu)
    grad(std::integral_constant<int, kActSilu>{});
  else
    grad(std::integral_constant<int, kActGelu>{});
#pragma unroll
  for (int j = 0; j < W; j += 16)
    if (j < left) {
      store16(dg + j, &g[j], left - j);
      store16(dg + c.N + j, &u[j], left - j);
      store16(hh + j, v + j, left - j);
    }
}

// Sums of 16 columns of a projection -> act(v + bias) + residual, in out's type O (16 bits or
// f32), and v + bias in f32 where it is kept.  The residual's element and out's may be one.
template <typename O, int W>
__device__ __forceinline__ void load_out(const O* p, int left, float (&f)[W]) {
  // (a whole sector a thread, as load_sector; through L2 only, as the array may be out itself)
  if (left >= 16 && (reinterpret_cast<uintptr_t>(p) & 31) == 0) {
    uint32_t w[sizeof(O) * W / 4];
#pragma unroll
    for (int j = 0; j < (int)(sizeof(O) * W / 32); ++j)
      asm volatile("ld.global.cg.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=r"(w[8 * j]), "=r"(w[8 * j + 1]), "=r"(w[8 * j + 2]), "=r"(w[8 * j + 3]), "=r"(w[8 * j + 4]),
                     "=r"(w[8 * j + 5]), "=r"(w[8 * j + 6]), "=r"(w[8 * j + 7])
                   : "l"(reinterpret_cast<const uint32_t*>(p) + 8 * j));
    if constexpr (std::is_same<O, float>::value) {
#pragma unroll
      for (int i = 0; i < W; ++i) f[i] = __uint_as_float(w[i]);
    } else {
#pragma unroll
      for (int i = 0; i < W / 2; ++i) {
        const float2 v = unpack2<O>(w[i]);
        f[2 * i] = v.x;
        f[2 * i + 1] = v.y;
      }
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < W; j += 8)
    if (j < left) {
      Vec8<O> t;
      float v[8];
      t.load(p + j, 0);
      t.get(v);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[j + i] = v[i];
    }
}
template <typename O>
__device__ __forceinline__ void store_out(O* p, const float* v, int n) {
  if constexpr (std::is_same<O, float>::value) {
    store8(p, v);
    if (n >= 16) store8(p + 8, v + 8);
  } else {
    store16(p, v, n);
  }
}
template <typename O>
__device__ __forceinline__ void epilogue_linear(const DenseGemmParams& p, const DenseProblem& c, int m, int n, int left,
                                                float (&v)[16], const float (&r)[16], const float (&b)[16]) {
  if (left <= 0) return;
#pragma unroll
  for (int j = 0; j < 16; ++j) v[j] += b[j];
  if (p.gateup) store_out(p.gateup + (size_t)m * c.N + n, v, left);
  if (p.act == kActSilu) {
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] = act_f<kActSilu>(v[j]);
  } else if (p.act == kActGelu) {
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] = act_f<kActGelu>(v[j]);
  }
  if (p.residual) {
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] += r[j];
  }
  store_out(reinterpret_cast<O*>(c.out) + (size_t)m * c.N + n, v, left);
}
// The residual of 16 columns of a row.
template <typename O>
__device__ __forceinline__ void load_residual(const DenseGemmParams& p, const DenseProblem& c, int m, int n, int left,
                                              float (&r)[16]) {
  if (p.residual) load_out(reinterpret_cast<const O*>(p.residual) + (size_t)m * c.N + n, left, r);
}
// The same from a split tile's joined sums.
template <typename O>
__device__ __forceinline__ void epilogue_joined(const DenseGemmParams& p, const DenseProblem& c, int m, int n, int left,
                                                float (&v)[16]) {
  float r[16] = {}, b[16] = {};
  load_residual<O>(p, c, m, n, left, r);
  if (p.bias) load_out(p.bias + n, left, b);
  epilogue_linear<O>(p, c, m, n, left, v, r, b);
}

// What happens to the sums of W columns of a row (`left` of them inside the matrix, in
// eights): v, and for gate/up w the up sums.
template <typename X, int MODE, int W>
__device__ __forceinline__ void epilogue(const DenseGemmParams& p, const DenseProblem& c, int m, int n, int left, float (&v)[W],
                                         float (&w)[W]) {
  X* out = reinterpret_cast<X*>(c.out);
  if constexpr (MODE == kDenseStore || MODE == kDenseProducts) {
#pragma unroll
    for (int j = 0; j < W; j += 16)
      if (j < left) store16(out + (size_t)m * c.N + n + j, v + j, left - j);
  } else if constexpr (MODE == kDenseLinear) {
    epilogue_joined<X>(p, c, m, n, left, v);
  } else if constexpr (MODE == kDenseLinear32) {
    epilogue_joined<float>(p, c, m, n, left, v);
  } else if constexpr (MODE == kDenseGateUp) {
    if (p.gateup) {
      float* gu = p.gateup + (size_t)m * 2 * c.N + n;
#pragma unroll
      for (int j = 0; j < W; j += 8)
        if (j < left) {
          store8(gu + j, v + j);
          store8(gu + c.N + j, w + j);
        }
    }
    if (p.act == kActSilu) {
#pragma unroll
      for (int j = 0; j < W; ++j) v[j] = act_f<kActSilu>(v[j]) * w[j];
    } else {
#pragma unroll
      for (int j = 0; j < W; ++j) v[j] = act_f<kActGelu>(v[j]) * w[j];
    }
#pragma unroll
    for (int j = 0; j < W; j += 16)
      if (j < left) store16(out + (size_t)m * c.N + n + j, v + j, left - j);
  } else {
    float g[W], u[W];
    load_gateup(p, c, m, n, left, g, u);
    epilogue_grad<X>(p, c, m, n, left, v, g, u);
  }
}

template <typename X, int MODE, int BN, bool PAIR>
__global__ void __launch_bounds__(kDenseThreads, 1) dense_gemm_kernel(const __grid_constant__ DenseGemmParams p) {
  using C = DenseCfg<BN, PAIR>;
  constexpr bool kMany = MODE == kDenseProducts;
  extern __shared__ uint8_t dense_smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dense_smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t full_bar[C::kStages], empty_bar[C::kStages], accf_bar[2], acce_bar[2], drain_bar;
  __shared__ uint32_t tmem_slot;
  constexpr bool kLinear = MODE == kDenseLinear || MODE == kDenseLinear32;
  __shared__ __align__(16) float bias_s[kLinear ? kEpiWarps : 1][kLinear ? BN : 4];  // each epilogue warp's copy of a tile's
  __shared__ volatile uint32_t late;  // a wait of this launch gave up, in this block or its peer
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = PAIR ? cluster_rank() : 0u;
  const int bn = PAIR ? p.bn : BN;  // columns of a tile
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&accf_bar[b], 1);
      mbar_init(&acce_bar[b], kEpiWarps * C::kCtas);  // one lane of each epilogue warp
    }
    mbar_init(&drain_bar, 1);
    late = 0;
    fence_mbar_init();
    for (int i = 0; i < (kMany ? p.group : 1); ++i) {
      tma_prefetch_desc(&p.g[i].tm_a);
      tma_prefetch_desc(&p.g[i].tm_b);
    }
  }
  if (warp == 1) tmem_alloc_g<PAIR>(&tmem_slot, C::kTmemCols);
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) {  // the peer's barriers exist before anything arrives on them
    cluster_arrive_release();
    cluster_wait_acquire();
  }
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  pdl_wait();
  pdl_launch_dependents();

  Units<kMany> it(p, blockIdx.x / C::kCtas, gridDim.x / C::kCtas);

  if (warp == 0 || warp == 2 + kEpiWarps) {
    // ------------------------------------------------------------ TMA producers
    // (whole warps, in step) one of A, one of B: issuing a load takes about 125 cycles and
    // a stage's wait 190, so one warp for both could not keep up with the MMAs.
    // The pair's copies all count on one barrier.
    const bool of_b = warp != 0;
    const int b_cols = bn / C::kCtas;
    const uint32_t tx = (uint32_t)(C::kABytes + b_cols * 128) * C::kCtas;
    const uint32_t full0 = PAIR ? mapa_shared(smem_u32(full_bar), 0) : smem_u32(full_bar);
    const uint32_t base = smem_u32(smem) + (of_b ? C::kABytes : 0);
    int s = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (; it.on() && ok; it.next()) {
      const Unit w = it.get();
      const DenseProblem& g = p.g[kMany ? w.g : 0];
      const int m0 = w.m * C::kTileM + (int)rank * 128, nt = w.n;
      for (int k0 = w.k0; k0 < w.k1; k0 += C::kGroups) {
        if (!wait_warp(&empty_bar[s], phase ^ 1, p.wait_ns)) {
          give_up(&late, kStatusTimeoutProducer);
          ok = false;
          break;
        }
        const int n = min(C::kGroups, w.k1 - k0);
        const uint32_t bar = full0 + 8 * s;
        if (!of_b) mbar_arrive_expect_tx_if(lane == 0 && rank == 0, &full_bar[s], tx * n);
#pragma unroll
        for (int j = 0; j < C::kGroups; ++j) {
          if (j >= n) break;
          const int k = (k0 + j) * 64;
          const uint32_t dst = base + (s * C::kGroups + j) * C::kGroupBytes;
          if (!of_b) {
            if (g.a_mn) {
#pragma unroll
              for (int c = 0; c < 2; ++c) tma_load_2d<PAIR>(dst + c * 8192, &g.tm_a, bar, m0 + 64 * c, k);
            } else {
              tma_load_2d<PAIR>(dst, &g.tm_a, bar, k, m0);
            }
          } else if (g.b_mn) {
            const int n0 = nt * bn + (int)rank * b_cols;
            for (int c = 0; c < b_cols / 64; ++c) tma_load_2d<PAIR>(dst + c * 8192, &g.tm_b, bar, n0 + 64 * c, k);
          } else {
            // gate then up features; or this block's columns in one box
#pragma unroll
            for (int c = 0; c < (MODE == kDenseGateUp ? 2 / C::kCtas : 1); ++c) {
              const int row =
                  MODE == kDenseGateUp ? (PAIR ? (int)rank : c) * g.N + nt * (bn / 2) : nt * bn + (int)rank * b_cols;
              tma_load_2d<PAIR>(dst + c * (bn / 2) * 128, &g.tm_b, bar, k, row);
            }
          }
        }
        if (++s == C::kStages) {
          s = 0;
          phase ^= 1;
        }
      }
    }
    // the MMAs' arrivals on the second block's barriers are all there before it leaves
    if (PAIR && !of_b)
      for (int i = 0; i < C::kStages && ok; ++i) {
        ok = wait_warp(&empty_bar[s], phase ^ 1, p.wait_ns);
        if (!ok) give_up(&late, kStatusTimeoutProducer);
        if (++s == C::kStages) {
          s = 0;
          phase ^= 1;
        }
      }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    // (the whole warp, in step)
    if (rank == 0) {
      constexpr uint32_t kFmt = std::is_same<X, __half>::value ? 0u : 1u;  // operand format: f16 0, bf16 1
      int s = 0, i = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (; it.on() && ok; it.next(), ++i) {
        const Unit w = it.get();
        const DenseProblem& g = p.g[kMany ? w.g : 0];
        const uint32_t idesc = (1u << 4) | (kFmt << 7) | (kFmt << 10) | ((uint32_t)g.a_mn << 15) | ((uint32_t)g.b_mn << 16) |
                               ((uint32_t)(bn >> 3) << 17) | ((uint32_t)(C::kTileM >> 4) << 24);
        // K major: rows of 128 bytes in groups of 8 (1024 bytes), 32 bytes per K = 16 step.
        // MN major: 64 K rows of 128 bytes (64 values) per 8192-byte chunk, 8 K rows per
        // 1024 bytes, 2048 bytes per K = 16 step.
        const uint32_t a_step = g.a_mn ? 128 : 2, b_step = g.b_mn ? 128 : 2;  // in 16 bytes
        const uint64_t a_desc = smem_desc(smem_u32(smem), g.a_mn ? 8192 : 16, 1024, 2);
        const uint64_t b_desc = smem_desc(smem_u32(smem) + C::kABytes, g.b_mn ? 8192 : 16, 1024, 2);
        const int b = i & 1;
        const bool free = PAIR ? __all_sync(0xffffffffu, mbar_wait_cluster_bounded(&acce_bar[b], ((i >> 1) & 1) ^ 1, p.wait_ns))
                               : wait_warp(&acce_bar[b], ((i >> 1) & 1) ^ 1, p.wait_ns);
        if (!free) {
          give_up(&late, kStatusTimeoutMain);
          break;
        }
        tc_fence_after();
        const uint32_t acc = tmem + b * BN;
        for (int k0 = w.k0; k0 < w.k1; k0 += C::kGroups) {
          if (!wait_warp(&full_bar[s], phase, p.wait_ns)) {
            give_up(&late, kStatusTimeoutMain);
            ok = false;
            break;
          }
          tc_fence_after();
          const int n = min(C::kGroups, w.k1 - k0);
#pragma unroll
          for (int j = 0; j < C::kGroups; ++j) {
            if (j >= n) break;
            const uint64_t at = (uint64_t)((s * C::kGroups + j) * (C::kGroupBytes / 16));
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              mma_f16<PAIR>(acc, a_desc + at + (uint64_t)(a_step * ks), b_desc + at + (uint64_t)(b_step * ks), idesc,
                            k0 > w.k0 || j > 0 || ks > 0 ? 1u : 0u);
          }
          commit<PAIR>(&empty_bar[s]);
          if (++s == C::kStages) {
            s = 0;
            phase ^= 1;
          }
        }
        if (ok) commit<PAIR>(&accf_bar[b]);
      }
      // all tensor-core work is done before the tensor memory is freed (known to this block
      // alone: nothing would keep the second one until an arrival of its own)
      commit_own<PAIR>(&drain_bar);
      wait_warp(&drain_bar, 0, kDrainLimit);
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3, part0 = 16 * ((warp - 2) >> 2);  // tensor-memory lane quarter; its first columns
    int i = 0;
    for (; it.on(); it.next(), ++i) {
      const Unit t = it.get();
      const DenseProblem& g = p.g[kMany ? t.g : 0];
      const int b = i & 1;
      const int r = (int)rank * 128 + q * 32 + lane, m = t.m * C::kTileM + r;  // row in the tile, in the matrix
      const bool live = m < g.M;
      // the first g, u come in while the MMAs run
      const int cols = MODE == kDenseGateUp ? bn / 2 : bn;
      constexpr bool kGrad = MODE == kDenseGateUpGrad;
      constexpr int kStep = 16 * kParts;  // a warp takes 16 columns of every kStep
      const int n0 = t.n * cols, end = min(g.N - n0, cols);
      float gs[kGrad ? kAhead + 1 : 1][16], us[kGrad ? kAhead + 1 : 1][16];
      if constexpr (kGrad)
        if (live && t.slot < 0) {
#pragma unroll
          for (int j = 0; j < kAhead; ++j) {
            const int c = part0 + kStep * j;
            load_gateup(p, g, m, n0 + c, end - c, gs[j], us[j]);
          }
        }
      // a projection's bias, and the first of its residual
      using O = std::conditional_t<MODE == kDenseLinear32, float, X>;
      float rs[kLinear ? kAhead + 1 : 1][16];
      if constexpr (kLinear)
        if (t.slot < 0) {
          float* b = bias_s[warp - 2];
          for (int j = lane; j < cols; j += 32) b[j] = p.bias && j < end ? __ldcg(p.bias + n0 + j) : 0.f;
          if (live) {
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
              const int c = part0 + kStep * j;
              load_residual<O>(p, g, m, n0 + c, end - c, rs[j]);
            }
          }
          __syncwarp();
        }
      // (one answer for the warp: its lanes leave together, or all go on to the warp's
      // tensor-memory loads)
      if (!wait_warp(&accf_bar[b], (i >> 1) & 1, p.wait_ns)) {
        give_up(&late, kStatusTimeoutEpi);
        break;
      }
      tc_fence_after();
      const uint32_t acc = tmem + ((uint32_t)(q * 32) << 16) + b * BN;
      if (!kMany && t.slot >= 0 && p.splits > 1) {
        // a K slice's sums as they are: [slot][row of the tile][bn]
        float* part = p.partial + ((size_t)t.slot * C::kTileM + r) * bn;
#pragma unroll 1
        for (int c = part0; c < bn; c += kStep) {
          uint32_t raw[16];
          float v[16];
          tmem_ld_32x32b_x16(acc + c, raw);
          tmem_wait_ld();
          landed(raw, v);
          if (live) {
#pragma unroll
            for (int j = 0; j < 16; j += 8) store8(part + c + j, v + j);
          }
          __syncwarp();  // the next tensor-memory load is the whole warp's
        }
      } else if constexpr (kGrad) {
        // 16 columns at a time, the g, u of the next kAhead times on their way meanwhile
#pragma unroll 1
        for (int c0 = part0; c0 < cols; c0 += kStep * (kAhead + 1))
#pragma unroll
          for (int j = 0; j <= kAhead; ++j) {
            const int c = c0 + kStep * j;
            if (c >= cols) break;
            constexpr int kAll = kAhead + 1;
            const int next = c + kStep * kAhead;
            if (live) load_gateup(p, g, m, n0 + next, end - next, gs[(j + kAhead) % kAll], us[(j + kAhead) % kAll]);
            uint32_t raw[16];
            float v[16];
            tmem_ld_32x32b_x16(acc + c, raw);
            tmem_wait_ld();
            landed(raw, v);
            if (live && c < end) epilogue_grad<X>(p, g, m, n0 + c, end - c, v, gs[j], us[j]);
            __syncwarp();
          }
      } else if constexpr (kLinear) {
        // as above, with the residual; its loads in step with the arithmetic cost a memory round
        // trip each (2048 x 4096 -> 4096 onto f32: 54 us)
        const float* bias = bias_s[warp - 2];
#pragma unroll 1
        for (int c0 = part0; c0 < cols; c0 += kStep * (kAhead + 1))
#pragma unroll
          for (int j = 0; j <= kAhead; ++j) {
            const int c = c0 + kStep * j;
            if (c >= cols) break;
            constexpr int kAll = kAhead + 1;
            const int next = c + kStep * kAhead;
            if (live) load_residual<O>(p, g, m, n0 + next, end - next, rs[(j + kAhead) % kAll]);
            uint32_t raw[16];
            float v[16], b[16];
            tmem_ld_32x32b_x16(acc + c, raw);
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
              const float4 q4 = *reinterpret_cast<const float4*>(bias + c + i);
              b[i] = q4.x; b[i + 1] = q4.y; b[i + 2] = q4.z; b[i + 3] = q4.w;
            }
            tmem_wait_ld();
            landed(raw, v);
            if (live && c < end) epilogue_linear<O>(p, g, m, n0 + c, end - c, v, rs[j], b);
            __syncwarp();
          }
      } else {
#pragma unroll 1
        for (int c = part0; c < cols; c += kStep) {
          uint32_t raw[16], raw_up[16];
          float v[16], w[16];
          tmem_ld_32x32b_x16(acc + c, raw);
          if constexpr (MODE == kDenseGateUp) tmem_ld_32x32b_x16(acc + bn / 2 + c, raw_up);
          tmem_wait_ld();
          landed(raw, v);
          if constexpr (MODE == kDenseGateUp) landed(raw_up, w);
          if (live) epilogue<X, MODE, 16>(p, g, m, n0 + c, end - c, v, w);  // end - c: a multiple of 8
          __syncwarp();
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (PAIR)
          mbar_arrive_cluster(mapa_shared(smem_u32(&acce_bar[b]), 0));
        else
          mbar_arrive(&acce_bar[b]);
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) {  // neither block's memory goes while the other may still use it
    if (threadIdx.x == 0 && late) st_cluster_u32(mapa_shared(smem_u32(const_cast<uint32_t*>(&late)), rank ^ 1), 1);
    __syncwarp();
    cluster_arrive_release();
    cluster_wait_acquire();
  }
  tc_fence_after();
  // Ordinarily every copy has been consumed by now.  After a time-out of either block some
  // may still be on their way: stay until they have surely landed.
  if (threadIdx.x == 0 && late) {
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < kLandingNs) __nanosleep(1000);
  }
  __syncthreads();
  if (warp == 1) tmem_dealloc_g<PAIR>(tmem, C::kTmemCols);
}

// ------------------------------------------------------------------ projections of a batch
// Up to 128 tokens: the weights' rows (for the gradient into x, their columns: an MN-major
// operand) are the MMA's M, the tokens its N, so that every SM
// streams weights and the results of a warp are neighbours in memory.  A block takes 128 rows;
// the blocks of a cluster split K and push their sums, by token, into the shared memory of the
// block that finishes the token (added there in rank order): one launch where the tiles above
// need a second one to join their K slices.
template <int TN>
struct BatchCfg {
  static constexpr int kStageBytes = 16384 + TN * 128;  // 64 values of K
  static constexpr int kStages = TN == 128 ? 4 : TN == 64 ? 3 : 4;
  static constexpr int kSumBytes = TN * 128 * 4;
  static constexpr int kSmemBytes = kStages * kStageBytes + kSumBytes + 1024;
  static constexpr int kPerSm = TN == 128 ? 1 : 2;
};
constexpr int kBatchEpiWarps = 8, kBatchThreads = 64 + 32 * kBatchEpiWarps, kBatchMaxSplit = 8;

template <typename X, int TN, bool WIDE>
__global__ void __launch_bounds__(kBatchThreads, BatchCfg<TN>::kPerSm) linear_batch_kernel(const __grid_constant__ DenseGemmParams p) {
  using C = BatchCfg<TN>;
  using O = std::conditional_t<WIDE, float, X>;
  extern __shared__ uint8_t dense_smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dense_smem_raw) + 1023) & ~uintptr_t(1023));
  float* const sums = reinterpret_cast<float*>(smem + C::kStages * C::kStageBytes);  // [split][token of this block's][row]
  __shared__ uint64_t full_bar[C::kStages], empty_bar[C::kStages], acc_bar;
  __shared__ uint32_t tmem_slot;
  __shared__ volatile uint32_t late;
  const DenseProblem& g = p.g[0];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, S = p.splits;
  const int rank = S > 1 ? (int)cluster_rank() : 0, tile = blockIdx.x / S;
  const int k0 = (int)((long long)rank * g.kgroups / S), k1 = (int)((long long)(rank + 1) * g.kgroups / S);
  const int per = (g.M + S - 1) / S;  // tokens that a block finishes
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    mbar_init(&acc_bar, 1);
    late = 0;
    fence_mbar_init();
    tma_prefetch_desc(&g.tm_a);
    tma_prefetch_desc(&g.tm_b);
  }
  constexpr uint32_t kCols = TN < 32 ? 32 : TN;
  if (warp == 1) {
    tmem_alloc(&tmem_slot, kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  if (S > 1) cluster_arrive_release();  // (this block has started: its sums may be written)
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  pdl_wait();
  pdl_launch_dependents();
  if (warp == 0) {
    const uint32_t base = smem_u32(smem);
    int s = 0;
    uint32_t phase = 0;
    for (int k = k0; k < k1; ++k) {
      if (!wait_warp(&empty_bar[s], phase ^ 1, p.wait_ns)) {
        give_up(&late, kStatusTimeoutProducer);
        break;
      }
      const uint32_t bar = smem_u32(&full_bar[s]), dst = base + s * C::kStageBytes;
      mbar_arrive_expect_tx_if(lane == 0, &full_bar[s], C::kStageBytes);
      if (g.a_mn) {
#pragma unroll
        for (int c = 0; c < 2; ++c) tma_load_2d<false>(dst + c * 8192, &g.tm_a, bar, tile * 128 + 64 * c, k * 64);
      } else {
        tma_load_2d<false>(dst, &g.tm_a, bar, k * 64, tile * 128);
      }
      tma_load_2d<false>(dst + 16384, &g.tm_b, bar, k * 64, 0);
      if (++s == C::kStages) {
        s = 0;
        phase ^= 1;
      }
    }
  } else if (warp == 1) {
    constexpr uint32_t kFmt = std::is_same<X, __half>::value ? 0u : 1u;
    const uint32_t idesc =
        (1u << 4) | (kFmt << 7) | (kFmt << 10) | ((uint32_t)g.a_mn << 15) | ((uint32_t)(TN >> 3) << 17) | ((128u >> 4) << 24);
    const uint32_t a_step = g.a_mn ? 128 : 2;  // (operand forms as in dense_gemm_kernel)
    const uint64_t a_desc = smem_desc(smem_u32(smem), g.a_mn ? 8192 : 16, 1024, 2);
    const uint64_t b_desc = smem_desc(smem_u32(smem) + 16384, 16, 1024, 2);
    int s = 0;
    uint32_t phase = 0;
    for (int k = k0; k < k1; ++k) {
      if (!wait_warp(&full_bar[s], phase, p.wait_ns)) {
        give_up(&late, kStatusTimeoutMain);
        break;
      }
      tc_fence_after();
      const uint64_t at = (uint64_t)(s * (C::kStageBytes / 16));
#pragma unroll
      for (int ks = 0; ks < 4; ++ks)
        mma_f16<false>(tmem, a_desc + at + (uint64_t)(a_step * ks), b_desc + at + (uint64_t)(2 * ks), idesc,
                       k > k0 || ks > 0 ? 1u : 0u);
      commit<false>(&empty_bar[s]);
      if (++s == C::kStages) {
        s = 0;
        phase ^= 1;
      }
    }
    // (also after a time-out: the sums' readers and the tensor memory's release wait for what was issued)
    commit<false>(&acc_bar);
    if (!wait_warp(&acc_bar, 0, kDrainLimit)) give_up(&late, kStatusTimeoutMain);
  }
  // the tokens that this block finishes, a warp to each in turn, a lane to four neighbouring rows;
  // the residual of the first ones comes in while the products run
  constexpr int kAtOnce = 4;
  const int n = tile * 128 + 4 * lane, mine = min(per, g.M - rank * per), w0 = warp - 2;
  using Four = std::conditional_t<WIDE, uint4, uint2>;
  Four res[kAtOnce];
  auto load_residual4 = [&](int i0) {
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const int t = w0 + kBatchEpiWarps * (i0 + i);
      if (p.residual && t < mine && n < g.N)
        res[i] = __ldcg(reinterpret_cast<const Four*>(reinterpret_cast<const O*>(p.residual) + (size_t)(rank * per + t) * g.N + n));
    }
  };
  if (warp >= 2) load_residual4(0);
  const int q = warp & 3, row = q * 32 + lane;
  if (warp >= 2 && !wait_warp(&acc_bar, 0, p.wait_ns + kDrainLimit)) give_up(&late, kStatusTimeoutEpi);
  __syncwarp();
  if (S > 1) cluster_wait_acquire();
  tc_fence_after();
  if (warp >= 2) {
    // (two warps a quarter of the rows, sixteen tokens each in turn)
#pragma unroll 1
    for (int c = 16 * (w0 >> 2); c < g.M; c += 32) {
      int owner = c / per, local = c - owner * per;  // of token c + i
      uint32_t raw[16];
      float v[16];
      tmem_ld_32x32b_x16(tmem + ((uint32_t)(q * 32) << 16) + c, raw);
      const uint32_t first = smem_u32(sums + rank * per * 128 + row);  // of the owner's first token
      uint32_t to = (S > 1 ? mapa_shared(first, owner) : first) + local * 512;
      tmem_wait_ld();
      landed(raw, v);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        if (c + i >= g.M) break;
        if (S > 1)
          asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to), "f"(v[i]) : "memory");
        else
          asm volatile("st.shared.f32 [%0], %1;" ::"r"(to), "f"(v[i]) : "memory");
        to += 512;
        if (++local == per) {
          local = 0;
          ++owner;
          to = S > 1 && owner < S ? mapa_shared(first, owner) : first;
        }
      }
      __syncwarp();
    }
    tc_fence_before();
  }
  __syncwarp();
  __syncthreads();
  if (S > 1) {
    cluster_arrive_release();
    cluster_wait_acquire();
  }
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, kCols);
  if (warp >= 2 && n < g.N) {  // (N is a multiple of 8: four rows are all in it, or none)
    float bias[4] = {};
    if (p.bias) {
      const float4 b = __ldcg(reinterpret_cast<const float4*>(p.bias + n));
      bias[0] = b.x; bias[1] = b.y; bias[2] = b.z; bias[3] = b.w;
    }
    O* out = reinterpret_cast<O*>(g.out);
    for (int i0 = 0; w0 + kBatchEpiWarps * i0 < mine; i0 += kAtOnce) {
      if (i0 > 0) load_residual4(i0);
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        const int t = w0 + kBatchEpiWarps * (i0 + i);
        if (t >= mine) break;
        const size_t at = (size_t)(rank * per + t) * g.N + n;
        float v[4] = {};
        for (int b = 0; b < S; ++b) {
          const float4 f = *reinterpret_cast<const float4*>(sums + (b * per + t) * 128 + 4 * lane);
          v[0] += f.x; v[1] += f.y; v[2] += f.z; v[3] += f.w;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] += bias[j];
        if (p.gateup) *reinterpret_cast<float4*>(p.gateup + at) = make_float4(v[0], v[1], v[2], v[3]);
        if (p.act == kActSilu) {
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] = act_f<kActSilu>(v[j]);
        } else if (p.act == kActGelu) {
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] = act_f<kActGelu>(v[j]);
        }
        if constexpr (WIDE) {
          if (p.residual) {
            v[0] += __uint_as_float(res[i].x); v[1] += __uint_as_float(res[i].y);
            v[2] += __uint_as_float(res[i].z); v[3] += __uint_as_float(res[i].w);
          }
          *reinterpret_cast<float4*>(out + at) = make_float4(v[0], v[1], v[2], v[3]);
        } else {
          if (p.residual) {
            const float2 a = unpack2<X>(res[i].x), b = unpack2<X>(res[i].y);
            v[0] += a.x; v[1] += a.y; v[2] += b.x; v[3] += b.y;
          }
          *reinterpret_cast<uint2*>(out + at) = make_uint2(pack2<X>(v[0], v[1]), pack2<X>(v[2], v[3]));
        }
      }
    }
  }
  // after a time-out some copies may still be on their way: stay until they have surely landed
  __syncthreads();
  if (threadIdx.x == 0 && late) {
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < kLandingNs) __nanosleep(1000);
  }
}

// The split tiles: the slices' sums in slice order, then the epilogue (about 4 us, from L2).
// 16 columns (of gate and of up) per thread.
template <typename X, int MODE>
__global__ void __launch_bounds__(256) dense_join_kernel(const __grid_constant__ DenseGemmParams p, int tile_rows, int bn) {
  pdl_wait();
  pdl_launch_dependents();
  const int cols = MODE == kDenseGateUp ? bn / 2 : bn, per_row = cols / 16;
  const long long i = blockIdx.x * 256LL + threadIdx.x;
  const int c = (int)(i % per_row) * 16;
  const int r = (int)(i / per_row % tile_rows), tile = (int)(i / per_row / tile_rows);
  const DenseProblem& g = p.g[0];
  if (p.full + tile >= g.tiles_m * g.tiles_n) return;
  const Unit t = map_unit(p, p.full + tile * p.splits);
  const int m = t.m * tile_rows + r, n = t.n * cols + c;
  if (m >= g.M || n >= g.N) return;
  float v[16], w[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) v[j] = w[j] = 0.f;
  for (int s = 0; s < p.splits; ++s) {
    const float* part = p.partial + ((size_t)(tile * p.splits + s) * tile_rows + r) * bn + c;
    float f[8];
#pragma unroll
    for (int j = 0; j < 16; j += 8) {
      load8(f, part + j);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[j + k] += f[k];
      if constexpr (MODE == kDenseGateUp) {
        load8(f, part + cols + j);
#pragma unroll
        for (int k = 0; k < 8; ++k) w[j + k] += f[k];
      }
    }
  }
  epilogue<X, MODE, 16>(p, g, m, n, g.N - n, v, w);
}

// ------------------------------------------------------------------ host side
struct Shape {
  int bn;
  bool pair;
  int tiles_m, tiles_n, full, splits;
  float time;  // estimated cycles
};

// Tile shape and split by estimated time, in cycles.  A unit's K group (64 values) takes
// what its MMAs, its operand bytes and the issuing of both need; a round of whole tiles
// takes all SMs, and the tiles of a last, partial round may be cut along K so that its
// slices fill the SMs, at the price of f32 partial sums written and read and one more
// launch.  The constants are fitted to measured products: a 256-column pair tile takes 540
// cycles a K group, one of 192 columns and less 440 (issuing), one-SM tiles of 128 and 64
// columns 530 and 335; HBM gives each SM 23 bytes a cycle.  Widths between the powers of two
// (2048 tokens x 4096 x 14336: 367 us with them, 375 without) are for K-major B only: an
// MN-major one comes in whole chunks of 64 columns.
Shape estimate_shape(int M, int N, int K, int mode, bool b_mn, int sms) {
  const int kg = ceil_div(K, 64), cols = mode == kDenseGateUp ? 2 * N : N;
  const float hbm = ((float)M + (float)cols) * (float)K * 2.f / (23.f * (float)sms);
  Shape best{};
  float best_time = 0.f;
  for (int config = 0; config < 7; ++config) {
    Shape s{};
    s.pair = config < 5;
    s.bn = s.pair ? 256 - 32 * config : config == 5 ? 128 : 64;
    if (s.pair && (M <= 128 || (b_mn && s.bn % 128))) continue;
    const int tile_m = s.pair ? 256 : 128, workers = s.pair ? sms / 2 : sms;
    s.tiles_m = ceil_div(M, tile_m);
    s.tiles_n = mode == kDenseGateUp ? ceil_div(N, s.bn / 2) : ceil_div(cols, s.bn);
    const int rows = M < 128 ? M : 128;
    const float group = s.pair ? fmaxf(2.12f * s.bn, 440.f) : s.bn == 128 ? 530.f : 335.f;
    const int tiles = s.tiles_m * s.tiles_n, rem = tiles % workers;
    for (int splits = 1; splits <= kDenseMaxSplits && (splits == 1 || kg / splits >= 4); ++splits) {
      s.splits = splits;
      s.full = splits == 1 ? tiles : tiles - rem;
      if (splits > 1 && rem == 0) break;
      float time = (float)ceil_div(s.full, workers) * ((float)kg * group + 1000.f);
      if (splits > 1) {
        const float slice = (float)ceil_div(kg, splits) * group + 1500.f;
        const float moved = (float)rem * splits * (float)(s.pair ? 256 : rows) * s.bn * 8.f;
        time += (float)ceil_div(rem * splits, workers) * slice + moved / 2500.f + 5000.f;
      }
      // (of as many columns the narrower tile: the last one's epilogue has no MMAs to hide behind)
      if (mode == kDenseLinear) time += 20.f * s.bn;
      if (time < hbm) time = hbm + 0.1f * time;  // (ties on the HBM bound go to the smaller work)
      if (best_time == 0.f || time < best_time) {
        best_time = time;
        best = s;
        best.time = time;
      }
    }
  }
  return best;
}
// The estimate is a function of the sizes alone; the last ones are kept per thread, since a
// small product's launch would wait for its 0.9 us otherwise.
Shape pick_shape(int M, int N, int K, int mode, bool b_mn) {
  if (mode == kDenseLinear32) mode = kDenseLinear;
  struct Entry {
    int M, N, K, key;
    Shape s;
  };
  static thread_local Entry kept[16] = {};
  const int sms = device_sms(), key = sms * 16 + mode * 2 + b_mn;
  Entry& e = kept[((unsigned)M * 31u + (unsigned)N * 7u + (unsigned)K * 3u + (unsigned)key) * 2654435761u >> 28];
  if (e.M != M || e.N != N || e.K != K || e.key != key) e = {M, N, K, key, estimate_shape(M, N, K, mode, b_mn, sms)};
  return e.s;
}

typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
  static EncodeTiled fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiled>(f);
  });
  return fn;
}

// A 16-bit matrix as boxes of 64 columns (128 bytes, swizzled) by `box_rows` rows.
bool operand_map(CUtensorMap* map, const DenseOperand& o, int box_rows, int dtype) {
  EncodeTiled enc = encode_tiled();
  if (!enc) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)o.cols, (cuuint64_t)o.rows};
  const cuuint64_t strides[1] = {(cuuint64_t)o.cols * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)box_rows}, es[2] = {1, 1};
  return enc(map, dtype == kDtypeF16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
             const_cast<void*>(o.ptr), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Blocks that are resident together: pairs may not fill every SM.
template <typename Kern>
cudaError_t resident_blocks(Kern kern, int smem, bool pair, std::atomic<int> (&cached)[kMaxDevices], int* blocks) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 0 && dev < kMaxDevices && (*blocks = cached[dev].load(std::memory_order_relaxed)) > 0) return cudaSuccess;
  int n = 0;
  if (pair) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(kDenseThreads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {2, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg);
    n *= 2;
  } else {
    e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  }
  if (e != cudaSuccess) return e;
  if (n < 2) n = 2;
  if (dev >= 0 && dev < kMaxDevices) cached[dev].store(n, std::memory_order_relaxed);
  *blocks = n;
  return cudaSuccess;
}

template <typename X, int MODE, int BN, bool PAIR>
cudaError_t launch_kernel(const DenseGemmParams& p, long long units, cudaStream_t stream) {
  using C = DenseCfg<BN, PAIR>;
  auto kern = dense_gemm_kernel<X, MODE, BN, PAIR>;
  static SmemOptIn opt_in;
  cudaError_t e = opt_in.ensure(kern, C::kSmemBytes);
  if (e != cudaSuccess) return e;
  static std::atomic<int> cached[kMaxDevices] = {};
  int blocks = 0;
  e = resident_blocks(kern, C::kSmemBytes, PAIR, cached, &blocks);
  if (e != cudaSuccess) return e;
  if (units * C::kCtas < blocks) blocks = (int)units * C::kCtas;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(kDenseThreads);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {2, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = PAIR ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

template <typename X, int MODE>
cudaError_t launch_mode(const DenseGemmParams& p, const Shape& s, cudaStream_t stream) {
  const long long units = s.full + (long long)(s.tiles_m * s.tiles_n - s.full) * s.splits;
  const cudaError_t e = s.pair         ? launch_kernel<X, MODE, 256, true>(p, units, stream)
                        : s.bn == 128 ? launch_kernel<X, MODE, 128, false>(p, units, stream)
                                      : launch_kernel<X, MODE, 64, false>(p, units, stream);
  if (e != cudaSuccess || s.splits == 1) return e;
  const int tile_rows = s.pair ? 256 : 128;
  const long long threads =
      (long long)(s.tiles_m * s.tiles_n - s.full) * tile_rows * ((MODE == kDenseGateUp ? s.bn / 2 : s.bn) / 16);
  return launch_pdl(dense_join_kernel<X, MODE>, dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, stream, p, tile_rows,
                    s.bn);
}

template <typename X>
cudaError_t launch_type(const DenseGemmParams& p, const Shape& s, int mode, cudaStream_t stream) {
  if (mode == kDenseGateUp) return launch_mode<X, kDenseGateUp>(p, s, stream);
  if (mode == kDenseGateUpGrad) return launch_mode<X, kDenseGateUpGrad>(p, s, stream);
  if (mode == kDenseLinear) return launch_mode<X, kDenseLinear>(p, s, stream);
  if (mode == kDenseLinear32) return launch_mode<X, kDenseLinear32>(p, s, stream);
  return launch_mode<X, kDenseStore>(p, s, stream);
}

}  // namespace

size_t dense_partial_bytes(int M, int N, int K, int mode, bool b_mn) {
  const Shape s = pick_shape(M, N, K, mode, b_mn);
  if (s.splits == 1) return 0;
  return (size_t)(s.tiles_m * s.tiles_n - s.full) * s.splits * (s.pair ? 256 : 128) * s.bn * sizeof(float);
}

// A product's operands and tiles into its place.
bool set_problem(DenseProblem& g, const DenseOperand& a, const DenseOperand& b, int b_box, int tiles_m, int tiles_n,
                 int dtype) {
  g.a_mn = a.mn_major;
  g.b_mn = b.mn_major;
  g.tiles_m = tiles_m;
  g.tiles_n = tiles_n;
  g.kgroups = ceil_div(g.K, 64);
  return operand_map(&g.tm_a, a, a.mn_major ? 64 : 128, dtype) && operand_map(&g.tm_b, b, b.mn_major ? 64 : b_box, dtype);
}

int launch_dense_gemm(DenseGemmParams p, const DenseOperand& a, const DenseOperand& b, int mode, int dtype,
                      cudaStream_t stream) {
  DenseProblem& g = p.g[0];
  const Shape s = pick_shape(g.M, g.N, g.K, mode, b.mn_major);
  p.bn = s.bn;
  p.full = s.full;
  p.splits = s.splits;
  p.wait_ns = gemm_wait_limit_ns();
  if (!set_problem(g, a, b, s.pair || mode == kDenseGateUp ? s.bn / 2 : s.bn, s.tiles_m, s.tiles_n, dtype))
    return MOE_ERR_CUDA;
  const cudaError_t e = dtype == kDtypeF16 ? launch_type<__half>(p, s, mode, stream)
                                           : launch_type<__nv_bfloat16>(p, s, mode, stream);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

int launch_dense_products(DenseGemmParams p, int n, const DenseOperand* a, const DenseOperand* b, int dtype, bool few_rows,
                          cudaStream_t stream) {
  // the class of the larger K first
  int order[kDenseGroup] = {0, 1, 2};
  for (int i = 1; i < n; ++i)
    for (int j = i; j > 0 && p.g[order[j]].K > p.g[order[j - 1]].K; --j) std::swap(order[j], order[j - 1]);
  DenseGemmParams q = p;
  q.group = n;
  q.long_n = 0;
  q.bn = 256;
  q.splits = 1;
  q.wait_ns = gemm_wait_limit_ns();
  const int workers = device_sms() / 2;
  long long tiles[2] = {0, 0};  // of the long and of the short class
  float apart = 0.f;
  for (int i = 0; i < n; ++i) {
    const DenseProblem& g = p.g[order[i]];
    const bool is_long = g.K == p.g[order[0]].K;
    q.long_n += is_long;
    tiles[is_long ? 0 : 1] += (long long)ceil_div(g.M, 256) * ceil_div(g.N, 256);
    apart += pick_shape(g.M, g.N, g.K, kDenseStore, b[order[i]].mn_major).time;
  }
  // estimated as in pick_shape; every launch has a start and an end of about 5000 cycles
  const float len[2] = {ceil_div(p.g[order[0]].K, 64) * 540.f, ceil_div(p.g[order[n - 1]].K, 64) * 540.f};
  q.lead = q.long_n < n ? (int)(len[0] / len[1] + 0.5f) : 0;
  const float work = (float)tiles[0] * len[0] + (q.long_n < n ? (float)tiles[1] * len[1] : 0.f);
  float together = work / (float)workers + 0.5f * len[q.long_n < n ? 1 : 0] + 1000.f;
  // a few long tiles that cannot be shared out take as long as one of them: both gradients of 200 x 1024
  // -> 8192 take 27.1 us apart and 43.8 together, of 256 x 1024 -> 32768 60 and 158 (but 256 x 4096 ->
  // 14336, whose weights' tiles would have hidden them, 79.9 and 75.1)
  if (few_rows) together = fmaxf(together, (float)ceil_div((int)tiles[0], workers) * len[0] + 1000.f);
  if (n < 2 || together > apart + 5000.f * (float)(n - 1)) {
    for (int i = 0; i < n; ++i) {
      DenseGemmParams one = p;
      one.g[0] = p.g[i];
      const int st = launch_dense_gemm(one, a[i], b[i], kDenseStore, dtype, stream);
      if (st != MOE_OK) return st;
    }
    return MOE_OK;
  }
  for (int i = 0; i < n; ++i) {
    q.g[i] = p.g[order[i]];
    if (!set_problem(q.g[i], a[order[i]], b[order[i]], 128, ceil_div(q.g[i].M, 256), ceil_div(q.g[i].N, 256), dtype))
      return MOE_ERR_CUDA;
  }
  const cudaError_t e = dtype == kDtypeF16
                            ? launch_kernel<__half, kDenseProducts, 256, true>(q, tiles[0] + tiles[1], stream)
                            : launch_kernel<__nv_bfloat16, kDenseProducts, 256, true>(q, tiles[0] + tiles[1], stream);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

namespace {
template <typename X, int TN, bool WIDE>
cudaError_t launch_batch_t(const DenseGemmParams& p, cudaStream_t stream) {
  using C = BatchCfg<TN>;
  auto kern = linear_batch_kernel<X, TN, WIDE>;
  static SmemOptIn opt_in;
  const cudaError_t e = opt_in.ensure(kern, C::kSmemBytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ceil_div(p.g[0].N, 128) * p.splits);
  cfg.blockDim = dim3(kBatchThreads);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {(unsigned)p.splits, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = p.splits > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}
template <typename X, int TN>
cudaError_t launch_batch_out(const DenseGemmParams& p, bool wide, cudaStream_t stream) {
  return wide ? launch_batch_t<X, TN, true>(p, stream) : launch_batch_t<X, TN, false>(p, stream);
}
template <typename X>
cudaError_t launch_batch_x(const DenseGemmParams& p, int tn, bool wide, cudaStream_t stream) {
  return tn == 32 ? launch_batch_out<X, 32>(p, wide, stream)
         : tn == 64 ? launch_batch_out<X, 64>(p, wide, stream)
                    : launch_batch_out<X, 128>(p, wide, stream);
}
}  // namespace

int launch_linear_batch(DenseGemmParams p, const DenseOperand& x, const DenseOperand& w, int dtype, bool wide, cudaStream_t stream) {
  DenseProblem& g = p.g[0];
  const int tn = g.M <= 32 ? 32 : g.M <= 64 ? 64 : 128, tiles = ceil_div(g.N, 128);
  g.kgroups = ceil_div(g.K, 64);
  p.wait_ns = gemm_wait_limit_ns();
  // K is split while the blocks find room and keep two groups each
  p.splits = 1;
  while (p.splits < kBatchMaxSplit && tiles * 2 * p.splits <= (tn == 128 ? 1 : 2) * device_sms() && g.kgroups >= 4 * p.splits)
    p.splits *= 2;
  g.a_mn = w.mn_major;
  if (!operand_map(&g.tm_a, w, w.mn_major ? 64 : 128, dtype) || !operand_map(&g.tm_b, x, tn, dtype)) return MOE_ERR_CUDA;
  const cudaError_t e = dtype == kDtypeF16 ? launch_batch_x<__half>(p, tn, wide, stream)
                                           : launch_batch_x<__nv_bfloat16>(p, tn, wide, stream);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

uint32_t* dense_status_word() {
  void* p = nullptr;
  return cudaGetSymbolAddress(&p, g_dense_status) == cudaSuccess ? static_cast<uint32_t*>(p) : nullptr;
}

}  // namespace moe
