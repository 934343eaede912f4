// Products of a few tokens with many weight rows (decode): MXFP4 weights, and the
// 16-bit weights of the dense feed-forward block.
//   plain  y[t, n] = sum_k x[t, k] W[n, k] (+ bias[n])
//   gated  h[t, i] = act(g) u,  g and u the products with gate row i and up row i
//
// At these sizes every weight byte is read once and used for a few tokens, so the kernels
// are bound by HBM, and what matters is the bytes in flight and the instructions spent
// per weight.  The products run on mma.sync (m16n8k16, f32 sums): 16 weight rows are one
// operand, up to 8 tokens (a column group) the other.  The sum over K is free to take its
// terms in any order, so each lane's 16-byte weight read is its own operand fragments, with
// x permuted to match: no shuffles.  Sums are added in a fixed order everywhere.
//
// MXFP4: two codes become an f16 pair by one conversion instruction (exact); a group's
// 32 products are summed by two MMAs and then scaled in f32 by the group's scale, kept
// relative to the largest of its row (taken out of the sum once, at the end).
// x as f16: a power of two per token brings its largest value to [2^14, 2^15), so bf16
// values are exact down to 2^-28 of the largest (absolute error 2^-39 of it below), and is
// taken out again in f32, together with the row's scale.
#include "moe_dense.cuh"
#include "sm100_ptx.cuh"

namespace moe {

namespace {

constexpr int kThinThreads = 256;
__device__ uint32_t g_thin_status;  // bits as in the layer's status word
constexpr int kThinWarps = kThinThreads / 32;

template <typename X>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__half>(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                 uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
               "%2, %3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, "
               "%1, %2, %3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// d = a b of f16 operands (no addend).
__device__ __forceinline__ void mma16816_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, "
               "%10, %10};"
               : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// The eight E2M1 codes of a word as four f16 pairs (low nibble first).
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// Byte b of a prepared scale word as 2^(byte - 127), 0 for byte 0 (bytes are at most 127).
__device__ __forceinline__ float group_scale(uint32_t word, int b) {
  return __uint_as_float(__byte_perm(word, 0, 0x0444 | (b << 12)) >> 1);
}

__device__ __forceinline__ uint4 load_weights(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// Adds the eight warps' sums of a tile (fragment layout: register pair c < 2 is row g,
// c >= 2 row g + 8, token 2 t + (c & 1)) in warp order and writes the block's outputs.
constexpr int kFinishStride = kThinRows + 4;
template <int NT>
__device__ __host__ constexpr int finish_bytes() {
  return kThinWarps * NT * 8 * kFinishStride * 4;
}
template <typename X, int NT, bool GATED, int ACT>
__device__ __forceinline__ void finish(const ThinParams& p, const float (&total)[NT][4], float* red, int tile) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int c = 0; c < 4; ++c)
      red[(warp * NT * 8 + n * 8 + 2 * t + (c & 1)) * kFinishStride + g + 8 * (c >> 1)] = total[n][c];
  __syncthreads();
  constexpr int kOut = GATED ? kThinRows / 2 : kThinRows;
  X* out = reinterpret_cast<X*>(p.out);
  for (int i = threadIdx.x; i < p.T * kOut; i += kThinThreads) {
    const int tok = i / kOut, o = i % kOut, f = tile * kOut + o;
    if (f >= p.n_out) continue;
    const size_t row = (size_t)tok;
    auto sum = [&](int r) {
      float v = red[tok * kFinishStride + r];
#pragma unroll
      for (int w = 1; w < kThinWarps; ++w) v += red[(w * NT * 8 + tok) * kFinishStride + r];
      return v;
    };
    if constexpr (GATED) {
      const float gv = sum(o), uv = sum(o + 8);
      if (p.gateup) {
        p.gateup[row * 2 * p.n_out + f] = gv;
        p.gateup[row * 2 * p.n_out + p.n_out + f] = uv;
      }
      out[row * p.n_out + f] = static_cast<X>(act_f<ACT>(gv) * uv);
    } else {
      out[row * p.n_out + f] = static_cast<X>(sum(o));
    }
  }
}

// x as f16.  bf16: a power of two, 2^126 at most, that brings the largest finite exponent (of
// the values scaled together) to 14 takes values to f16, and its inverse's exponent is
// returned; 2^126 leaves subnormals, whose smallest step is 2^-133, exact.  f16 as it is.
template <typename X>
__device__ __forceinline__ uint32_t max_exponent(const uint4& v) {
  if constexpr (std::is_same<X, __half>::value) return 0;
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t e = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t lo = (w[j] >> 7) & 0xFFu, hi = (w[j] >> 23) & 0xFFu;
    e = max(e, max(lo == 255u ? 0u : lo, hi == 255u ? 0u : hi));
  }
  return e;
}
template <typename X>
__device__ __forceinline__ int scale_to_f16(uint4& v, uint32_t emax) {
  if constexpr (std::is_same<X, __half>::value) return 0;
  const int pw = min(126, 14 + 127 - (int)emax);
  const float up = pow2_int(pw);
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = unpack2<__nv_bfloat16>(w[j]);
    w[j] = pack2<__half>(f.x * up, f.y * up);
  }
  v = make_uint4(w[0], w[1], w[2], w[3]);
  return -pw;
}
__device__ __forceinline__ void st_cluster_f32x4(uint32_t addr, const float (&v)[4]) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3])
               : "memory");
}

// ------------------------------------------------------------------ MXFP4 weights
// A block's eight warps take a tile each and walk K together.  A pipeline stage is one or
// two K units of the block's tiles (contiguous in the prepared weights: one bulk copy)
// and, where x is not resident, the same units of x; the warps refill the stages in turn.
// So the bytes in flight do not depend on registers or on how far the arithmetic has got,
// and the 16-byte shared-memory reads are the fragments.
// x, as f16, comes in one of two ways:
//   resident (few tokens, short K): the block converts it itself, once; rows padded by 64
//     bytes, so that two tokens' 64-byte pieces fall into different banks;
//   packed: a launch before wrote it to the workspace in fragment order.
// Blocks are persistent over row groups; where there are too few groups to fill the GPU,
// a cluster of blocks splits K and each block finishes its share of the tokens, from the
// fragments that the others write into its shared memory, added in rank order.  (K split
// between the warps of a block, with a copy per slice and stage, measured slower: one token
// x 131072 x 4096 67.8 us against 53.2.)
// What bounds it: over many rows HBM and the ALU pipe nearly alike (that product: 5.36 TB/s
// of a copy's 6.7, the ALU pipe 0.59 busy with the codes' conversions, the last of 2.25
// rounds a quarter full); at 16 tokens the instructions (gated 14336 x 4096: 21.6 us, of
// them about 3 for packing x); below 10 MB the launch (2880 x 2880: 5.1 us).
constexpr int kUnitBytes = kMatvecUnitBytes;
constexpr int kGroupBytes = kMatvecGroup * kUnitBytes;  // one K unit of eight tiles
constexpr uint64_t kMatvecWaitNs = 1000000000ull;       // a wait may take 1 s
constexpr int kMatvecMaxSplit = 4;                      // blocks of a cluster
constexpr int kResidentPieces = 64;                     // resident x: (token, unit) pairs, at most
static_assert(kMatvecGroup == kThinWarps, "one tile per warp and group");

template <int NT, bool PACKED>
struct MatvecCfg {
  static constexpr int kPerSm = NT == 4 ? 2 : 3;  // resident blocks, by registers
  // K units per stage: two where registers and memory allow (the eight warps meet at every
  // stage; one token x 131072 x 4096: 53.6 us, 60.8 with one unit and twice the stages)
  static constexpr int kUnits = NT == 1 ? 2 : 1;
  static constexpr int kStages = NT == 1 ? 3 : NT == 2 ? 5 : 6;
  static constexpr int kUnitTotal = kGroupBytes + (PACKED ? NT * 2048 : 0);
  static constexpr int kStageBytes = kUnits * kUnitTotal;
  static constexpr int kRingBytes = kStages * kStageBytes;
  static_assert((NT > kMatvecMaxSplit ? NT : kMatvecMaxSplit) * kThinWarps * 512 <= kRingBytes,
                "a cluster's fragments take the ring's memory");
};
__host__ __device__ inline int resident_row_halves(int ku) { return ku * 128 + 32; }
inline bool matvec_resident(int tokens, int ku) { return tokens <= 8 && tokens * ku <= kResidentPieces; }

// One K unit of a row tile against NT column groups: `sum` += products, scaled by the
// groups' scales.  `read_x(blk, n8)` gives this lane's x fragment.
template <int NT, typename ReadX>
__device__ __forceinline__ void unit_product(const uint8_t* unit, float (&sum)[NT][4], ReadX read_x) {
  const int lane = threadIdx.x & 31, g = lane >> 2;
  const uint4 w0 = *reinterpret_cast<const uint4*>(unit + lane * 16);
  const uint4 w1 = *reinterpret_cast<const uint4*>(unit + 512 + lane * 16);
  const uint2 sc = *reinterpret_cast<const uint2*>(unit + 1024 + g * 8);
#pragma unroll
  for (int blk = 0; blk < 4; ++blk) {
    uint32_t h0[4], h1[4];
    e2m1x8_to_f16(blk == 0 ? w0.x : blk == 1 ? w0.y : blk == 2 ? w0.z : w0.w, h0);
    e2m1x8_to_f16(blk == 0 ? w1.x : blk == 1 ? w1.y : blk == 2 ? w1.z : w1.w, h1);
    const float s0 = group_scale(sc.x, blk), s1 = group_scale(sc.y, blk);
#pragma unroll
    for (int n8 = 0; n8 < NT; ++n8) {
      const uint4 x = read_x(blk, n8);
      float d[4];
      mma16816_zero(d, h0[0], h1[0], h0[1], h1[1], x.x, x.y);
      mma16816<__half>(d, h0[2], h1[2], h0[3], h1[3], x.z, x.w);
      sum[n8][0] = fmaf(d[0], s0, sum[n8][0]);
      sum[n8][1] = fmaf(d[1], s0, sum[n8][1]);
      sum[n8][2] = fmaf(d[2], s1, sum[n8][2]);
      sum[n8][3] = fmaf(d[3], s1, sum[n8][3]);
    }
  }
}

// A sum times 2^e, plus the bias.  e, of the token's scale and of the row's largest group
// scale together, is in [-253, 240], so the power goes in two halves: one scale after the
// other would leave f32's range on the way to results inside it (values near 2^120 against
// scales near 2^-120, and the reverse).  Each half is a normal f32: -126 in place of -127
// for the least e is as good, the result being zero with either.
__device__ __forceinline__ float scaled(float sum, int e, float bias) {
  const int half = e >> 1;
  return fmaf(sum * pow2_int(max(half, -126)), pow2_int(max(e - half, -126)), bias);
}

// ---- packed x: [token group][K units][4 groups][NT][32 lanes][16 bytes] f16, then the
// tokens' exponents.  One block per token of the padded groups.
template <int NT>
inline size_t packed_bytes(int T, int ku) { return (size_t)ceil_div(T, NT * 8) * ku * NT * 2048; }

template <typename X, int NT>
__global__ void __launch_bounds__(256) matvec_pack_kernel(const __grid_constant__ ThinParams p) {
  __shared__ uint32_t s_max[8];
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  const int tok = blockIdx.x, vecs = p.ku * 16;
  const uint4* row = reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p.x) + (size_t)tok * p.K);
  auto load = [&](int i) { return tok < p.T && 8 * i < p.K ? __ldcg(row + i) : make_uint4(0, 0, 0, 0); };
  uint4 first[4];  // rows of up to 8192 values are read once
  uint32_t emax = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int i = threadIdx.x + 256 * j;
    first[j] = i < vecs ? load(i) : make_uint4(0, 0, 0, 0);
    emax = max(emax, max_exponent<X>(first[j]));
  }
  for (int i = threadIdx.x + 1024; i < vecs; i += 256) emax = max(emax, max_exponent<X>(load(i)));
  emax = __reduce_max_sync(0xffffffffu, emax);
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = emax;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) emax = max(emax, s_max[w]);
  const int group = tok / (NT * 8), r = tok - group * NT * 8;
  int down = 0;
  auto put = [&](int i, uint4 v) {
    down = scale_to_f16<X>(v, emax);
    // vector i: unit i / 16, its group (i % 16) / 4, fragment lane 4 (token % 8) + i % 4
    uint8_t* unit = p.packed + ((size_t)group * p.ku + (i >> 4)) * (NT * 2048);
    *reinterpret_cast<uint4*>(unit + (((i >> 2) & 3) * NT + (r >> 3)) * 512 + (4 * (r & 7) + (i & 3)) * 16) = v;
  };
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int i = threadIdx.x + 256 * j;
    if (i < vecs) put(i, first[j]);
  }
  for (int i = threadIdx.x + 1024; i < vecs; i += 256) put(i, load(i));
  if (threadIdx.x == 0) p.x_exp[tok] = down;
}

template <typename X, int NT, bool PACKED, bool GATED, int ACT>
__global__ void __launch_bounds__(kThinThreads, MatvecCfg<NT, PACKED>::kPerSm)
    matvec_kernel(const __grid_constant__ ThinParams p) {
  using C = MatvecCfg<NT, PACKED>;
  static_assert(PACKED || NT == 1, "resident x: one column group");
  extern __shared__ __align__(128) uint8_t thin_smem[];
  __shared__ uint64_t full_bar[C::kStages], empty_bar[C::kStages];
  __shared__ uint32_t s_max[8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int log_s = p.log_kw, S = 1 << log_s, rank = blockIdx.x & (S - 1), groups = p.tiles / kMatvecGroup;
  const int t0 = blockIdx.y * NT * 8, nt = min(p.T - t0, NT * 8);
  const int k_begin = rank * p.ku >> log_s, k_units = ((rank + 1) * p.ku >> log_s) - k_begin;
  const int steps = (k_units + C::kUnits - 1) / C::kUnits;  // stages of a group
  const int grp_step = gridDim.x >> log_s, grp0 = blockIdx.x >> log_s;
  uint8_t* const xs = thin_smem + C::kRingBytes;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      ptx::mbar_init(&full_bar[i], 1);
      ptx::mbar_init(&empty_bar[i], kThinWarps);
    }
    ptx::fence_mbar_init();
  }
  if (!PACKED && threadIdx.x < 8) s_max[threadIdx.x] = 0;
  __syncthreads();
  // step `at` of group grp into stage s: its weights, and its units of x
  auto issue_w = [&](int s, int grp, int at) {
    const int u = at * C::kUnits, n = min(C::kUnits, k_units - u);
    ptx::mbar_arrive_expect_tx(&full_bar[s], n * C::kUnitTotal);
    ptx::bulk_load(thin_smem + s * C::kStageBytes,
                   reinterpret_cast<const uint8_t*>(p.w) + ((size_t)grp * p.ku + k_begin + u) * kGroupBytes, n * kGroupBytes,
                   &full_bar[s]);
  };
  auto issue_x = [&](int s, int at) {
    const int u = at * C::kUnits, n = min(C::kUnits, k_units - u);
    ptx::bulk_load(thin_smem + s * C::kStageBytes + C::kUnits * kGroupBytes,
                   p.packed + ((size_t)blockIdx.y * p.ku + k_begin + u) * (NT * 2048), n * NT * 2048, &full_bar[s]);
  };
  // `by` steps on from step `at` of group grp (steps wrap into the block's next groups)
  auto advance = [&](int& grp, int& at, int by) {
    for (at += by; at >= steps; at -= steps) grp += grp_step;
  };
  auto first_stages = [&](auto f) {
    int grp = grp0, at = 0;
    for (int s = 0; s < C::kStages && grp < groups; ++s, advance(grp, at, 1)) f(s, grp, at);
  };
  // Weights of packed x's kernel may be read before the dependency wait: the launch before
  // it is the packing one, which began its work only when all earlier work had completed.
  if (PACKED && threadIdx.x == 0) first_stages([&](int s, int grp, int at) { issue_w(s, grp, at); });
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  if (threadIdx.x == 0)
    first_stages([&](int s, int grp, int at) {
      if (PACKED) issue_x(s, at);
      else issue_w(s, grp, at);
    });
  int down[2] = {0, 0};  // exponents of x's tokens 2 t, 2 t + 1 (resident x)
  const int row_halves = resident_row_halves(p.ku);
  if constexpr (!PACKED) {
    // 16 lanes take one (token, unit), 8 values each; zero past K
    const int pieces = nt * p.ku, l = lane & 15;
    uint4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int q = (threadIdx.x >> 4) + 16 * i, tok = q / p.ku, u = q - tok * p.ku, k = u * 128 + l * 8;
      v[i] = make_uint4(0, 0, 0, 0);
      if (q < pieces && k < p.K) {
        v[i] = __ldcg(reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p.x) + (size_t)tok * p.K + k));
        if constexpr (!std::is_same<X, __half>::value) atomicMax(&s_max[tok], max_exponent<X>(v[i]));
      }
    }
    if constexpr (!std::is_same<X, __half>::value) __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int q = (threadIdx.x >> 4) + 16 * i, tok = q / p.ku, u = q - tok * p.ku;
      if (q >= pieces) continue;
      scale_to_f16<X>(v[i], s_max[tok]);
      *reinterpret_cast<uint4*>(xs + ((size_t)tok * row_halves + u * 128 + l * 8) * 2) = v[i];
    }
    __syncthreads();
    if constexpr (!std::is_same<X, __half>::value) {
      uint4 none = make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int c = 0; c < 2; ++c) down[c] = scale_to_f16<X>(none, s_max[min(2 * t + c, 7)]);
    }
  }
  // resident x: lanes of absent tokens read the last token's row; their columns are never written
  const uint8_t* const x_row = xs + (min(g, nt - 1) * row_halves + 8 * t) * 2;
  X* const out = reinterpret_cast<X*>(p.out);

  int s = 0, prev = C::kStages - 1, turn = 0;  // this step's stage, the one before, the warp that refills
  uint32_t phase = 0;
  bool ok = true;
  for (int grp = grp0; grp < groups; grp += grp_step) {
    float total[NT][4] = {};
    for (int at = 0; at < steps; ++at) {
      if (ok && !ptx::mbar_wait_bounded(&full_bar[s], phase, kMatvecWaitNs)) ok = false;
      const uint8_t* st = thin_smem + s * C::kStageBytes;
#pragma unroll
      for (int j = 0; j < C::kUnits; ++j) {
        const int u = at * C::kUnits + j;
        if (u >= k_units) break;
        unit_product<NT>(st + j * kGroupBytes + warp * kUnitBytes, total, [&](int blk, int n8) {
          if constexpr (PACKED)
            return *reinterpret_cast<const uint4*>(st + C::kUnits * kGroupBytes + ((j * 4 + blk) * NT + n8) * 512 + lane * 16);
          else
            return *reinterpret_cast<const uint4*>(x_row + ((k_begin + u) * 128 + 32 * blk) * 2);
        });
      }
      __syncwarp();
      if (lane == 0) {
        ptx::mbar_arrive(&empty_bar[s]);
        // refill the stage before this one, which the other warps have most likely left too
        if (warp == turn && (grp != grp0 || at > 0)) {
          int next = grp, to = at - 1;
          advance(next, to, C::kStages);
          if (next < groups) {
            // (that stage's phase is this one's, unless the ring wrapped between them)
            if (!ptx::mbar_wait_bounded(&empty_bar[prev], prev > s ? phase ^ 1 : phase, kMatvecWaitNs)) ok = false;
            if (ok) {
              issue_w(prev, next, to);
              if (PACKED) issue_x(prev, to);
            }
          }
        }
      }
      turn = (turn + 1) & (kThinWarps - 1);
      prev = s;
      if (++s == C::kStages) {
        s = 0;
        phase ^= 1;
      }
    }
    const int tile0 = grp * kMatvecGroup;
    if (S > 1) {
      // (one group per cluster) Each block finishes the column groups n8 = rank (mod S): the
      // others send theirs to its ring, [n8 / S][sender][warp][lane], whose copies have all
      // been consumed once its warps have arrived.  (The first lane may still be in the last
      // refill's branch, and the barrier's instruction is the whole warp's.)
      __syncwarp();
      ptx::cluster_arrive_release();
      ptx::cluster_wait_acquire();
      const uint32_t slot = (warp * 32 + lane) * 16;
#pragma unroll
      for (int n8 = 0; n8 < NT; ++n8)
        if ((n8 & (S - 1)) != rank)
          st_cluster_f32x4(ptx::mapa_shared(ptx::smem_u32(thin_smem) + ((n8 >> log_s) * S + rank) * kThinWarps * 512 + slot,
                                            n8 & (S - 1)), total[n8]);
      ptx::cluster_arrive_release();
      ptx::cluster_wait_acquire();
#pragma unroll
      for (int n8 = 0; n8 < NT; ++n8)
        if ((n8 & (S - 1)) == rank)
          for (int r = 0; r < S; ++r) {
            if (r == rank) continue;
            const float4 v = *reinterpret_cast<const float4*>(thin_smem + ((n8 >> log_s) * S + r) * kThinWarps * 512 + slot);
            total[n8][0] += v.x;
            total[n8][1] += v.y;
            total[n8][2] += v.z;
            total[n8][3] += v.w;
          }
    }
    // this warp's outputs straight from its fragments: row g and g + 8, tokens 2 t, 2 t + 1
    const int tile = tile0 + warp, f = tile * (GATED ? 8 : 16) + g;
    if (f >= p.n_out) continue;
    const int f8 = GATED ? p.n_out + f : f + 8;  // the weight row of the second half
    const bool low = GATED || f8 < p.n_out;
    const float b0 = p.bias ? p.bias[f] : 0.f, b1 = p.bias && low ? p.bias[f8] : 0.f;
    const int r0 = __ldg(p.row_exp + tile * 16 + g) - 127, r1 = __ldg(p.row_exp + tile * 16 + g + 8) - 127;
#pragma unroll
    for (int n8 = 0; n8 < NT; ++n8)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int tok = 8 * n8 + 2 * t + c;
        if (tok >= nt || (n8 & (S - 1)) != rank) continue;
        const size_t row = (size_t)(t0 + tok) * p.n_out;
        const int q = PACKED ? __ldcg(p.x_exp + t0 + tok) : down[c];
        const float v0 = scaled(total[n8][c], r0 + q, b0), v1 = scaled(total[n8][2 + c], r1 + q, b1);
        if constexpr (GATED) {
          out[row + f] = static_cast<X>(act_f<ACT>(v0) * v1);
        } else {
          out[row + f] = static_cast<X>(v0);
          if (low) out[row + f8] = static_cast<X>(v1);
        }
      }
  }
  // a copy waited for in vain may still land: report, and stay until it surely has
  if (!ok) {
    report_status(&g_thin_status, kStatusTimeoutMain);
    const uint64_t start = ptx::globaltimer_ns();
    while (ptx::globaltimer_ns() - start < kMatvecWaitNs / 50) __nanosleep(1000);
  }
}

// The largest group scale of each weight row, in tile order (127 past the matrix).
__device__ __forceinline__ long long matvec_raw_row(const MatvecLayout& L, long long tile, int r) {
  if (!L.gated) return tile * 16 + r < L.rows ? tile * 16 + r : -1;
  const long long f = tile * 8 + (r & 7);
  return f < L.rows / 2 ? f + (r >= 8 ? L.rows / 2 : 0) : -1;
}
// Byte offset of a tile's K unit.
__device__ __forceinline__ size_t matvec_unit_offset(const MatvecLayout& L, long long tile, int u) {
  return (((size_t)(tile / kMatvecGroup) * L.ku + u) * kMatvecGroup + tile % kMatvecGroup) * kMatvecUnitBytes;
}
__global__ void __launch_bounds__(256) matvec_row_exp_kernel(MatvecPrepareParams p) {
  const MatvecLayout& L = p.L;
  const long long i = (blockIdx.x * 256LL + threadIdx.x) >> 5;
  if (i >= (long long)L.tiles * 16) return;  // whole warps
  const long long row = matvec_raw_row(L, i >> 4, (int)(i & 15));
  const int groups = L.K / 32;
  uint32_t m = 0;
  if (row >= 0)
    for (int b = threadIdx.x & 31; b < groups; b += 32) {
      const uint32_t s = p.scales[(size_t)row * groups + b];
      if (s == 255) atomicOr(reinterpret_cast<unsigned int*>(p.dst + L.flag_off), 1u);
      m = max(m, s);
    }
  m = __reduce_max_sync(0xffffffffu, m);
  if ((threadIdx.x & 31) == 0) p.dst[L.exp_off + i] = row >= 0 ? (uint8_t)m : 127;
}

// One thread per 16-byte chunk of the prepared codes, then one per scale byte (relative
// to its row's largest, which the kernel before found).
__global__ void matvec_prepare_kernel(MatvecPrepareParams p) {
  const MatvecLayout& L = p.L;
  const int groups = L.K / 32;
  const long long chunks = (long long)L.tiles * L.ku * 64, scales = (long long)L.tiles * L.ku * 64;
  for (long long i = blockIdx.x * (long long)blockDim.x + threadIdx.x; i < chunks + scales;
       i += (long long)gridDim.x * blockDim.x) {
    if (i < chunks) {
      const int lane = (int)(i & 31), half = (int)((i >> 5) & 1);
      const long long unit = i >> 6, tile = unit / L.ku;
      const int u = (int)(unit - tile * L.ku);
      const long long row = matvec_raw_row(L, tile, (lane >> 2) + 8 * half);
      uint32_t w[4];
#pragma unroll
      for (int b = 0; b < 4; ++b)
        w[b] = row >= 0 && 128 * u + 32 * b < L.K
                   ? __ldg(reinterpret_cast<const uint32_t*>(p.codes + (size_t)row * (L.K / 2) + u * 64 + 16 * b) +
                           (lane & 3))
                   : 0u;
      reinterpret_cast<uint4*>(p.dst + matvec_unit_offset(L, tile, u))[i & 63] = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      const long long q = i - chunks, unit = q >> 6, tile = unit / L.ku;
      const int u = (int)(unit - tile * L.ku), g = (int)(q >> 3) & 7, half = (int)(q >> 2) & 1, b = (int)q & 3;
      const long long row = matvec_raw_row(L, tile, g + 8 * half);
      int s = 0;
      if (row >= 0 && 4 * u + b < groups) {
        s = 127 + (int)p.scales[(size_t)row * groups + 4 * u + b] - (int)p.dst[L.exp_off + tile * 16 + g + 8 * half];
        if (s < 0) s = 0;
      }
      p.dst[matvec_unit_offset(L, tile, u) + 1024 + (q & 63)] = (uint8_t)s;
    }
  }
}

// ------------------------------------------------------------------ 16-bit weights
// One tile of 16 rows per block; its eight warps split K, each loading eight units of 32
// values (16 bytes a lane and row) at a time straight to registers, so that two blocks per
// SM have 128 KB in flight.  Two or four tiles per block, which share the x fragments,
// measured slower at every size (16 tokens, 4096 x 14336: 71 and 76 us against 70; one
// token 57 and 70 against 55, 0.96 of the measured copy rate), and so did three and four
// blocks per SM with fewer units each.  Bound by HBM; at 2880 x 2880, where the two launches
// take 13.0 us for 50 MB, by their starts and by 1.2 and 0.6 rounds of blocks.
template <typename X, int NT, bool GATED, int ACT>
__global__ void __launch_bounds__(kThinThreads, 2) thin16_kernel(const __grid_constant__ ThinParams p) {
  constexpr int kUnits = 8;
  extern __shared__ __align__(128) uint8_t thin_smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int tile = blockIdx.x;
  const int u_end = (int)((long long)(warp + 1) * p.ku / kThinWarps);
  int u = (int)((long long)warp * p.ku / kThinWarps);
  // the two weight rows of this lane (rows past the matrix read the last row and are
  // dropped at the end)
  const int f = tile * (GATED ? 8 : 16) + g, last = p.n_out - 1;
  const uint16_t* w = reinterpret_cast<const uint16_t*>(p.w) + 8 * t;
  const uint16_t* row0 = w + (size_t)min(f, last) * p.K;
  const uint16_t* row1 = w + (size_t)(GATED ? p.n_out + min(f, last) : min(f + 8, last)) * p.K;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  uint4 wr[kUnits][2];
  auto load = [&](int from) {
#pragma unroll
    for (int j = 0; j < kUnits; ++j) {
      const bool live = from + j < u_end && (from + j) * 32 + 8 * t < p.K;
      wr[j][0] = live ? load_weights(row0 + (from + j) * 32) : zero;
      wr[j][1] = live ? load_weights(row1 + (from + j) * 32) : zero;
    }
  };
  if (p.early) {  // the weights, where the launch before is one of the same call
    load(u);
    ptx::pdl_wait();
    ptx::pdl_launch_dependents();
  } else {
    ptx::pdl_wait();
    ptx::pdl_launch_dependents();
    load(u);
  }
  const uint16_t* x = reinterpret_cast<const uint16_t*>(p.x) + 8 * t;
  float total[NT][4] = {};
  while (true) {
#pragma unroll
    for (int j = 0; j < kUnits; ++j) {
      const bool live = u + j < u_end && (u + j) * 32 + 8 * t < p.K;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const uint4 xf =
            live && g + 8 * n < p.T ? __ldcg(reinterpret_cast<const uint4*>(x + (size_t)(g + 8 * n) * p.K + (u + j) * 32)) : zero;
        const uint4 a = wr[j][0], b = wr[j][1];
        mma16816<X>(total[n], a.x, b.x, a.y, b.y, xf.x, xf.y);
        mma16816<X>(total[n], a.z, b.z, a.w, b.w, xf.z, xf.w);
      }
    }
    u += kUnits;
    if (u >= u_end) break;
    load(u);
  }
  finish<X, NT, GATED, ACT>(p, total, reinterpret_cast<float*>(thin_smem), tile);
}

// ------------------------------------------------------------------ launchers
template <typename X, int NT, bool PACKED, bool GATED, int ACT>
cudaError_t launch_matvec_t(ThinParams p, cudaStream_t stream) {
  using C = MatvecCfg<NT, PACKED>;
  const int groups_t = ceil_div(p.T, NT * 8);
  cudaError_t e;
  if constexpr (PACKED) {
    p.x_exp = reinterpret_cast<int32_t*>(p.packed + packed_bytes<NT>(p.T, p.ku));
    e = launch_pdl(matvec_pack_kernel<X, NT>, dim3(groups_t * NT * 8), dim3(256), 0, stream, p);
    if (e != cudaSuccess) return e;
  }
  // clusters along K while whole groups leave resident blocks idle and a block keeps two units
  const int groups = p.tiles / kMatvecGroup, resident = C::kPerSm * device_sms();
  p.log_kw = 0;
  while ((2 << p.log_kw) <= kMatvecMaxSplit && 2 * groups * groups_t << p.log_kw <= resident && p.ku >= 4 << p.log_kw)
    ++p.log_kw;
  const int split = 1 << p.log_kw;
  const int blocks = split > 1 || groups * groups_t < resident ? groups * split : max(1, resident / groups_t);
  const int smem = C::kRingBytes + (PACKED ? 0 : p.T * resident_row_halves(p.ku) * 2);
  auto kern = matvec_kernel<X, NT, PACKED, GATED, ACT>;
  static SmemOptIn opt_in;
  e = opt_in.ensure(kern, C::kRingBytes + (PACKED ? 0 : kResidentPieces * 256 + 8 * 64));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks, groups_t);
  cfg.blockDim = dim3(kThinThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {(unsigned)split, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = split > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

// Column groups of 8 tokens per block: up to four.
template <typename X, bool GATED, int ACT>
cudaError_t launch_matvec_nt(const ThinParams& p, cudaStream_t stream) {
  if (matvec_resident(p.T, p.ku)) return launch_matvec_t<X, 1, false, GATED, ACT>(p, stream);
  if (p.T <= 8) return launch_matvec_t<X, 1, true, GATED, ACT>(p, stream);
  if (p.T <= 16) return launch_matvec_t<X, 2, true, GATED, ACT>(p, stream);
  return launch_matvec_t<X, 4, true, GATED, ACT>(p, stream);
}

template <typename X, int NT, bool GATED, int ACT>
cudaError_t launch_thin16_t(const ThinParams& p, cudaStream_t stream) {
  return launch_pdl(thin16_kernel<X, NT, GATED, ACT>, dim3(p.tiles), dim3(kThinThreads), finish_bytes<NT>(), stream, p);
}

template <bool MX, typename X, bool GATED, int ACT>
cudaError_t launch_nt(const ThinParams& p, cudaStream_t stream) {
  if constexpr (MX) return launch_matvec_nt<X, GATED, ACT>(p, stream);
  return p.T <= 8 ? launch_thin16_t<X, 1, GATED, ACT>(p, stream) : launch_thin16_t<X, 2, GATED, ACT>(p, stream);
}

template <bool MX, typename X>
cudaError_t launch_act(const ThinParams& p, bool gated, cudaStream_t stream) {
  if (!gated) return launch_nt<MX, X, false, kActSilu>(p, stream);
  return p.act == kActSilu ? launch_nt<MX, X, true, kActSilu>(p, stream) : launch_nt<MX, X, true, kActGelu>(p, stream);
}

}  // namespace

cudaError_t launch_matvec(const ThinParams& p, int dtype, bool gated, cudaStream_t stream) {
  return dtype == kDtypeBf16 ? launch_act<true, __nv_bfloat16>(p, gated, stream)
                             : launch_act<true, __half>(p, gated, stream);
}

cudaError_t launch_thin16(const ThinParams& p, int dtype, bool gated, cudaStream_t stream) {
  return dtype == kDtypeBf16 ? launch_act<false, __nv_bfloat16>(p, gated, stream)
                             : launch_act<false, __half>(p, gated, stream);
}

size_t matvec_workspace_bytes(int T, int K) {
  const int ku = ceil_div(K, 128);
  if (matvec_resident(T, ku)) return 0;
  const size_t x = T <= 8 ? packed_bytes<1>(T, ku) : T <= 16 ? packed_bytes<2>(T, ku) : packed_bytes<4>(T, ku);
  return x + kMatvecMaxTokens * sizeof(int32_t);
}

uint32_t* thin_status_word() {
  void* p = nullptr;
  return cudaGetSymbolAddress(&p, g_thin_status) == cudaSuccess ? static_cast<uint32_t*>(p) : nullptr;
}

cudaError_t launch_matvec_prepare(const MatvecPrepareParams& p, cudaStream_t stream) {
  const long long rows = (long long)p.L.tiles * 16;
  matvec_row_exp_kernel<<<(unsigned)((rows + 7) / 8), 256, 0, stream>>>(p);
  matvec_prepare_kernel<<<1184, 256, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace moe
