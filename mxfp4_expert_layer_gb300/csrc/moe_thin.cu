// Products of a few tokens with many weight rows (decode): MXFP4 weights, and the
// 16-bit weights of the dense feed-forward block.
//   plain  y[t, n] = sum_k x[t, k] W[n, k] (+ bias[n])
//   gated  h[t, i] = act(g) u,  g and u the products with gate row i and up row i
//
// At these sizes every weight byte is read once and used for at most 16 tokens, so the
// kernels are bound by HBM, and what matters is the bytes in flight and the
// instructions spent per weight.  One block takes RT tiles of 16 weight rows; its eight
// warps split K and add their sums through shared memory in warp order (no partial
// sums leave the block, and the order is fixed).  The products run on mma.sync
// (m16n8k16, f32 sums): the weights are the 16-row operand, up to 8 tokens a column
// group.  The sum over K is free to take its terms in any order, so each lane's
// 16-byte weight load is its own operand fragments, with x permuted to match: no
// shuffles and no shared memory on the weight side.
//
// MXFP4: two codes become an f16 pair by one conversion instruction (exact); a group's
// 32 products are summed by two MMAs and then scaled in f32 by the group's E8M0 scale.
// x as f16: a power of two per (token, K chunk) brings its largest value to [2^14,
// 2^15), so bf16 values are exact down to 2^-28 of the largest (absolute error 2^-39 of
// it below), and is taken out again in f32.
#include "moe_dense.cuh"
#include "sm100_ptx.cuh"

namespace moe {

namespace {

constexpr int kThinThreads = 256;
constexpr int kThinWarps = kThinThreads / 32;

template <typename X>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__half>(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                 uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
               "%2, %3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, "
               "%1, %2, %3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The eight E2M1 codes of a word as four f16 pairs (low nibble first).
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// 2^(byte - 127); byte 0 is the subnormal 2^-127.
__device__ __forceinline__ float e8m0_f32(uint32_t word, int b) {
  return __uint_as_float(max(((word >> (8 * b)) & 0xFFu) << 23, 0x00400000u));
}

__device__ __forceinline__ uint4 load_weights(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// Adds the warps' sums (fragment layout: register pair c < 2 is row g, c >= 2 row g + 8,
// token 2 t + (c & 1)) in warp order and writes the block's outputs.
template <typename X, int NT, int RT, bool GATED, int ACT>
__device__ __forceinline__ void finish(const ThinParams& p, const float (&total)[RT][NT][4], float* red, int tile0,
                                       int t0, int nt) {
  constexpr int kRows = RT * kThinRows, kStride = kRows + 4;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 4; ++c)
        red[(warp * NT * 8 + n * 8 + 2 * t + (c & 1)) * kStride + rt * 16 + g + 8 * (c >> 1)] = total[rt][n][c];
  __syncthreads();
  constexpr int kOut = GATED ? kRows / 2 : kRows;
  X* out = reinterpret_cast<X*>(p.out);
  for (int i = threadIdx.x; i < nt * kOut; i += kThinThreads) {
    const int tok = i / kOut, o = i - tok * kOut;
    const size_t row = (size_t)(t0 + tok);
    auto sum = [&](int r) {
      float v = red[tok * kStride + r];
#pragma unroll
      for (int w = 1; w < kThinWarps; ++w) v += red[(w * NT * 8 + tok) * kStride + r];
      return v;
    };
    if constexpr (GATED) {
      const int f = tile0 * 8 + o, r = (o >> 3) * 16 + (o & 7);
      if (f >= p.n_out) continue;
      float gv = sum(r), uv = sum(r + 8);
      if (p.bias) {
        gv += p.bias[f];
        uv += p.bias[p.n_out + f];
      }
      if (p.gateup) {
        p.gateup[row * 2 * p.n_out + f] = gv;
        p.gateup[row * 2 * p.n_out + p.n_out + f] = uv;
      }
      out[row * p.n_out + f] = static_cast<X>(act_f<ACT>(gv) * uv);
    } else {
      const int f = tile0 * 16 + o;
      if (f >= p.n_out) continue;
      float v = sum(o);
      if (p.bias) v += p.bias[f];
      out[row * p.n_out + f] = static_cast<X>(v);
    }
  }
}

// ------------------------------------------------------------------ MXFP4 weights
template <typename X, int NT, int RT>
struct MatvecCfg {
  static constexpr int kUnits = RT == 4 ? 1 : RT == 2 ? 2 : 4;  // K units per chunk: 4 unit tiles in flight
  static constexpr int kRowHalves = kUnits * 128 + 32;          // x row in shared memory (64 bytes of padding)
  static int smem(int tokens) {
    const int x = kThinWarps * tokens * kRowHalves * 2;
    const int red = kThinWarps * NT * 8 * (RT * kThinRows + 4) * 4;
    return x > red ? x : red;
  }
};

template <typename X, int NT, int RT, bool GATED, int ACT>
__global__ void __launch_bounds__(kThinThreads) matvec_kernel(const __grid_constant__ ThinParams p) {
  using C = MatvecCfg<X, NT, RT>;
  extern __shared__ __align__(128) uint8_t thin_smem[];
  __shared__ float s_scale[kThinWarps][NT * 8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int tile0 = blockIdx.x * RT, t0 = blockIdx.y * kThinTokens;
  const int nt = min(p.T - t0, NT * 8);
  const int u_end = (int)((long long)(warp + 1) * p.ku / kThinWarps);
  int u = (int)((long long)warp * p.ku / kThinWarps);
  uint16_t* xs = reinterpret_cast<uint16_t*>(thin_smem) + (size_t)warp * nt * C::kRowHalves;
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  float total[RT][NT][4] = {};
  for (; u < u_end; u += C::kUnits) {
    // this chunk's weights, all loads in flight at once
    uint4 wr[RT][C::kUnits][2];
    uint2 sc[RT][C::kUnits];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const size_t tile = min(tile0 + rt, p.tiles - 1);
#pragma unroll
      for (int j = 0; j < C::kUnits; ++j) {
        const size_t unit = tile * p.ku + min(u + j, p.ku - 1);
        const uint8_t* src = reinterpret_cast<const uint8_t*>(p.w) + unit * 1024 + lane * 16;
        wr[rt][j][0] = load_weights(src);
        wr[rt][j][1] = load_weights(src + 512);
        sc[rt][j] = __ldg(reinterpret_cast<const uint2*>(p.w_sf + unit * 64) + g);
      }
    }
    // x of this chunk as f16 in shared memory (this warp's own), zero past K and past
    // the warp's last unit
    const int k0 = u * 128, k1 = min(u_end * 128, p.K);
    __syncwarp();
    for (int tok = 0; tok < nt; ++tok) {
      const uint4* row = reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p.x) + (size_t)(t0 + tok) * p.K);
      constexpr int kVecs = C::kUnits * 16, kPer = (kVecs + 31) / 32;
      uint4 v[kPer];
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int q = lane + 32 * i;
        v[i] = make_uint4(0, 0, 0, 0);
        if (q < kVecs && k0 + 8 * q < k1) v[i] = __ldcg(row + (k0 >> 3) + q);
      }
      if constexpr (sizeof(X) == 2 && !std::is_same<X, __half>::value) {
        // largest finite exponent of the chunk, then x * 2^p with that exponent at 14
        uint32_t emax = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t lo = (w[j] >> 7) & 0xFFu, hi = (w[j] >> 23) & 0xFFu;
            emax = max(emax, max(lo == 255u ? 0u : lo, hi == 255u ? 0u : hi));
          }
        }
        emax = __reduce_max_sync(0xffffffffu, emax);
        const int pw = emax == 0 ? 0 : min(126, 14 + 127 - (int)emax);
        const float up = pow2_int(pw);
        if (lane == 0) s_scale[warp][tok] = pow2_int(-pw);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 f = unpack2<__nv_bfloat16>(w[j]);
            w[j] = pack2<__half>(f.x * up, f.y * up);
          }
          v[i] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int q = lane + 32 * i;
        if (q < kVecs) *reinterpret_cast<uint4*>(xs + tok * C::kRowHalves + 8 * q) = v[i];
      }
    }
    __syncwarp();
    float acc[RT][NT][4] = {};
#pragma unroll
    for (int j = 0; j < C::kUnits; ++j) {
      if (u + j >= u_end) break;
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        uint4 xf[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          xf[n] = make_uint4(0, 0, 0, 0);
          if (g + 8 * n < nt)
            xf[n] = *reinterpret_cast<const uint4*>(xs + (g + 8 * n) * C::kRowHalves + j * 128 + 32 * b + 8 * t);
        }
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          const uint4 w0 = wr[rt][j][0], w1 = wr[rt][j][1];
          uint32_t h0[4], h1[4];
          e2m1x8_to_f16(b == 0 ? w0.x : b == 1 ? w0.y : b == 2 ? w0.z : w0.w, h0);
          e2m1x8_to_f16(b == 0 ? w1.x : b == 1 ? w1.y : b == 2 ? w1.z : w1.w, h1);
          const float s0 = e8m0_f32(sc[rt][j].x, b), s1 = e8m0_f32(sc[rt][j].y, b);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            float d[4] = {0.f, 0.f, 0.f, 0.f};
            mma16816<__half>(d, h0[0], h1[0], h0[1], h1[1], xf[n].x, xf[n].y);
            mma16816<__half>(d, h0[2], h1[2], h0[3], h1[3], xf[n].z, xf[n].w);
            acc[rt][n][0] = fmaf(d[0], s0, acc[rt][n][0]);
            acc[rt][n][1] = fmaf(d[1], s0, acc[rt][n][1]);
            acc[rt][n][2] = fmaf(d[2], s1, acc[rt][n][2]);
            acc[rt][n][3] = fmaf(d[3], s1, acc[rt][n][3]);
          }
        }
      }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float q0 = 1.f, q1 = 1.f;
      if constexpr (!std::is_same<X, __half>::value) {
        const int a = 8 * n + 2 * t;
        q0 = a < nt ? s_scale[warp][a] : 0.f;
        q1 = a + 1 < nt ? s_scale[warp][a + 1] : 0.f;
      }
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        total[rt][n][0] = fmaf(acc[rt][n][0], q0, total[rt][n][0]);
        total[rt][n][1] = fmaf(acc[rt][n][1], q1, total[rt][n][1]);
        total[rt][n][2] = fmaf(acc[rt][n][2], q0, total[rt][n][2]);
        total[rt][n][3] = fmaf(acc[rt][n][3], q1, total[rt][n][3]);
      }
    }
  }
  __syncthreads();  // every warp is done with its x before the sums take the same memory
  finish<X, NT, RT, GATED, ACT>(p, total, reinterpret_cast<float*>(thin_smem), tile0, t0, nt);
}

// One thread per 16-byte chunk of the prepared codes, then one per scale byte.
__global__ void matvec_prepare_kernel(MatvecPrepareParams p) {
  const MatvecLayout& L = p.L;
  const int half_rows = L.rows / 2, groups = L.K / 32;
  auto row_of = [&](long long tile, int r) -> long long {  // raw row, or -1
    if (!L.gated) return tile * 16 + r < L.rows ? tile * 16 + r : -1;
    const long long f = tile * 8 + (r & 7);
    return f < half_rows ? f + (r >= 8 ? half_rows : 0) : -1;
  };
  const long long chunks = (long long)L.tiles * L.ku * 64, scales = (long long)L.tiles * L.ku * 64;
  for (long long i = blockIdx.x * (long long)blockDim.x + threadIdx.x; i < chunks + scales;
       i += (long long)gridDim.x * blockDim.x) {
    if (i < chunks) {
      const int lane = (int)(i & 31), half = (int)((i >> 5) & 1);
      const long long unit = i >> 6, tile = unit / L.ku;
      const int u = (int)(unit - tile * L.ku);
      const long long row = row_of(tile, (lane >> 2) + 8 * half);
      uint32_t w[4];
#pragma unroll
      for (int b = 0; b < 4; ++b)
        w[b] = row >= 0 && 128 * u + 32 * b < L.K
                   ? __ldg(reinterpret_cast<const uint32_t*>(p.codes + (size_t)row * (L.K / 2) + u * 64 + 16 * b) +
                           (lane & 3))
                   : 0u;
      reinterpret_cast<uint4*>(p.dst)[i] = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      const long long q = i - chunks, unit = q >> 6, tile = unit / L.ku;
      const int u = (int)(unit - tile * L.ku), g = (int)(q >> 3) & 7, half = (int)(q >> 2) & 1, b = (int)q & 3;
      const long long row = row_of(tile, g + 8 * half);
      uint8_t s = 127;
      if (row >= 0 && 4 * u + b < groups) {
        s = p.scales[(size_t)row * groups + 4 * u + b];
        if (s == 255) atomicOr(reinterpret_cast<unsigned int*>(p.dst + L.flag_off), 1u);
      }
      p.dst[L.scales_off + q] = s;
    }
  }
}

// ------------------------------------------------------------------ 16-bit weights
template <typename X, int NT, int RT, bool GATED, int ACT>
__global__ void __launch_bounds__(kThinThreads) thin16_kernel(const __grid_constant__ ThinParams p) {
  constexpr int kUnits = RT == 4 ? 2 : RT == 2 ? 4 : 8;  // 32-value units per chunk: 8 unit tiles in flight
  extern __shared__ __align__(128) uint8_t thin_smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int tile0 = blockIdx.x * RT, t0 = blockIdx.y * kThinTokens;
  const int nt = min(p.T - t0, NT * 8);
  const int u_end = (int)((long long)(warp + 1) * p.ku / kThinWarps);
  int u = (int)((long long)warp * p.ku / kThinWarps);
  // the two weight rows of this lane in each tile (rows past the matrix read the last row
  // and are dropped at the end)
  const uint16_t* w = reinterpret_cast<const uint16_t*>(p.w);
  const uint16_t* rows[RT][2];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    if constexpr (GATED) {
      const int f = min((tile0 + rt) * 8 + g, p.n_out - 1);
      rows[rt][0] = w + (size_t)f * p.K;
      rows[rt][1] = w + (size_t)(p.n_out + f) * p.K;
    } else {
      const int f = (tile0 + rt) * 16 + g;
      rows[rt][0] = w + (size_t)min(f, p.n_out - 1) * p.K;
      rows[rt][1] = w + (size_t)min(f + 8, p.n_out - 1) * p.K;
    }
  }
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  const uint16_t* x = reinterpret_cast<const uint16_t*>(p.x) + (size_t)t0 * p.K;
  float total[RT][NT][4] = {};
  const uint4 zero = make_uint4(0, 0, 0, 0);
  for (; u < u_end; u += kUnits) {
    uint4 wr[RT][kUnits][2];
#pragma unroll
    for (int j = 0; j < kUnits; ++j) {
      const int k = (u + j) * 32 + 8 * t;
      const bool live = u + j < u_end && k < p.K;
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        wr[rt][j][0] = live ? load_weights(rows[rt][0] + k) : zero;
        wr[rt][j][1] = live ? load_weights(rows[rt][1] + k) : zero;
      }
    }
#pragma unroll
    for (int j = 0; j < kUnits; ++j) {
      const int k = (u + j) * 32 + 8 * t;
      const bool live = u + j < u_end && k < p.K;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const uint4 xf =
            live && g + 8 * n < nt ? __ldcg(reinterpret_cast<const uint4*>(x + (size_t)(g + 8 * n) * p.K + k)) : zero;
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          const uint4 a = wr[rt][j][0], b = wr[rt][j][1];
          mma16816<X>(total[rt][n], a.x, b.x, a.y, b.y, xf.x, xf.y);
          mma16816<X>(total[rt][n], a.z, b.z, a.w, b.w, xf.z, xf.w);
        }
      }
    }
  }
  finish<X, NT, RT, GATED, ACT>(p, total, reinterpret_cast<float*>(thin_smem), tile0, t0, nt);
}

// ------------------------------------------------------------------ launchers
template <bool MX, typename X, int NT, int RT, bool GATED, int ACT>
cudaError_t launch_t(const ThinParams& p, cudaStream_t stream) {
  const int red = kThinWarps * NT * 8 * (RT * kThinRows + 4) * 4;
  const dim3 grid(ceil_div(p.tiles, RT), ceil_div(p.T, kThinTokens));
  static SmemOptIn opt_in;
  if constexpr (MX) {
    auto kern = matvec_kernel<X, NT, RT, GATED, ACT>;
    const int tokens = p.T < NT * 8 ? p.T : NT * 8;
    const cudaError_t e = opt_in.ensure(kern, MatvecCfg<X, NT, RT>::smem(NT * 8));
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, grid, dim3(kThinThreads), MatvecCfg<X, NT, RT>::smem(tokens), stream, p);
  } else {
    auto kern = thin16_kernel<X, NT, RT, GATED, ACT>;
    const cudaError_t e = opt_in.ensure(kern, red);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, grid, dim3(kThinThreads), red, stream, p);
  }
}

// Row tiles per block: as many (up to four) as leave two blocks for every SM -- more
// tiles share each x fragment, fewer leave SMs without work.
template <bool MX, typename X, int NT, bool GATED, int ACT>
cudaError_t launch_rt(const ThinParams& p, cudaStream_t stream) {
  const int want = 2 * kMaxCtas;
  if (ceil_div(p.tiles, 4) >= want) return launch_t<MX, X, NT, 4, GATED, ACT>(p, stream);
  if (ceil_div(p.tiles, 2) >= want) return launch_t<MX, X, NT, 2, GATED, ACT>(p, stream);
  return launch_t<MX, X, NT, 1, GATED, ACT>(p, stream);
}

template <bool MX, typename X, bool GATED, int ACT>
cudaError_t launch_nt(const ThinParams& p, cudaStream_t stream) {
  return p.T <= 8 ? launch_rt<MX, X, 1, GATED, ACT>(p, stream) : launch_rt<MX, X, 2, GATED, ACT>(p, stream);
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

cudaError_t launch_matvec_prepare(const MatvecPrepareParams& p, cudaStream_t stream) {
  matvec_prepare_kernel<<<1184, 256, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace moe
