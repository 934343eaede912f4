// Launch parameters and launchers of the dense operators around the expert layer: the
// norms before and after a block, the gated feed-forward block and the products of a
// few tokens with MXFP4 weights (internal to the library).
#pragma once

#include <cuda.h>

#include "moe_common.cuh"
#include "moe_kernels.cuh"

namespace moe {

// SMs of the current device (looked up once per device).
inline int device_sms() {
  static std::atomic<int> cached[kMaxDevices] = {};
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return kMaxCtas;
  const bool keep = dev >= 0 && dev < kMaxDevices;
  if (keep && (n = cached[dev].load(std::memory_order_relaxed)) > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) return kMaxCtas;
  if (keep) cached[dev].store(n, std::memory_order_relaxed);
  return n;
}

// ------------------------------------------------------------------ element types
constexpr int kDtypeBf16 = 0, kDtypeF16 = 1, kDtypeF32 = 2;

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }

// Two 16-bit values of one 32-bit word as floats, and back (nearest, ties to even).
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t w);
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Eight consecutive values as floats.  load() reads through L2 only: the kernels overlap
// their neighbours, and a row updated in place by the kernel before may share a sector
// with a row that this SM read earlier.  load_weight() may use L1.
template <typename T>
struct Vec8 {
  uint4 raw;
  __device__ __forceinline__ void load(const void* base, size_t vec) {
    raw = __ldcg(reinterpret_cast<const uint4*>(base) + vec);
  }
  __device__ __forceinline__ void load_weight(const void* base, size_t vec) {
    raw = reinterpret_cast<const uint4*>(base)[vec];
  }
  __device__ __forceinline__ void load_shared(const void* base, int vec) { raw = reinterpret_cast<const uint4*>(base)[vec]; }
  __device__ __forceinline__ void zero() { raw = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = unpack2<T>(w[i]);
      f[2 * i] = v.x;
      f[2 * i + 1] = v.y;
    }
  }
  __device__ __forceinline__ void set(const float (&f)[8]) {
    raw = make_uint4(pack2<T>(f[0], f[1]), pack2<T>(f[2], f[3]), pack2<T>(f[4], f[5]), pack2<T>(f[6], f[7]));
  }
  __device__ __forceinline__ void store(void* base, size_t vec) const { reinterpret_cast<uint4*>(base)[vec] = raw; }
};
template <>
struct Vec8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const void* base, size_t vec) {
    a = __ldcg(reinterpret_cast<const float4*>(base) + 2 * vec);
    b = __ldcg(reinterpret_cast<const float4*>(base) + 2 * vec + 1);
  }
  __device__ __forceinline__ void load_shared(const void* base, int vec) {
    a = reinterpret_cast<const float4*>(base)[2 * vec];
    b = reinterpret_cast<const float4*>(base)[2 * vec + 1];
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
  __device__ __forceinline__ void set(const float (&f)[8]) {
    a = make_float4(f[0], f[1], f[2], f[3]);
    b = make_float4(f[4], f[5], f[6], f[7]);
  }
  __device__ __forceinline__ void store(void* base, size_t vec) const {
    reinterpret_cast<float4*>(base)[2 * vec] = a;
    reinterpret_cast<float4*>(base)[2 * vec + 1] = b;
  }
};

// ------------------------------------------------------------------ activations
constexpr int kActSilu = 0, kActGelu = 1, kActNone = 2;

// act(g) and, in the second form, its derivative too.  SiLU: g * s with s = 1 / (1 +
// e^-g), derivative s (1 + g (1 - s)).  GELU (tanh form): with t = tanh(c (g + b g^3)),
// g (1 + t) / 2 and (1 + t) / 2 + g (1 - t^2) c (1 + 3 b g^2) / 2; (1 + t) / 2 is taken
// as 1 / (1 + e^-2v), which keeps the left tail's relative precision.
__device__ __forceinline__ float sigmoid_f(float v) { return __fdividef(1.f, 1.f + __expf(-v)); }
template <int ACT>
__device__ __forceinline__ float act_f(float g) {
  if constexpr (ACT == kActSilu) return g * sigmoid_f(g);
  constexpr float c = 0.7978845608028654f, b = 0.044715f;
  return g * sigmoid_f(2.f * c * (g + b * g * g * g));
}
template <int ACT>
__device__ __forceinline__ float act_f(float g, float& slope) {
  if constexpr (ACT == kActSilu) {
    const float s = sigmoid_f(g);
    slope = s * (1.f + g * (1.f - s));
    return g * s;
  }
  constexpr float c = 0.7978845608028654f, b = 0.044715f;
  const float s = sigmoid_f(2.f * c * (g + b * g * g * g));  // (1 + t) / 2
  slope = s + g * (2.f * s * (1.f - s)) * (c * (1.f + 3.f * b * g * g));
  return g * s;
}

// ------------------------------------------------------------------ norms around a block
constexpr int kGateNone = 0, kGateFeature = 1, kGateToken = 2, kGateFull = 3;
constexpr int kNormBlocks = 152;    // blocks of the backward, each a row of partial weight gradients
constexpr int kNormMaxGroups = 15;  // rows that one of them takes side by side (a named barrier each)

struct BlockNormParams {
  const void* block;        // z [T, H]
  const void* norm_w;       // [H] or null: no norm after the block
  const void* gate;         // [H], f32 [T] or [T, H] by gate_kind
  const void* residual;     // r [T, H] (stream type) or null
  const void* next_w;       // [H] or null: no norm before the next block
  int gate_kind, T, H;
  float scale, eps;
  void* residual_out;       // s [T, H] (stream type) or null
  void* out;                // y [T, H]; beside an 8-bit output, or null
  uint8_t* codes;           // 8-bit output: [T, H] E4M3
  void* scales;             // its scales: E8M0 [T, H / 32] or f32 [T]
};
// The form of the norm's output: y as it is, or E4M3 codes with an E8M0 scale for 32 values, or
// with an f32 scale for a row.
constexpr int kOut16 = 0, kOutMx = 1, kOutRow = 2;
struct BlockNormBackwardParams {
  BlockNormParams f;          // residual unused; residual_out is the forward's s, read
  const void* d_residual_out; // [T, H] (stream type) or null
  const void* d_out;          // [T, H]; null without next_w
  void* d_block;              // [T, H]
  void* d_residual;           // [T, H] (stream type) or null
  void* d_gate;               // f32 [H], f32 [T] or [T, H] by gate_kind, or null
  float* d_norm_w;            // f32 [H] or null
  float* d_next_w;            // f32 [H] or null
  float* partial;             // f32 [rows of partials][3][H]: next, norm, feature gate
  int blocks;                 // persistent blocks = rows of partials
};
cudaError_t launch_block_norm(const BlockNormParams& p, int dtype, int stream_dtype, int out_kind, cudaStream_t stream);
int block_norm_backward_groups(int H);
int block_norm_backward_blocks(int T, int H);
uint32_t* norm_status_word();
cudaError_t launch_block_norm_backward(const BlockNormBackwardParams& p, int dtype, int stream_dtype,
                                       cudaStream_t stream);

// ------------------------------------------------------------------ tokens sorted by expert
struct SortParams {
  const int32_t* idx;       // [T, k]; outside [0, E): dropped
  const void *x, *scales;   // [T] rows of row_bytes, and of scale_bytes (or null)
  int T, k, E, row_bytes, scale_bytes;
  int32_t *offsets, *perm, *inv_perm;  // [E + 1], [T k], [T k]
  void *rows, *row_scales;  // [T k] rows
  uint64_t wait_ns;         // limit of a wait for a row
};
struct UnsortParams {
  const void* y;            // [T k, H]
  const int32_t* inv_perm;  // [T, k]; negative: dropped
  const float* w;           // [T, k] or null: 1
  int T, k, H;
  void* out;                // [T, H]
  uint64_t wait_ns;         // limit of a wait for a row
};
struct UnsortBackwardParams {
  UnsortParams f;           // out unused
  const void* d_out;        // [T, H]
  void* d_y;                // [T k, H] or null
  float* d_w;               // [T, k] or null
};
struct RouteBackwardParams {
  const float *d_w, *logits, *w;  // [T, k], [T, E], [T, k]
  const int32_t* idx;       // [T, k]
  int T, k, E, gating;
  float* d_logits;          // [T, E]
};
uint32_t* sort_status_word();
cudaError_t launch_sort(const SortParams& p, cudaStream_t stream);
cudaError_t launch_unsort(const UnsortParams& p, int dtype, cudaStream_t stream);
cudaError_t launch_unsort_backward(const UnsortBackwardParams& q, int dtype, cudaStream_t stream);
cudaError_t launch_route_backward(const RouteBackwardParams& p, cudaStream_t stream);

// ------------------------------------------------------------------ products of a few tokens
constexpr int kThinTokens = 16;   // tokens of the 16-bit few-token kernel
constexpr int kThinRows = 16;     // weight rows of one of their tiles (MMA M)
constexpr int kMatvecMaxTokens = 64;

// Prepared MXFP4 weights of the few-token products.  Tiles of 16 rows (plain: rows 16 i
// ..; gated: gate rows 8 i .. then up rows 8 i ..), cut along K into units of 128 codes:
//   [tiles / 8][KU][8 tiles] units of 1088 bytes: [2][32 lanes][16 bytes] codes -- lane
//   4 g + t holds, of row g (first half) or g + 8 (second), word t (codes 8 t .. 8 t + 7)
//   of each of the unit's four 32-code groups, so one 16-byte read per lane and half feeds
//   eight MMAs -- then [8 g][2 halves][4 groups] scale bytes, 127 + the E8M0 byte - the
//   row's largest (0, which counts as a scale of 0, for groups below 2^-126 of it);
//   [tiles][16] the rows' largest E8M0 bytes;
//   trailer (256 bytes): set when a scale byte of 255 (NaN) was met.
// Tiles are rounded up to eight; rows and codes past the matrix are zero.  Eight tiles' K
// units, and so a run of K for 128 rows, are contiguous.
constexpr int kMatvecUnitBytes = 1024 + 64;
constexpr int kMatvecGroup = 8;
struct MatvecLayout {
  int rows, K, gated, tiles, ku;  // tiles: rounded up to whole groups
  size_t exp_off, flag_off, total;
};
inline MatvecLayout make_matvec_layout(int rows, int K, int gated) {
  MatvecLayout L{};
  L.rows = rows;
  L.K = K;
  L.gated = gated;
  L.tiles = gated ? ceil_div(rows / 2, kThinRows / 2) : ceil_div(rows, kThinRows);
  L.tiles = ceil_div(L.tiles, kMatvecGroup) * kMatvecGroup;
  L.ku = ceil_div(K, 128);
  L.exp_off = (size_t)L.tiles * L.ku * kMatvecUnitBytes;
  L.flag_off = align_up(L.exp_off + (size_t)L.tiles * 16, 256);
  L.total = L.flag_off + 256;
  return L;
}
struct MatvecPrepareParams {
  const uint8_t *codes, *scales;
  MatvecLayout L;
  uint8_t* dst;
};
cudaError_t launch_matvec_prepare(const MatvecPrepareParams& p, cudaStream_t stream);

struct ThinParams {
  const void* x;            // [T, K]
  const void* w;            // prepared MXFP4 tiles, or 16-bit rows [rows, K]
  const float* bias;        // f32 [rows] or null (MXFP4 only)
  int T, K, n_out;          // n_out: output features (gated: half the rows)
  int tiles, ku;            // row tiles, K units (128 codes, or 32 16-bit values)
  int act;
  int early;                // 16-bit: the weights may be read before the dependency wait
  int log_kw;               // MXFP4: log2 of the blocks of a cluster, which split K
  const uint8_t* row_exp;   // MXFP4: the rows' largest E8M0 bytes, tile order
  uint8_t* packed;          // MXFP4: workspace for x in fragment order
  int32_t* x_exp;           // MXFP4: and, behind it, the powers of two taken out of its tokens
  void* out;                // [T, n_out]
  float* gateup;            // f32 [T, 2 n_out] or null: the products before the activation
  const void* residual;     // projections: [T, n_out] of out's type, or null
  int out_f32;              // projections: out's type
};
// Outer products of up to kThinOuterTokens tokens: out [N, K] = a^T b, a [T, N], b [T, K].
constexpr int kThinOuterTokens = 64;
struct ThinOuterParams {
  const void *a, *b;
  int T, N, K;
  void* out;
};
cudaError_t launch_thin_outer(const ThinOuterParams& p, int dtype, cudaStream_t stream);
cudaError_t launch_thin_linear(const ThinParams& p, int dtype, cudaStream_t stream);
cudaError_t launch_matvec(const ThinParams& p, int dtype, bool gated, cudaStream_t stream);
cudaError_t launch_thin16(const ThinParams& p, int dtype, bool gated, cudaStream_t stream);
size_t matvec_workspace_bytes(int T, int K);
uint32_t* thin_status_word();  // device addresses on the current device, or null
uint32_t* dense_status_word();

// ------------------------------------------------------------------ gradient of a projection's epilogue
// dp = d_out act'(pre), rounded to 16 bits, and its column sums before that rounding.
struct LinearGradParams {
  const void* d_out;        // [T, N] of `dtype` or f32
  const float* pre;         // f32 [T, N]; null: no activation
  void* dp;                 // 16-bit [T, N] or null
  float* d_bias;            // f32 [N] or null
  float* partial;           // f32 [splits][N]
  int T, N, act, splits;    // splits: blocks along T
};
int linear_grad_splits(int T, int N);
cudaError_t launch_linear_grad(const LinearGradParams& p, int dtype, int out_dtype, cudaStream_t stream);

// ------------------------------------------------------------------ dense GEMMs
// C[m, n] = sum_k A[m, k] B[n, k] of 16-bit operands, each stored with K or with M / N
// contiguous, and one of several epilogues.
constexpr int kDenseStore = 0;       // C in the operands' type
constexpr int kDenseGateUp = 1;      // B rows: gate, then up; h = act(g) u, and g, u in f32 when asked for
constexpr int kDenseGateUpGrad = 2;  // C = dh: dg, du from the saved g, u; and h again
constexpr int kDenseProducts = 3;    // several products, each as kDenseStore
constexpr int kDenseLinear = 4;      // out = act(C + bias) + residual; and C + bias in f32 when asked for
constexpr int kDenseLinear32 = 5;    // the same with out and residual in f32
constexpr int kDenseMaxSplits = 16;

// One product: C [M, N] = A B^T.
struct DenseProblem {
  CUtensorMap tm_a, tm_b;
  int M, N, K;              // N: output columns (gate/up: features, half of B's rows)
  int a_mn, b_mn;           // operand stored with M (N) contiguous
  int tiles_m, tiles_n, kgroups;  // K groups of 64
  void* out;                // 16-bit [M, N]; gate/up grad: dgu [M, 2 N]
};
constexpr int kDenseGroup = 3;  // products of one launch
struct DenseGemmParams {
  DenseProblem g[kDenseGroup];
  int bn;                   // columns of a tile
  int full, splits;         // tiles after the first `full` are cut into `splits` slices of K
  int group, long_n, lead;  // several products: how many, those of the long class, and the lead (see below)
  int act;
  void* out_h;              // gate/up grad: h [M, N]
  float* gateup;            // f32 [M, 2 N]: written by gate/up (or null), read by its gradient; linear: [M, N] or null
  const float* bias;        // linear: f32 [N] or null
  const void* residual;     // linear: [M, N] of out's type, or null
  float* partial;           // f32 [slices][tile rows][tile columns]
  uint64_t wait_ns;
};
struct DenseOperand {
  const void* ptr;
  int rows, cols;           // as stored, row major
  int mn_major;             // the columns are M (or N), the rows K
};
// One product with the tile shape chosen by size; `partial` (f32) holds
// dense_partial_bytes() bytes and is used when K is split.
size_t dense_partial_bytes(int M, int N, int K, int mode, bool b_mn);
int launch_dense_gemm(DenseGemmParams p, const DenseOperand& a, const DenseOperand& b, int mode, int dtype,
                      cudaStream_t stream);
// A projection (bias, act, residual, gateup as kDenseLinear) of up to kBatchTokens tokens, or,
// with w MN-major, the product with its columns.
constexpr int kBatchTokens = 128;
int launch_linear_batch(DenseGemmParams p, const DenseOperand& x, const DenseOperand& w, int dtype, bool wide, cudaStream_t stream);
// Up to kDenseGroup plain products (g[i].M, N, K, out set) whose K takes at most two values,
// in one launch where that is estimated to be faster.  few_rows: the estimate takes account of
// tiles too few to fill the GPU (the feed-forward block's does not: its results stay what they are).
int launch_dense_products(DenseGemmParams p, int n, const DenseOperand* a, const DenseOperand* b, int dtype, bool few_rows,
                          cudaStream_t stream);

}  // namespace moe
