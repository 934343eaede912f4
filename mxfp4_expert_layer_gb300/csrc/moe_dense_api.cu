// C ABI of the dense operators around the expert layer: argument checks and launches.
#include <cuda_runtime.h>

#include "moe_dense.cuh"

using namespace moe;

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool overlap(const void* a, size_t a_bytes, const void* b, size_t b_bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + b_bytes && y < x + a_bytes;
}
int cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

static_assert(MOE_DTYPE_BF16 == kDtypeBf16 && MOE_DTYPE_F16 == kDtypeF16 && MOE_DTYPE_F32 == kDtypeF32, "dtype codes");
static_assert(MOE_GATE_NONE == kGateNone && MOE_GATE_FEATURE == kGateFeature && MOE_GATE_TOKEN == kGateToken &&
                  MOE_GATE_FULL == kGateFull, "gate kinds");
static_assert(MOE_ACT_SILU == kActSilu && MOE_ACT_GELU == kActGelu && MOE_ACT_NONE == kActNone, "activations");

constexpr int kMaxRows = 1 << 24;      // tokens of a call
constexpr int kMaxNormDim = 8192;      // a row sits in one block's registers
constexpr int kMaxFfnDim = 1 << 17;    // H and I of the feed-forward block
constexpr int kMaxLinearOut = 1 << 20;   // N of a projection (K as kMaxFfnDim)
constexpr int kMaxMovedBytes = 1 << 16;  // a row moved between token and expert order
constexpr int kMaxScaleBytes = 1 << 12;  // and its scales
constexpr int kMaxMatvecRows = 1 << 22, kMaxMatvecDim = 1 << 16;

bool dtype16(int d) { return d == MOE_DTYPE_BF16 || d == MOE_DTYPE_F16; }

int check_norm(const void* block, const void* norm_weight, const void* gate, int gate_kind, const void* next_weight,
               float scale, float eps, int T, int H, int dtype, int stream_dtype) {
  if (T < 1 || T > kMaxRows || H < 8 || H > kMaxNormDim || H % 8) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!dtype16(dtype) || (stream_dtype != dtype && stream_dtype != MOE_DTYPE_F32)) return MOE_ERR_INVALID_ARG;
  if (gate_kind < MOE_GATE_NONE || gate_kind > MOE_GATE_FULL) return MOE_ERR_INVALID_ARG;
  if ((gate_kind == MOE_GATE_NONE) != (gate == nullptr)) return MOE_ERR_INVALID_ARG;
  if (!block || !aligned(block, 16) || !aligned(norm_weight, 16) || !aligned(next_weight, 16)) return MOE_ERR_INVALID_ARG;
  if (!aligned(gate, gate_kind == MOE_GATE_TOKEN ? 4 : 16)) return MOE_ERR_INVALID_ARG;
  if (!(eps >= 0.f) || !(eps < 3.0e38f)) return MOE_ERR_INVALID_ARG;                 // negative, NaN or infinite
  if (!(scale > -3.0e38f) || !(scale < 3.0e38f)) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

BlockNormParams norm_params(const void* block, const void* norm_weight, const void* gate, int gate_kind,
                            const void* next_weight, float scale, float eps, int T, int H) {
  BlockNormParams p{};
  p.block = block;
  p.norm_w = norm_weight;
  p.gate = gate;
  p.gate_kind = gate_kind;
  p.next_w = next_weight;
  p.scale = scale;
  p.eps = eps;
  p.T = T;
  p.H = H;
  return p;
}

// Feed-forward workspace: h [T, I] (and, backward, dgu [T, 2 I]), then the partial sums
// of whichever product splits K.
struct FfnLayout {
  size_t h, dgu, partial, total;
};
FfnLayout ffn_layout(int T, int H, int I, bool backward) {
  FfnLayout L{};
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t r = o;
    o = align_up(o + bytes, 256);
    return r;
  };
  L.h = take((size_t)T * I * 2);
  size_t part = 0;
  auto need = [&](int M, int N, int K, int mode) {
    const size_t b = dense_partial_bytes(M, N, K, mode, backward);  // (the backward's B are all MN-major)
    if (b > part) part = b;
  };
  if (backward) {
    L.dgu = take((size_t)T * I * 4);
    need(T, I, H, kDenseGateUpGrad);
    need(T, H, 2 * I, kDenseStore);
    need(2 * I, H, T, kDenseStore);
    need(H, I, T, kDenseStore);
  } else if (T > kThinTokens) {
    need(T, I, H, kDenseGateUp);
    need(T, H, I, kDenseStore);
  }
  L.partial = take(part);
  L.total = o;
  return L;
}

int check_ffn(int T, int H, int I, int dtype, int act) {
  if (T < 1 || T > kMaxRows || H < 8 || I < 8 || H % 8 || I % 8 || H > kMaxFfnDim || I > kMaxFfnDim)
    return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!dtype16(dtype) || (act != MOE_ACT_SILU && act != MOE_ACT_GELU)) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

// A projection's workspace: dp [T, N] and the bias gradient's partial sums (backward), then
// the partial sums of whichever product splits K.  By sizes alone: a call without an activation, or
// without some of the gradients, leaves parts of it unused.
struct LinearLayout {
  size_t sums, partial, total;
};
// Which kernel a projection takes, by sizes (us on one GB300, 16 bits, with bias and residual):
//   thin    a block for 16 rows of W, while those are one round of blocks: 8 x 4096 -> 4096 8.0 against
//           9.6 of a batch, 16 x 4096 -> 4096 9.2 against 9.9; beyond, or with more of x to read again by
//           every block, a batch is faster: 8 x 2880 -> 5120 9.5 against 8.8, 16 x 14336 -> 4096 25.2
//           against 22.2; one to four tokens stay thin up to 16384 rows, 3.4 rounds of two blocks on each
//           of 152 SMs (1 x 4096 -> 14336 20.8 against 23.5, but 1 x 2880 -> 32768 34.8 against 31.3), however
//           long K is (131072 -> 24: 1 token 69.1, and 17 as a batch 69.6);
//   batch   up to 32 tokens (24 x 4096 -> 2880 8.3, tiles 11.6), 64 where K is not short (64 x 4096 ->
//           2880 9.7 against 12.2, but 64 x 1024 -> 4096 7.3 against 6.4), 128 where K is cut in four at
//           least (128 x 4096 -> 4096 13.0 against 14.6, but 128 x 2880 -> 5120 15.0 against 12.2);
//   tiles   else.
// The gradient into x of a batch takes the same kernel (64 tokens: 22.8 us against the tiles' 26.8 at
// 4096 <- 14336, 8.7 against 10.2 at 2880 <- 2880).
enum class LinearPath { thin, batch, tiles };
bool linear_batch(int T, int K, int N) {
  return T <= 32 || (T <= 64 && K > 1024) || (T <= kBatchTokens && K > 1024 && 4 * ceil_div(N, 128) <= device_sms());
}
LinearPath linear_path(int T, int K, int N) {
  const int sms = device_sms(), rows16 = ceil_div(N, kThinRows);
  if (T <= 4 ? N <= 16384 : T <= kThinTokens && rows16 <= 2 * sms && T * K <= 98304) return LinearPath::thin;
  return linear_batch(T, K, N) ? LinearPath::batch : LinearPath::tiles;
}
LinearLayout linear_layout(int T, int K, int N, bool backward) {
  LinearLayout L{};
  size_t part = 0;
  auto need = [&](int m, int n, int k) {
    const size_t b = dense_partial_bytes(m, n, k, backward ? kDenseStore : kDenseLinear, backward);
    if (b > part) part = b;
  };
  if (backward) {
    L.sums = align_up((size_t)T * N * 2, 256);
    L.partial = align_up(L.sums + (size_t)linear_grad_splits(T, N) * N * sizeof(float), 256);
    if (!linear_batch(T, N, K)) need(T, K, N);
    need(N, K, T);
  } else if (linear_path(T, K, N) == LinearPath::tiles) {
    need(T, N, K);
  }
  L.total = L.partial + align_up(part, 256);
  return L;
}
int check_linear(int T, int K, int N, int dtype, int out_dtype, int act) {
  if (T < 1 || T > kMaxRows || K < 8 || N < 8 || K % 8 || N % 8 || K > kMaxFfnDim || N > kMaxLinearOut)
    return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!dtype16(dtype) || (out_dtype != dtype && out_dtype != MOE_DTYPE_F32)) return MOE_ERR_INVALID_ARG;
  if (act != MOE_ACT_SILU && act != MOE_ACT_GELU && act != MOE_ACT_NONE) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}
// An array, and whether it overlaps another.
struct Span {
  const void* p;
  size_t bytes;
};
template <int N, int M>
bool any_overlap(const Span (&a)[N], const Span (&b)[M]) {
  for (const Span& x : a)
    for (const Span& y : b)
      if (x.p && y.p && overlap(x.p, x.bytes, y.p, y.bytes)) return true;
  return false;
}
// Whether any two of them overlap.
template <int N>
bool overlap_within(const Span (&a)[N]) {
  for (int i = 0; i < N; ++i)
    for (int j = 0; j < i; ++j)
      if (a[i].p && a[j].p && overlap(a[i].p, a[i].bytes, a[j].p, a[j].bytes)) return true;
  return false;
}

// Tokens and experts of a routing, as the layer's.
bool routing_shape(int T, int k, int E) {
  return T >= 1 && k >= 1 && k <= kMaxTopK && k <= E && E <= kMaxExperts && (long long)T * k <= kMaxRows;
}
// Rows of `H` values that the moves between token and expert order take.
bool moved_shape(int T, int k, int H, int dtype) {
  return routing_shape(T, k, kMaxExperts) && H >= 8 && H % 8 == 0 && H <= (dtype == MOE_DTYPE_F32 ? kMaxMovedBytes / 4 : kMaxMovedBytes / 2);
}
bool dtype_any(int d) { return dtype16(d) || d == MOE_DTYPE_F32; }

}  // namespace

extern "C" {

size_t moe_ffn_workspace_bytes(int T, int H, int I, int backward) {
  if (check_ffn(T, H, I, MOE_DTYPE_BF16, MOE_ACT_SILU) != MOE_OK) return 0;
  return ffn_layout(T, H, I, backward != 0).total;
}

int moe_ffn_forward(const void* x, const void* w_gateup, const void* w_down, int T, int H, int I, int act, int dtype,
                    float* gateup_out, void* out, void* workspace, size_t workspace_bytes, moe_stream_t stream) {
  int st = check_ffn(T, H, I, dtype, act);
  if (st != MOE_OK) return st;
  const void* need[] = {x, w_gateup, w_down, out};
  for (const void* q : need)
    if (!q || !aligned(q, 16)) return MOE_ERR_INVALID_ARG;
  if (!aligned(gateup_out, 16) || !workspace || !aligned(workspace, 256)) return MOE_ERR_INVALID_ARG;
  const FfnLayout L = ffn_layout(T, H, I, false);
  if (workspace_bytes < L.total) return MOE_ERR_WORKSPACE_TOO_SMALL;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  void* h = ws_ptr<uint8_t>(workspace, L.h);
  if (T <= kThinTokens) {
    ThinParams g{};
    g.x = x;
    g.w = w_gateup;
    g.T = T;
    g.K = H;
    g.n_out = I;
    g.tiles = ceil_div(I, kThinRows / 2);
    g.ku = ceil_div(H, 32);
    g.act = act;
    g.out = h;
    g.gateup = gateup_out;
    if (launch_thin16(g, dtype, true, s) != cudaSuccess) return MOE_ERR_CUDA;
    ThinParams d{};
    d.x = h;
    d.w = w_down;
    d.T = T;
    d.K = I;
    d.n_out = H;
    d.tiles = ceil_div(H, kThinRows);
    d.ku = ceil_div(I, 32);
    d.early = 1;
    d.out = out;
    return cuda_status(launch_thin16(d, dtype, false, s));
  }
  DenseGemmParams g{};
  g.g[0].M = T; g.g[0].N = I; g.g[0].K = H;
  g.g[0].out = h;
  g.act = act;
  g.gateup = gateup_out;
  g.partial = ws_ptr<float>(workspace, L.partial);
  st = launch_dense_gemm(g, {x, T, H, 0}, {w_gateup, 2 * I, H, 0}, kDenseGateUp, dtype, s);
  if (st != MOE_OK) return st;
  DenseGemmParams d{};
  d.g[0].M = T; d.g[0].N = H; d.g[0].K = I;
  d.g[0].out = out;
  d.partial = ws_ptr<float>(workspace, L.partial);
  return launch_dense_gemm(d, {h, T, I, 0}, {w_down, H, I, 0}, kDenseStore, dtype, s);
}

int moe_ffn_backward(const void* d_out, const void* x, const float* gateup, const void* w_gateup, const void* w_down,
                     int T, int H, int I, int act, int dtype, void* d_x, void* d_w_gateup, void* d_w_down,
                     void* workspace, size_t workspace_bytes, moe_stream_t stream) {
  int st = check_ffn(T, H, I, dtype, act);
  if (st != MOE_OK) return st;
  const void* need[] = {d_out, x, gateup, w_gateup, w_down};
  for (const void* q : need)
    if (!q || !aligned(q, 16)) return MOE_ERR_INVALID_ARG;
  if (!aligned(d_x, 16) || !aligned(d_w_gateup, 16) || !aligned(d_w_down, 16)) return MOE_ERR_INVALID_ARG;
  if (!d_x && !d_w_gateup && !d_w_down) return MOE_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 256)) return MOE_ERR_INVALID_ARG;
  const FfnLayout L = ffn_layout(T, H, I, true);
  if (workspace_bytes < L.total) return MOE_ERR_WORKSPACE_TOO_SMALL;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  void* h = ws_ptr<uint8_t>(workspace, L.h);
  void* dgu = ws_ptr<uint8_t>(workspace, L.dgu);
  float* partial = ws_ptr<float>(workspace, L.partial);
  DenseGemmParams p{};  // dh = d_out W_down, and from it dg, du, h
  p.g[0].M = T; p.g[0].N = I; p.g[0].K = H;
  p.g[0].out = dgu;
  p.act = act;
  p.out_h = h;
  p.gateup = const_cast<float*>(gateup);
  p.partial = partial;
  st = launch_dense_gemm(p, {d_out, T, H, 0}, {w_down, H, I, 1}, kDenseGateUpGrad, dtype, s);
  if (st != MOE_OK) return st;
  DenseGemmParams q{};  // what of it is asked for: dx = dgu W_gateup, dW_gateup = dgu^T x, dW_down = dout^T h
  q.partial = partial;
  DenseOperand a[kDenseGroup], b[kDenseGroup];
  int n = 0;
  auto product = [&](int M, int N, int K, const DenseOperand& am, const DenseOperand& bm, void* out) {
    if (!out) return;
    q.g[n].M = M; q.g[n].N = N; q.g[n].K = K;
    q.g[n].out = out;
    a[n] = am;
    b[n++] = bm;
  };
  product(T, H, 2 * I, {dgu, T, 2 * I, 0}, {w_gateup, 2 * I, H, 1}, d_x);
  product(2 * I, H, T, {dgu, T, 2 * I, 1}, {x, T, H, 1}, d_w_gateup);
  product(H, I, T, {d_out, T, H, 1}, {h, T, I, 1}, d_w_down);
  return launch_dense_products(q, n, a, b, dtype, false, s);
}

size_t moe_linear_workspace_bytes(int T, int K, int N, int backward) {
  if (check_linear(T, K, N, MOE_DTYPE_BF16, MOE_DTYPE_BF16, MOE_ACT_NONE) != MOE_OK) return 0;
  return linear_layout(T, K, N, backward != 0).total;
}

int moe_linear_forward(const void* x, const void* weight, const float* bias, const void* residual, int T, int K, int N, int act,
                       int dtype, int out_dtype, float* pre_out, void* out, void* workspace, size_t workspace_bytes,
                       moe_stream_t stream) {
  const int st = check_linear(T, K, N, dtype, out_dtype, act);
  if (st != MOE_OK) return st;
  if (!x || !weight || !out) return MOE_ERR_INVALID_ARG;
  const void* all[] = {x, weight, bias, residual, pre_out, out};
  for (const void* q : all)
    if (!aligned(q, 16)) return MOE_ERR_INVALID_ARG;
  if (pre_out && act == MOE_ACT_NONE) return MOE_ERR_INVALID_ARG;
  const size_t size = out_dtype == MOE_DTYPE_F32 ? 4 : 2, cells = (size_t)T * N;
  // (tiles are written while others still read; the residual is read by the thread that writes its element)
  const Span in[] = {{x, (size_t)T * K * 2}, {weight, (size_t)N * K * 2}, {bias, (size_t)N * 4},
                     {residual == out ? nullptr : residual, cells * size}, {pre_out, cells * 4}};
  const Span written[] = {{out, cells * size}};
  if (any_overlap(written, in)) return MOE_ERR_INVALID_ARG;
  const Span read[] = {in[0], in[1], in[2], {residual, cells * size}}, kept[] = {{pre_out, cells * 4}};
  if (any_overlap(kept, read)) return MOE_ERR_INVALID_ARG;
  const LinearLayout L = linear_layout(T, K, N, false);
  if (L.total && (!workspace || !aligned(workspace, 256))) return MOE_ERR_INVALID_ARG;
  if (workspace_bytes < L.total) return MOE_ERR_WORKSPACE_TOO_SMALL;
  const Span ws[] = {{L.total ? workspace : nullptr, L.total}};
  if (any_overlap(ws, read) || any_overlap(ws, kept) || any_overlap(ws, written)) return MOE_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const LinearPath path = linear_path(T, K, N);
  if (path == LinearPath::thin) {
    ThinParams g{};
    g.x = x;
    g.w = weight;
    g.bias = bias;
    g.T = T;
    g.K = K;
    g.n_out = N;
    g.tiles = ceil_div(N, kThinRows);
    g.ku = ceil_div(K, 32);
    g.act = act;
    g.out = out;
    g.gateup = pre_out;
    g.residual = residual;
    g.out_f32 = out_dtype == MOE_DTYPE_F32;
    return cuda_status(launch_thin_linear(g, dtype, s));
  }
  DenseGemmParams g{};
  g.g[0].M = T; g.g[0].N = N; g.g[0].K = K;
  g.g[0].out = out;
  g.act = act;
  g.gateup = pre_out;
  g.bias = bias;
  g.residual = residual;
  g.partial = ws_ptr<float>(workspace, L.partial);
  if (path == LinearPath::batch) return launch_linear_batch(g, {x, T, K, 0}, {weight, N, K, 0}, dtype, out_dtype == MOE_DTYPE_F32, s);
  return launch_dense_gemm(g, {x, T, K, 0}, {weight, N, K, 0}, out_dtype == MOE_DTYPE_F32 ? kDenseLinear32 : kDenseLinear,
                           dtype, s);
}

int moe_linear_backward(const void* d_out, const void* x, const void* weight, const float* pre, int T, int K, int N, int act,
                        int dtype, int out_dtype, void* d_x, void* d_weight, float* d_bias, void* workspace,
                        size_t workspace_bytes, moe_stream_t stream) {
  const int st = check_linear(T, K, N, dtype, out_dtype, act);
  if (st != MOE_OK) return st;
  if (!d_out || (!d_x && !d_weight && !d_bias) || (d_x && !weight) || (d_weight && !x)) return MOE_ERR_INVALID_ARG;
  if ((act != MOE_ACT_NONE) != (pre != nullptr)) return MOE_ERR_INVALID_ARG;
  const void* all[] = {d_out, x, weight, pre, d_x, d_weight, d_bias};
  for (const void* q : all)
    if (!aligned(q, 16)) return MOE_ERR_INVALID_ARG;
  const size_t cells = (size_t)T * N;
  const Span in[] = {{d_out, cells * (out_dtype == MOE_DTYPE_F32 ? 4 : 2)}, {x, (size_t)T * K * 2}, {weight, (size_t)N * K * 2},
                     {pre, cells * 4}};
  const Span out[] = {{d_x, (size_t)T * K * 2}, {d_weight, (size_t)N * K * 2}, {d_bias, (size_t)N * 4}};
  if (any_overlap(out, in) || overlap_within(out)) return MOE_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 256)) return MOE_ERR_INVALID_ARG;
  const LinearLayout L = linear_layout(T, K, N, true);
  if (workspace_bytes < L.total) return MOE_ERR_WORKSPACE_TOO_SMALL;
  const Span ws[] = {{workspace, L.total}};
  if (any_overlap(ws, in) || any_overlap(ws, out)) return MOE_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool products = d_x || d_weight;
  const void* dp = d_out;  // without an activation, a 16-bit d_out is dp
  LinearGradParams g{};
  if (products && (pre || out_dtype == MOE_DTYPE_F32)) dp = g.dp = workspace;
  if (g.dp || d_bias) {
    g.d_out = d_out;
    g.pre = pre;
    g.d_bias = d_bias;
    g.partial = ws_ptr<float>(workspace, L.sums);
    g.T = T;
    g.N = N;
    g.act = act;
    g.splits = linear_grad_splits(T, N);
    if (launch_linear_grad(g, dtype, out_dtype, s) != cudaSuccess) return MOE_ERR_CUDA;
  }
  if (!products) return MOE_OK;
  const bool batch = d_x && linear_batch(T, N, K);
  if (batch) {
    DenseGemmParams b{};
    b.g[0].M = T; b.g[0].N = K; b.g[0].K = N;
    b.g[0].out = d_x;
    b.act = MOE_ACT_NONE;
    const int launched = launch_linear_batch(b, {dp, T, N, 0}, {weight, N, K, 1}, dtype, false, s);
    if (launched != MOE_OK || !d_weight) return launched;
  }
  // The weights' gradient from few tokens is written more than computed (us, tiles against this: 1 x
  // 4096 -> 14336 38.8 and 27.0, 16 tokens 37.3 and 35.3, 64 37.6 and 55.8; 64 x 1024 -> 4096 5.8 and 4.8).
  const bool outer = T <= 16 || (T <= kThinOuterTokens && (long long)N * K <= 1 << 23);
  if (outer && d_weight && (batch || !d_x)) {
    ThinOuterParams o{};
    o.a = dp;
    o.b = x;
    o.T = T;
    o.N = N;
    o.K = K;
    o.out = d_weight;
    return cuda_status(launch_thin_outer(o, dtype, s));
  }
  DenseGemmParams q{};
  q.partial = ws_ptr<float>(workspace, L.partial);
  DenseOperand a[kDenseGroup], b[kDenseGroup];
  int n = 0;
  auto product = [&](int m, int cols, int k, const DenseOperand& am, const DenseOperand& bm, void* to) {
    if (!to) return;
    q.g[n].M = m; q.g[n].N = cols; q.g[n].K = k;
    q.g[n].out = to;
    a[n] = am;
    b[n++] = bm;
  };
  product(T, K, N, {dp, T, N, 0}, {weight, N, K, 1}, batch ? nullptr : d_x);
  product(N, K, T, {dp, T, N, 1}, {x, T, K, 1}, d_weight);
  return launch_dense_products(q, n, a, b, dtype, true, s);
}

int moe_dense_status(int* status, moe_stream_t stream) {
  if (!status) return MOE_ERR_INVALID_ARG;
  uint32_t* words[] = {dense_status_word(), thin_status_word(), norm_status_word(), sort_status_word()};
  int all = 0;
  for (uint32_t* word : words) {
    if (!word) return MOE_ERR_CUDA;
    int bits = 0;
    const int st = read_and_clear_status(word, sizeof(uint32_t), reinterpret_cast<cudaStream_t>(stream), &bits);
    if (st == MOE_ERR_CUDA) return st;
    all |= bits;
  }
  *status = all;
  return all ? MOE_ERR_DEVICE_TIMEOUT : MOE_OK;
}

int moe_block_norm(const void* block, const void* norm_weight, const void* gate, int gate_kind, const void* residual,
                   float residual_scale, const void* next_weight, float eps, int T, int H, int dtype, int stream_dtype,
                   void* residual_out, void* out, moe_stream_t stream) {
  const int st = check_norm(block, norm_weight, gate, gate_kind, next_weight, residual_scale, eps, T, H, dtype,
                            stream_dtype);
  if (st != MOE_OK) return st;
  if (!aligned(residual, 16) || !aligned(residual_out, 16) || !aligned(out, 16)) return MOE_ERR_INVALID_ARG;
  if ((next_weight != nullptr) != (out != nullptr) || (!residual_out && !out)) return MOE_ERR_INVALID_ARG;
  if (residual_out == out) return MOE_ERR_INVALID_ARG;
  BlockNormParams p = norm_params(block, norm_weight, gate, gate_kind, next_weight, residual_scale, eps, T, H);
  p.residual = residual;
  p.residual_out = residual_out;
  p.out = out;
  return cuda_status(launch_block_norm(p, dtype, stream_dtype, kOut16, reinterpret_cast<cudaStream_t>(stream)));
}

int moe_block_norm_8bit(const void* block, const void* norm_weight, const void* gate, int gate_kind, const void* residual,
                        float residual_scale, const void* next_weight, float eps, int T, int H, int dtype, int stream_dtype,
                        int scale_kind, void* residual_out, uint8_t* codes, void* scales, void* out, moe_stream_t stream) {
  const int st = check_norm(block, norm_weight, gate, gate_kind, next_weight, residual_scale, eps, T, H, dtype,
                            stream_dtype);
  if (st != MOE_OK) return st;
  if (scale_kind != MOE_SCALE_MX && scale_kind != MOE_SCALE_ROW) return MOE_ERR_INVALID_ARG;
  if (scale_kind == MOE_SCALE_MX && H % kMxBlock) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!next_weight || !codes || !scales) return MOE_ERR_INVALID_ARG;
  const void* all[] = {residual, residual_out, codes, scales, out};
  for (const void* q : all)
    if (!aligned(q, 16)) return MOE_ERR_INVALID_ARG;
  // (rows are written while others are still read; s and y go where their own element was read)
  const size_t cells = (size_t)T * H, size = stream_dtype == MOE_DTYPE_F32 ? 4 : 2;
  const size_t scale_bytes = scale_kind == MOE_SCALE_MX ? cells / kMxBlock : (size_t)T * 4;
  const size_t gate_bytes = gate_kind == MOE_GATE_FEATURE ? (size_t)H * 2 : gate_kind == MOE_GATE_TOKEN ? (size_t)T * 4 : cells * 2;
  const Span in[] = {{block, cells * 2}, {norm_weight, (size_t)H * 2}, {gate, gate_bytes}, {residual, cells * size},
                     {next_weight, (size_t)H * 2}};
  const Span eight[] = {{codes, cells}, {scales, scale_bytes}}, s_out[] = {{residual_out, cells * size}}, y_out[] = {{out, cells * 2}};
  const Span not_s[] = {in[0], in[1], in[2], {residual == residual_out ? nullptr : residual, cells * size}, in[4]};
  const Span not_y[] = {{block == out ? nullptr : block, cells * 2}, in[1], in[2], in[3], in[4]};
  if (any_overlap(eight, in) || any_overlap(s_out, not_s) || any_overlap(y_out, not_y) || any_overlap(eight, s_out) ||
      any_overlap(eight, y_out) || any_overlap(s_out, y_out) || overlap(codes, cells, scales, scale_bytes))
    return MOE_ERR_INVALID_ARG;
  BlockNormParams p = norm_params(block, norm_weight, gate, gate_kind, next_weight, residual_scale, eps, T, H);
  p.residual = residual;
  p.residual_out = residual_out;
  p.out = out;
  p.codes = codes;
  p.scales = scales;
  return cuda_status(launch_block_norm(p, dtype, stream_dtype, scale_kind == MOE_SCALE_MX ? kOutMx : kOutRow,
                                       reinterpret_cast<cudaStream_t>(stream)));
}

size_t moe_block_norm_workspace_bytes(int T, int H) {
  if (T < 1 || T > kMaxRows || H < 8 || H > kMaxNormDim || H % 8) return 0;
  return (size_t)block_norm_backward_blocks(T, H) * 3 * H * sizeof(float);
}

int moe_block_norm_backward(const void* d_residual_out, const void* d_out, const void* block, const void* norm_weight,
                            const void* gate, int gate_kind, const void* residual_out, float residual_scale,
                            const void* next_weight, float eps, int T, int H, int dtype, int stream_dtype,
                            void* d_block, void* d_residual, float* d_norm_weight, void* d_gate, float* d_next_weight,
                            void* workspace, size_t workspace_bytes, moe_stream_t stream) {
  const int st = check_norm(block, norm_weight, gate, gate_kind, next_weight, residual_scale, eps, T, H, dtype,
                            stream_dtype);
  if (st != MOE_OK) return st;
  if ((next_weight != nullptr) != (d_out != nullptr) || (next_weight && !residual_out)) return MOE_ERR_INVALID_ARG;
  if (!d_residual_out && !d_out) return MOE_ERR_INVALID_ARG;
  if (!d_block || !workspace) return MOE_ERR_INVALID_ARG;
  if ((d_norm_weight && !norm_weight) || (d_next_weight && !next_weight) || (d_gate && gate_kind == MOE_GATE_NONE))
    return MOE_ERR_INVALID_ARG;
  const void* all[] = {d_residual_out, d_out, residual_out, d_block, d_residual, d_norm_weight, d_next_weight};
  for (const void* q : all)
    if (!aligned(q, 16)) return MOE_ERR_INVALID_ARG;
  if (!aligned(d_gate, gate_kind == MOE_GATE_TOKEN ? 4 : 16) || !aligned(workspace, 256)) return MOE_ERR_INVALID_ARG;
  if (workspace_bytes < moe_block_norm_workspace_bytes(T, H)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  BlockNormBackwardParams q{};
  q.f = norm_params(block, norm_weight, gate, gate_kind, next_weight, residual_scale, eps, T, H);
  q.f.residual_out = const_cast<void*>(residual_out);
  q.d_residual_out = d_residual_out;
  q.d_out = d_out;
  q.d_block = d_block;
  q.d_residual = d_residual;
  q.d_gate = d_gate;
  q.d_norm_w = d_norm_weight;
  q.d_next_w = d_next_weight;
  q.partial = static_cast<float*>(workspace);
  q.blocks = block_norm_backward_blocks(T, H);
  return cuda_status(launch_block_norm_backward(q, dtype, stream_dtype, reinterpret_cast<cudaStream_t>(stream)));
}

int moe_sort_tokens(const void* x, const void* scales, const int32_t* topk_idx, int T, int k, int E, int row_bytes,
                    int scale_bytes, int32_t* offsets, int32_t* perm, int32_t* inv_perm, void* rows, void* row_scales,
                    moe_stream_t stream) {
  if (!routing_shape(T, k, E) || row_bytes < 16 || row_bytes % 16 || row_bytes > kMaxMovedBytes) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (scale_bytes < 0 || scale_bytes > kMaxScaleBytes) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!x || !topk_idx || !offsets || !perm || !inv_perm || !rows) return MOE_ERR_INVALID_ARG;
  if ((scales != nullptr) != (scale_bytes > 0) || (row_scales != nullptr) != (scale_bytes > 0)) return MOE_ERR_INVALID_ARG;
  const void *moved[] = {x, rows}, *words[] = {topk_idx, offsets, perm, inv_perm};
  for (const void* q : moved)
    if (!aligned(q, 16)) return MOE_ERR_INVALID_ARG;
  for (const void* q : words)
    if (!aligned(q, 4)) return MOE_ERR_INVALID_ARG;
  // (rows are written while others are still read)
  const size_t n = (size_t)T * k;
  const Span in[] = {{x, (size_t)T * row_bytes}, {scales, (size_t)T * scale_bytes}, {topk_idx, n * 4}};
  const Span out[] = {{offsets, (size_t)(E + 1) * 4}, {perm, n * 4}, {inv_perm, n * 4}, {rows, n * row_bytes},
                      {row_scales, n * scale_bytes}};
  if (any_overlap(out, in) || overlap_within(out)) return MOE_ERR_INVALID_ARG;
  SortParams p{};
  p.idx = topk_idx;
  p.x = x;
  p.scales = scales;
  p.T = T;
  p.k = k;
  p.E = E;
  p.row_bytes = row_bytes;
  p.scale_bytes = scale_bytes;
  p.offsets = offsets;
  p.perm = perm;
  p.inv_perm = inv_perm;
  p.rows = rows;
  p.row_scales = row_scales;
  p.wait_ns = gemm_wait_limit_ns();
  return cuda_status(launch_sort(p, reinterpret_cast<cudaStream_t>(stream)));
}

int moe_unsort_tokens(const void* y, const int32_t* inv_perm, const float* topk_w, int T, int k, int H, int dtype, void* out,
                      moe_stream_t stream) {
  if (!dtype_any(dtype)) return MOE_ERR_INVALID_ARG;
  if (!moved_shape(T, k, H, dtype)) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!y || !inv_perm || !out || !aligned(y, 16) || !aligned(inv_perm, 4) || !aligned(topk_w, 4) || !aligned(out, 16))
    return MOE_ERR_INVALID_ARG;
  const size_t bytes = (size_t)T * H * (dtype == MOE_DTYPE_F32 ? 4 : 2), n = (size_t)T * k * 4;
  const Span in[] = {{y, bytes * k}, {inv_perm, n}, {topk_w, n}}, written[] = {{out, bytes}};
  if (any_overlap(written, in)) return MOE_ERR_INVALID_ARG;
  UnsortParams p{};
  p.y = y;
  p.inv_perm = inv_perm;
  p.w = topk_w;
  p.T = T;
  p.k = k;
  p.H = H;
  p.out = out;
  p.wait_ns = gemm_wait_limit_ns();
  return cuda_status(launch_unsort(p, dtype, reinterpret_cast<cudaStream_t>(stream)));
}

int moe_unsort_tokens_backward(const void* d_out, const void* y, const int32_t* inv_perm, const float* topk_w, int T, int k,
                               int H, int dtype, void* d_y, float* d_topk_w, moe_stream_t stream) {
  if (!dtype_any(dtype)) return MOE_ERR_INVALID_ARG;
  if (!moved_shape(T, k, H, dtype)) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!d_out || !inv_perm || (!d_y && !d_topk_w) || (d_topk_w && !y)) return MOE_ERR_INVALID_ARG;
  const void *moved[] = {d_out, y, d_y}, *words[] = {inv_perm, topk_w, d_topk_w};
  for (const void* q : moved)
    if (!aligned(q, 16)) return MOE_ERR_INVALID_ARG;
  for (const void* q : words)
    if (!aligned(q, 4)) return MOE_ERR_INVALID_ARG;
  const size_t bytes = (size_t)T * H * (dtype == MOE_DTYPE_F32 ? 4 : 2), n = (size_t)T * k * 4;
  const Span in[] = {{d_out, bytes}, {y, bytes * k}, {inv_perm, n}, {topk_w, n}}, out[] = {{d_y, bytes * k}, {d_topk_w, n}};
  if (any_overlap(out, in) || overlap_within(out)) return MOE_ERR_INVALID_ARG;
  UnsortBackwardParams q{};
  q.f.y = y;
  q.f.inv_perm = inv_perm;
  q.f.w = topk_w;
  q.f.T = T;
  q.f.k = k;
  q.f.H = H;
  q.f.wait_ns = gemm_wait_limit_ns();
  q.d_out = d_out;
  q.d_y = d_y;
  q.d_w = d_topk_w;
  return cuda_status(launch_unsort_backward(q, dtype, reinterpret_cast<cudaStream_t>(stream)));
}

int moe_route_backward(const float* d_topk_w, const float* logits, const int32_t* topk_idx, const float* topk_w, int T, int k,
                       int E, int gating, float* d_logits, moe_stream_t stream) {
  if (!routing_shape(T, k, E)) return MOE_ERR_UNSUPPORTED_SHAPE;
  const int kind = gating & MOE_ROUTE_FROM_LOGITS ? -1 : gating_from_flags(gating);
  if (kind < 0) return MOE_ERR_INVALID_ARG;
  const void* need[] = {d_topk_w, logits, topk_idx, topk_w, d_logits};
  for (const void* q : need)
    if (!q || !aligned(q, 4)) return MOE_ERR_INVALID_ARG;
  const size_t all = (size_t)T * E * 4, n = (size_t)T * k * 4;
  const Span in[] = {{d_topk_w, n}, {logits, all}, {topk_idx, n}, {topk_w, n}}, out[] = {{d_logits, all}};
  if (any_overlap(out, in)) return MOE_ERR_INVALID_ARG;
  RouteBackwardParams p{};
  p.d_w = d_topk_w;
  p.logits = logits;
  p.w = topk_w;
  p.idx = topk_idx;
  p.T = T;
  p.k = k;
  p.E = E;
  p.gating = kind;
  p.d_logits = d_logits;
  return cuda_status(launch_route_backward(p, reinterpret_cast<cudaStream_t>(stream)));
}

size_t moe_prepared_matvec_bytes(int rows, int K, int kind) {
  if (rows < 1 || rows > kMaxMatvecRows || K < 32 || K > kMaxMatvecDim || K % 32) return 0;
  if (kind != MOE_WEIGHTS_GATEUP && kind != MOE_WEIGHTS_DOWN) return 0;
  if (kind == MOE_WEIGHTS_GATEUP && rows % 2) return 0;
  return make_matvec_layout(rows, K, kind == MOE_WEIGHTS_GATEUP).total;
}

int moe_prepare_matvec(const uint8_t* codes, const uint8_t* scales, int rows, int K, int kind, void* dst,
                       size_t dst_bytes, moe_stream_t stream) {
  const size_t need = moe_prepared_matvec_bytes(rows, K, kind);
  if (need == 0) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!codes || !scales || !dst || !aligned(codes, 16) || !aligned(dst, 256)) return MOE_ERR_INVALID_ARG;
  if (dst_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
  MatvecPrepareParams p{};
  p.codes = codes;
  p.scales = scales;
  p.L = make_matvec_layout(rows, K, kind == MOE_WEIGHTS_GATEUP);
  p.dst = static_cast<uint8_t*>(dst);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  uint8_t* flag = p.dst + p.L.flag_off;
  if (cudaMemsetAsync(flag, 0, 256, s) != cudaSuccess) return MOE_ERR_CUDA;
  if (launch_matvec_prepare(p, s) != cudaSuccess) return MOE_ERR_CUDA;
  uint32_t h = 0;
  if (cudaMemcpyAsync(&h, flag, sizeof h, cudaMemcpyDeviceToHost, s) != cudaSuccess) return MOE_ERR_CUDA;
  if (cudaStreamSynchronize(s) != cudaSuccess) return MOE_ERR_CUDA;
  return h ? MOE_ERR_NAN_SCALE : MOE_OK;
}

size_t moe_matvec_workspace_bytes(int T, int K) {
  if (T < 1 || T > kMatvecMaxTokens || K < 32 || K > kMaxMatvecDim || K % 32) return 0;
  return matvec_workspace_bytes(T, K);
}

int moe_matvec_mxfp4(const void* x, const void* w, const float* bias, int T, int rows, int K, int kind, int act,
                     int dtype, void* out, void* workspace, size_t workspace_bytes, moe_stream_t stream) {
  if (T < 1 || T > kMatvecMaxTokens || moe_prepared_matvec_bytes(rows, K, kind) == 0) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!dtype16(dtype) || (act != MOE_ACT_SILU && act != MOE_ACT_GELU)) return MOE_ERR_INVALID_ARG;
  if (!x || !w || !out || !aligned(x, 16) || !aligned(w, 256) || !aligned(out, 16) || !aligned(bias, 4))
    return MOE_ERR_INVALID_ARG;
  const size_t need = matvec_workspace_bytes(T, K);
  if (need && (!workspace || !aligned(workspace, 256))) return MOE_ERR_INVALID_ARG;
  if (need > workspace_bytes) return MOE_ERR_WORKSPACE_TOO_SMALL;
  const bool gated = kind == MOE_WEIGHTS_GATEUP;
  const int n_out = gated ? rows / 2 : rows;
  // (the first blocks write their outputs while others still read x)
  if (overlap(x, (size_t)T * K * 2, out, (size_t)T * n_out * 2)) return MOE_ERR_INVALID_ARG;
  const MatvecLayout L = make_matvec_layout(rows, K, gated);
  ThinParams p{};
  p.x = x;
  p.w = w;
  p.row_exp = static_cast<const uint8_t*>(w) + L.exp_off;
  p.packed = static_cast<uint8_t*>(workspace);
  p.bias = bias;
  p.T = T;
  p.K = K;
  p.n_out = n_out;
  p.tiles = L.tiles;
  p.ku = L.ku;
  p.act = act;
  p.out = out;
  return cuda_status(launch_matvec(p, dtype, gated, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
