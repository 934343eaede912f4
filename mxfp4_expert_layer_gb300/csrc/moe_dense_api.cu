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
static_assert(MOE_ACT_SILU == kActSilu && MOE_ACT_GELU == kActGelu, "activations");

constexpr int kMaxRows = 1 << 24;      // tokens of a call
constexpr int kMaxNormDim = 8192;      // a row sits in one block's registers
constexpr int kMaxFfnDim = 1 << 17;    // H and I of the feed-forward block
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
  return launch_dense_products(q, n, a, b, dtype, s);
}

int moe_dense_status(int* status, moe_stream_t stream) {
  if (!status) return MOE_ERR_INVALID_ARG;
  uint32_t* words[] = {dense_status_word(), thin_status_word(), norm_status_word()};
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
  return cuda_status(launch_block_norm(p, dtype, stream_dtype, reinterpret_cast<cudaStream_t>(stream)));
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
