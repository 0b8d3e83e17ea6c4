// C ABI of the 8-bit operators (w8a8_*, include/w4a4.h; the rest of a feed-forward
// block, include/ffn8.h; kv8_*, include/kv8.h):
// argument validation, then the launches of one call.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "act8.h"
#include "ffn8.h"
#include "kv8.h"
#include "launch.h"
#include "w4a4.h"

using w4a4::KvBatch;
using w4a4::KvNew;
using w4a4::KvPool;
using w4a4::KvQuery;

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

hipStream_t as_stream(void* s) { return static_cast<hipStream_t>(s); }

w4a4_status_t launched() {
  return hipGetLastError() == hipSuccess ? W4A4_OK : W4A4_E_HIP;
}

constexpr int64_t kMaxI32 = (int64_t{1} << 31) - 1;

bool y_dtype_ok(int32_t t) { return t == W4A4_Y_F32 || t == W4A4_Y_F16 || t == W4A4_Y_BF16; }
bool x_dtype_ok(int32_t t) { return t == W4A4_Y_F16 || t == W4A4_Y_BF16; }

// Longest K of the W8A8 GEMM: 128^2 K < 2^31, a multiple of 16.
constexpr int64_t kMaxW8K = 131056;

// Most rows: one workgroup of 256 threads per row stays within a launch's 2^32.
constexpr int64_t kMaxW8Rows = int64_t{1} << 24;

bool w8_extents_ok(int64_t M, int64_t N, int64_t K) {
  return M >= 0 && N >= 0 && M < kMaxW8Rows && N < kMaxW8Rows && K > 0 && K % 16 == 0 && K <= kMaxW8K;
}

// Tokens of a batch, positions of a sequence: 16-position pages times 256
// threads stay within a launch's 2^32 threads.
constexpr int64_t kMaxTokens = int64_t{1} << 28;

// The pool's and the batch's extents.
bool kv_extents_ok(int64_t num_pages, int32_t heads, int32_t page, int32_t dim, int64_t table_ld, int64_t B, int64_t T,
                   int64_t max_new, int64_t max_len) {
  if (num_pages < 0 || num_pages > kMaxI32 || heads <= 0 || heads > 16384) return false;
  if (page < 16 || page > 256 || (page & (page - 1))) return false;
  if (dim < 64 || dim > 256 || dim % 64) return false;
  if (B < 0 || B > 65535 || T < 0 || T >= kMaxTokens) return false;
  if (max_new < 0 || max_new > kMaxI32 || max_len < 0 || max_len >= kMaxTokens) return false;
  return table_ld >= 0 && table_ld <= kMaxI32 && max_len <= table_ld * page;
}

KvPool pool(const int8_t* k, const int8_t* v, const float* ks, const float* vs, int64_t num_pages, int32_t heads,
            int32_t page, int32_t dim) {
  KvPool c;
  c.k = const_cast<int8_t*>(k);
  c.v = const_cast<int8_t*>(v);
  c.ks = const_cast<float*>(ks);
  c.vs = const_cast<float*>(vs);
  c.num_pages = (int)num_pages;
  c.heads = heads;
  c.page = page;
  c.dim = dim;
  c.log_page = __builtin_ctz((unsigned)page);
  return c;
}

KvBatch batch(const int32_t* table, int64_t table_ld, const int32_t* cu, const int32_t* lens, int64_t B, int64_t T,
              int64_t max_new, int64_t max_len) {
  KvBatch b;
  b.table = table;
  b.table_ld = table_ld;
  b.cu = cu;
  b.lens = lens;
  b.B = (int)B;
  b.T = (int)T;
  b.max_new = (int)(max_new < T ? max_new : T);
  b.max_len = (int)max_len;
  return b;
}

// Pointers every kv8 call needs; the pool and the table may be absent where no
// position can be cached (max_len == 0).
w4a4_status_t kv_pointers(const KvPool& c, const KvBatch& b) {
  if (!b.cu || !b.lens) return W4A4_E_NULL;
  if (!aligned(b.cu, 4) || !aligned(b.lens, 4)) return W4A4_E_ALIGN;
  if (b.max_len == 0) return W4A4_OK;
  if (!b.table || (c.num_pages > 0 && (!c.k || !c.v || !c.ks || !c.vs))) return W4A4_E_NULL;
  if (!aligned(b.table, 4) || !aligned(c.k, 16) || !aligned(c.v, 16) || !aligned(c.ks, 4) || !aligned(c.vs, 4))
    return W4A4_E_ALIGN;
  return W4A4_OK;
}

// Rows of a buffer: `rows` of `width` bytes, `pitch` bytes apart.
struct Rows {
  const void* at;
  int64_t rows, pitch, width;
  uintptr_t first() const { return reinterpret_cast<uintptr_t>(at); }
  uintptr_t end() const { return first() + (uintptr_t)(rows - 1) * (uintptr_t)pitch + (uintptr_t)width; }
};
Rows flat(const void* at, int64_t bytes) { return Rows{at, 1, bytes, bytes}; }

// Whether two buffers share memory (absent ones do not; neither do columns apart in rows of
// one pitch, nor a run between two rows).
bool meet(const Rows& a, const Rows& b) {
  if (!a.at || !b.at || a.rows == 0 || b.rows == 0 || a.width == 0 || b.width == 0) return false;
  if (a.first() >= b.end() || b.first() >= a.end()) return false;
  if ((a.rows == 1 && b.rows == 1) || (a.rows > 1 && b.rows > 1 && a.pitch != b.pitch)) return true;
  const int64_t pitch = a.rows > 1 ? a.pitch : b.pitch;
  const int64_t d = (int64_t)(b.first() - a.first()) % pitch, apart = d < 0 ? d + pitch : d;
  return apart < a.width || apart + b.width > pitch;
}
// An output that may also be the input itself.
bool meet_elsewhere(const Rows& out, const Rows& in) {
  return meet(out, in) && !(out.at == in.at && (out.rows == 1 || out.pitch == in.pitch));
}
template <class... R>
bool meets_any(const Rows& a, const R&... others) {
  return (meet(a, others) || ...);
}

}  // namespace

extern "C" {

w4a4_status_t w8a8_quantize_act(const void* x, int32_t x_dtype, int64_t M, int64_t K, int64_t ldx,
                                int8_t* xq, float* xs, void* stream) {
  if (!x_dtype_ok(x_dtype)) return W4A4_E_DTYPE;
  if (M < 0 || M >= kMaxW8Rows || K <= 0 || K % 16 || K > (int64_t{1} << 30) || ldx < K) return W4A4_E_SHAPE;
  if (ldx % 8) return W4A4_E_ALIGN;
  if (M == 0) return W4A4_OK;
  if (!x || !xq || !xs) return W4A4_E_NULL;
  if (!aligned(x, 16) || !aligned(xq, 16) || !aligned(xs, 4)) return W4A4_E_ALIGN;
  w4a4::launch_w8a8_quant(x, x_dtype == W4A4_Y_BF16, M, K, ldx, xq, xs, as_stream(stream));
  return launched();
}

w4a4_status_t w8a8_pack_weight(const void* w, int32_t w_dtype, int64_t N, int64_t K,
                               int8_t* wq, float* ws, void* stream) {
  return w8a8_quantize_act(w, w_dtype, N, K, K, wq, ws, stream);
}

int64_t w8a8_gemm_workspace(int64_t M, int64_t N, int64_t K) {
  if (!w8_extents_ok(M, N, K)) return -1;
  if (M == 0 || N == 0) return 0;
  return w4a4::w8a8_workspace(M, N, K);
}

w4a4_status_t w8a8_gemm(const int8_t* xq, const float* xs, const int8_t* wq, const float* ws, const float* bias,
                        int64_t M, int64_t N, int64_t K, void* workspace, int64_t workspace_bytes,
                        void* y, int32_t y_dtype, int64_t ldy, void* stream) {
  if (!w8_extents_ok(M, N, K)) return W4A4_E_SHAPE;
  if (!y_dtype_ok(y_dtype)) return W4A4_E_DTYPE;
  if (M == 0 || N == 0) return W4A4_OK;
  if (ldy < N) return W4A4_E_SHAPE;
  if (!xq || !xs || !wq || !ws || !y) return W4A4_E_NULL;
  if (!aligned(xq, 16) || !aligned(wq, 16) || !aligned(xs, 4) || !aligned(ws, 4) || !aligned(bias, 4) ||
      !aligned(y, y_dtype == W4A4_Y_F32 ? 4 : 2))
    return W4A4_E_ALIGN;
  const int64_t need = w8a8_gemm_workspace(M, N, K);
  if (workspace_bytes < need) return W4A4_E_SHAPE;
  if (need > 0 && !workspace) return W4A4_E_NULL;
  if (need > 0 && !aligned(workspace, 16)) return W4A4_E_ALIGN;
  w4a4::W8GemmArgs g = {};
  g.a = xq; g.sa = xs; g.w = wq; g.sw = ws; g.bias = bias;
  g.M = M; g.N = N; g.K = K;
  g.y = y; g.ydtype = y_dtype; g.ldy = ldy; g.workspace = workspace;
  w4a4::launch_w8a8_gemm(g, as_stream(stream));
  return launched();
}

// Codes, then scales, then the GEMM's partial sums, each on a 256-byte boundary.
static int64_t align256(int64_t n) { return (n + 255) & ~int64_t{255}; }

int64_t w8a8_linear_workspace(int64_t M, int64_t N, int64_t K) {
  const int64_t gemm = w8a8_gemm_workspace(M, N, K);
  if (gemm < 0) return -1;
  if (M == 0 || N == 0 || w4a4::w8a8_one_launch(M, N, K)) return 0;
  return align256(M * K) + align256(4 * M) + gemm;
}

w4a4_status_t w8a8_linear(const void* x, int32_t x_dtype, int64_t M, int64_t K, int64_t ldx,
                          const int8_t* wq, const float* ws, const float* bias, int64_t N,
                          void* workspace, int64_t workspace_bytes,
                          void* y, int32_t y_dtype, int64_t ldy, void* stream) {
  if (!w8_extents_ok(M, N, K) || ldx < K) return W4A4_E_SHAPE;
  if (!x_dtype_ok(x_dtype) || !y_dtype_ok(y_dtype)) return W4A4_E_DTYPE;
  if (ldx % 8) return W4A4_E_ALIGN;
  if (M == 0 || N == 0) return W4A4_OK;
  const int64_t need = w8a8_linear_workspace(M, N, K);
  if (ldy < N || workspace_bytes < need) return W4A4_E_SHAPE;
  if (!x || !wq || !ws || !y || (need > 0 && !workspace)) return W4A4_E_NULL;
  if (!aligned(x, 16) || (need > 0 && !aligned(workspace, 16)) || !aligned(wq, 16) || !aligned(ws, 4) || !aligned(bias, 4) ||
      !aligned(y, y_dtype == W4A4_Y_F32 ? 4 : 2))
    return W4A4_E_ALIGN;
  w4a4::W8GemmArgs g = {};
  g.w = wq; g.sw = ws; g.bias = bias;
  g.M = M; g.N = N; g.K = K;
  g.y = y; g.ydtype = y_dtype; g.ldy = ldy;
  if (need == 0) {
    w4a4::launch_w8a8_small(g, x, x_dtype == W4A4_Y_BF16, ldx, as_stream(stream));
    return launched();
  }
  int8_t* xq = static_cast<int8_t*>(workspace);
  float* xs = reinterpret_cast<float*>(xq + align256(M * K));
  w4a4::launch_w8a8_quant(x, x_dtype == W4A4_Y_BF16, M, K, ldx, xq, xs, as_stream(stream));
  g.a = xq; g.sa = xs;
  g.workspace = xq + align256(M * K) + align256(4 * M);
  w4a4::launch_w8a8_gemm(g, as_stream(stream));
  return launched();
}

w4a4_status_t kv8_append(const void* k, const void* v, int32_t x_dtype, int64_t k_tok, int64_t k_head,
                         int64_t v_tok, int64_t v_head,
                         int8_t* k_cache, int8_t* v_cache, float* k_scale, float* v_scale,
                         int64_t num_pages, int32_t heads, int32_t page, int32_t dim,
                         const int32_t* block_table, int64_t table_ld, const int32_t* cu_seqlens,
                         const int32_t* seq_lens, int64_t B, int64_t T, int64_t max_new, int64_t max_len,
                         void* stream) {
  if (!x_dtype_ok(x_dtype)) return W4A4_E_DTYPE;
  if (!kv_extents_ok(num_pages, heads, page, dim, table_ld, B, T, max_new, max_len)) return W4A4_E_SHAPE;
  if (k_tok < 0 || k_head < 0 || v_tok < 0 || v_head < 0) return W4A4_E_SHAPE;
  if (k_tok % 8 || k_head % 8 || v_tok % 8 || v_head % 8) return W4A4_E_ALIGN;
  if (B == 0 || T == 0 || max_new == 0) return W4A4_OK;
  const KvPool c = pool(k_cache, v_cache, k_scale, v_scale, num_pages, heads, page, dim);
  const KvBatch b = batch(block_table, table_ld, cu_seqlens, seq_lens, B, T, max_new, max_len);
  const w4a4_status_t st = kv_pointers(c, b);
  if (st != W4A4_OK) return st;
  if (!k || !v) return W4A4_E_NULL;
  if (!aligned(k, 16) || !aligned(v, 16)) return W4A4_E_ALIGN;
  if (max_len == 0 || num_pages == 0) return W4A4_OK;
  const KvNew x{k, v, k_tok, k_head, v_tok, v_head, x_dtype == W4A4_Y_BF16};
  w4a4::launch_kv8_append(c, b, x, as_stream(stream));
  return launched();
}

w4a4_status_t kv8_gather(const int8_t* k_cache, const int8_t* v_cache, const float* k_scale, const float* v_scale,
                         int64_t num_pages, int32_t heads, int32_t page, int32_t dim,
                         const int32_t* block_table, int64_t table_ld, const int32_t* cu_seqlens,
                         const int32_t* seq_lens, int64_t B, int64_t T, int64_t max_new, int64_t max_len,
                         void* k, void* v, int32_t y_dtype, void* stream) {
  if (!y_dtype_ok(y_dtype)) return W4A4_E_DTYPE;
  if (!kv_extents_ok(num_pages, heads, page, dim, table_ld, B, T, max_new, max_len)) return W4A4_E_SHAPE;
  if (B == 0 || T == 0 || max_new == 0) return W4A4_OK;
  const KvPool c = pool(k_cache, v_cache, k_scale, v_scale, num_pages, heads, page, dim);
  const KvBatch b = batch(block_table, table_ld, cu_seqlens, seq_lens, B, T, max_new, max_len);
  const w4a4_status_t st = kv_pointers(c, b);
  if (st != W4A4_OK) return st;
  if (!k || !v) return W4A4_E_NULL;
  if (!aligned(k, 16) || !aligned(v, 16)) return W4A4_E_ALIGN;
  w4a4::launch_kv8_gather(c, b, k, v, y_dtype, as_stream(stream));
  return launched();
}

// T q_heads < 2^31: the kernels number query rows in 32 bits.
static bool kv_query_ok(int32_t q_heads, int32_t heads, int64_t T, int64_t window) {
  return q_heads > 0 && q_heads <= 65535 && heads > 0 && q_heads % heads == 0 && window >= 0 &&
         (T <= 0 || T <= kMaxI32 / q_heads);
}

int64_t kv8_attention_workspace(int32_t q_heads, int32_t heads, int32_t page, int32_t dim, int64_t B, int64_t T,
                                int64_t max_new, int64_t max_len, int32_t causal, int64_t window) {
  if (!kv_query_ok(q_heads, heads, T, window) ||
      !kv_extents_ok(0, heads, page, dim, (max_len + page - 1) / (page > 0 ? page : 1), B, T, max_new, max_len))
    return -1;
  if (B == 0 || T == 0 || max_new == 0) return 0;
  const KvPool c = pool(nullptr, nullptr, nullptr, nullptr, 0, heads, page, dim);
  const KvBatch b = batch(nullptr, 0, nullptr, nullptr, B, T, max_new, max_len);
  KvQuery q = {};
  q.heads = q_heads;
  q.causal = causal != 0;
  q.window = window < max_len ? (int)window : 0;
  return w4a4::kv8_attention_workspace(c, b, q);
}

w4a4_status_t kv8_attention(const void* q, int32_t x_dtype, int64_t q_tok, int64_t q_head, int32_t q_heads,
                            const int8_t* k_cache, const int8_t* v_cache, const float* k_scale, const float* v_scale,
                            int64_t num_pages, int32_t heads, int32_t page, int32_t dim,
                            const int32_t* block_table, int64_t table_ld, const int32_t* cu_seqlens,
                            const int32_t* seq_lens, int64_t B, int64_t T, int64_t max_new, int64_t max_len,
                            float scale, int32_t causal, int64_t window, void* workspace, int64_t workspace_bytes,
                            void* y, int32_t y_dtype, float* lse, void* stream) {
  if (!x_dtype_ok(x_dtype) || !y_dtype_ok(y_dtype)) return W4A4_E_DTYPE;
  if (!kv_query_ok(q_heads, heads, T, window)) return W4A4_E_SHAPE;
  if (!kv_extents_ok(num_pages, heads, page, dim, table_ld, B, T, max_new, max_len)) return W4A4_E_SHAPE;
  if (q_tok < 0 || q_head < 0) return W4A4_E_SHAPE;
  if (q_tok % 8 || q_head % 8) return W4A4_E_ALIGN;
  if (B == 0 || T == 0 || max_new == 0) return W4A4_OK;
  const KvPool c = pool(k_cache, v_cache, k_scale, v_scale, num_pages, heads, page, dim);
  KvBatch b = batch(block_table, table_ld, cu_seqlens, seq_lens, B, T, max_new, max_len);
  w4a4_status_t st = kv_pointers(c, b);
  if (st != W4A4_OK) return st;
  if (!q || !y) return W4A4_E_NULL;
  if (!aligned(q, 16) || !aligned(y, 16) || !aligned(lse, 4)) return W4A4_E_ALIGN;
  KvQuery a = {};
  a.q = q; a.q_tok = q_tok; a.q_head = q_head;
  a.bf16 = x_dtype == W4A4_Y_BF16;
  a.heads = q_heads;
  a.scale = scale;
  a.causal = causal != 0;
  a.window = window < max_len ? (int)window : 0;   // a window of every position is none
  a.y = y; a.ydtype = y_dtype; a.lse = lse;
  const int64_t need = w4a4::kv8_attention_workspace(c, b, a);
  if (need < 0 || workspace_bytes < need) return W4A4_E_SHAPE;
  if (need > 0 && !workspace) return W4A4_E_NULL;
  if (need > 0 && !aligned(workspace, 16)) return W4A4_E_ALIGN;
  if (num_pages == 0) b.max_len = 0;               // no page to read: every query sees nothing
  w4a4::launch_kv8_attention(c, b, a, workspace, as_stream(stream));
  return launched();
}

// ---- The rest of a feed-forward block (ffn8.h)

static_assert(W8A8_ACT_NONE == w4a4::ACT_NONE && W8A8_ACT_RELU == w4a4::ACT_RELU && W8A8_ACT_SILU == w4a4::ACT_SILU &&
              W8A8_ACT_GELU == w4a4::ACT_GELU && W8A8_ACT_GELU_TANH == w4a4::ACT_GELU_TANH, "activation codes");
static bool act_ok(int32_t act) { return act >= W8A8_ACT_NONE && act <= W8A8_ACT_GELU_TANH; }

w4a4_status_t w8a8_rmsnorm_quantize(const void* x, int32_t x_dtype, int64_t ldx, const void* residual, int64_t ldr,
                                    const void* weight, int32_t w_dtype, float eps, int64_t M, int64_t K,
                                    int8_t* xq, float* xs, void* h, int64_t ldh, void* y, int64_t ldy, void* stream) {
  if (!x_dtype_ok(x_dtype) || (w_dtype != W4A4_Y_F32 && w_dtype != x_dtype)) return W4A4_E_DTYPE;
  if (M < 0 || M >= kMaxW8Rows || K <= 0 || K % 16 || K > (int64_t{1} << 30) || ldx < K) return W4A4_E_SHAPE;
  if ((residual && (ldr < K || ldh < K)) || (y && ldy < K)) return W4A4_E_SHAPE;
  // a mean of squares below 2^-126 is off by up to 2^-150: nothing beside a normal eps
  if (!(eps >= 0x1p-126f) || !(eps < __builtin_inff())) return W4A4_E_SHAPE;
  if (ldx % 8 || (residual && (ldr % 8 || ldh % 8)) || (y && ldy % 8)) return W4A4_E_ALIGN;
  if (M == 0) return W4A4_OK;
  if (!x || !weight || !xq || !xs || (residual && !h)) return W4A4_E_NULL;
  if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(weight, 16) || !aligned(xq, 16) || !aligned(xs, 4) ||
      (residual && !aligned(h, 16)) || !aligned(y, 16))
    return W4A4_E_ALIGN;
  const Rows rx{x, M, 2 * ldx, 2 * K}, rr{residual, M, 2 * ldr, 2 * K}, rw = flat(weight, K * (w_dtype == W4A4_Y_F32 ? 4 : 2));
  const Rows rq = flat(xq, M * K), rs = flat(xs, 4 * M), ry{y, M, 2 * ldy, 2 * K};
  const Rows rh{residual ? h : nullptr, M, 2 * ldh, 2 * K};
  if (meets_any(rq, rx, rr, rw, rs, rh, ry) || meets_any(rs, rx, rr, rw, rh, ry) || meets_any(ry, rx, rr, rw, rh) ||
      meet(rh, rw) || meet_elsewhere(rh, rx) || meet_elsewhere(rh, rr))
    return W4A4_E_OVERLAP;
  w4a4::W8NormArgs a = {};
  a.x = x; a.residual = residual; a.weight = weight; a.h = h; a.y = y; a.q = xq; a.s = xs;
  a.ldx = ldx; a.ldr = ldr; a.ldh = ldh; a.ldy = ldy; a.M = M; a.K = K;
  a.eps = eps;
  a.bf16 = x_dtype == W4A4_Y_BF16;
  a.weight_f32 = w_dtype == W4A4_Y_F32;
  w4a4::launch_w8a8_rmsnorm(a, as_stream(stream));
  return launched();
}

// Channels of W for N outputs, and the extents of such a product.
static int64_t act_channels(int64_t N, int32_t gated) { return gated ? 2 * N : N; }
// Channels up to 2^22 - 4: a tile's 128 rows of int32 sums, padded to multiples of 4, span
// less than 2^31 bytes.
static bool act_extents_ok(int64_t M, int64_t N, int64_t K, int32_t gated) {
  return N >= 0 && N < kMaxW8Rows && act_channels(N, gated) <= (int64_t{1} << 22) - 4 &&
         w8_extents_ok(M, act_channels(N, gated), K);
}

int64_t w8a8_gemm_act_workspace(int64_t M, int64_t N, int64_t K, int32_t gated, int32_t wide) {
  if (!act_extents_ok(M, N, K, gated)) return -1;
  if (M == 0 || N == 0) return 0;
  return w4a4::w8a8_act_workspace(M, act_channels(N, gated), K, wide && N % 8 == 0);
}

int64_t w8a8_linear_act_workspace(int64_t M, int64_t N, int64_t K, int32_t gated, int32_t wide) {
  const int64_t gemm = w8a8_gemm_act_workspace(M, N, K, gated, wide);
  if (gemm < 0) return -1;
  if (M == 0 || N == 0 || w4a4::w8a8_one_launch(M, act_channels(N, gated), K)) return 0;
  return align256(M * K) + align256(4 * M) + gemm;
}

// Whether y or the workspace meets another buffer of such a product (y may be the
// residual itself). in: the tokens or their codes; xs: their scales, or absent.
static bool act_meets(const Rows& in, const float* xs, const w4a4::W8GemmArgs& g, const w4a4::W8Epilogue& e,
                      const void* workspace, int64_t need) {
  const int64_t outs = e.gated ? g.N / 2 : g.N;
  const Rows y{g.y, g.M, 2 * g.ldy, 2 * outs}, r{e.residual, g.M, 2 * e.ldr, 2 * outs}, space = flat(workspace, need);
  const Rows s = flat(xs, 4 * g.M), w = flat(g.w, g.N * g.K), sw = flat(g.sw, 4 * g.N), b = flat(g.bias, 4 * g.N);
  return meets_any(y, in, s, w, sw, b, space) || meet_elsewhere(y, r) || meets_any(space, in, s, w, sw, b, r);
}

// The checks and the descriptions that the two calls share.
static w4a4_status_t act_call(const int8_t* wq, const float* ws, const float* bias, int32_t act, int32_t gated,
                              const void* residual, int64_t ldr, int64_t M, int64_t N, int64_t K, const void* workspace,
                              void* y, int32_t y_dtype, int64_t ldy, w4a4::W8GemmArgs& g, w4a4::W8Epilogue& e) {
  if (!wq || !ws || !y) return W4A4_E_NULL;
  if (!aligned(wq, 16) || !aligned(ws, 4) || !aligned(bias, 4) || !aligned(y, 2) || !aligned(residual, 2) ||
      !aligned(workspace, 16))
    return W4A4_E_ALIGN;
  g = w4a4::W8GemmArgs{};
  g.w = wq; g.sw = ws; g.bias = bias;
  g.M = M; g.N = act_channels(N, gated); g.K = K;
  g.y = y; g.ydtype = y_dtype; g.ldy = ldy;
  e.act = act;
  e.gated = gated != 0;
  e.residual = residual;
  e.ldr = ldr;
  e.wide = w4a4::w8a8_wide_rows(N, y, ldy, residual, ldr);
  return W4A4_OK;
}

w4a4_status_t w8a8_gemm_act(const int8_t* xq, const float* xs, const int8_t* wq, const float* ws, const float* bias,
                            int32_t act, int32_t gated, const void* residual, int64_t ldr,
                            int64_t M, int64_t N, int64_t K, void* workspace, int64_t workspace_bytes,
                            void* y, int32_t y_dtype, int64_t ldy, void* stream) {
  if (!act_extents_ok(M, N, K, gated) || !act_ok(act)) return W4A4_E_SHAPE;
  if (!x_dtype_ok(y_dtype)) return W4A4_E_DTYPE;
  if (M == 0 || N == 0) return W4A4_OK;
  if (ldy < N || (residual && ldr < N)) return W4A4_E_SHAPE;
  if (!xq || !xs) return W4A4_E_NULL;
  if (!aligned(xq, 16) || !aligned(xs, 4)) return W4A4_E_ALIGN;
  w4a4::W8GemmArgs g;
  w4a4::W8Epilogue e;
  const w4a4_status_t st = act_call(wq, ws, bias, act, gated, residual, ldr, M, N, K, workspace, y, y_dtype, ldy, g, e);
  if (st != W4A4_OK) return st;
  const int64_t need = w8a8_gemm_act_workspace(M, N, K, gated, e.wide);
  if (workspace_bytes < need) return W4A4_E_SHAPE;
  if (need > 0 && !workspace) return W4A4_E_NULL;
  if (act_meets(flat(xq, M * K), xs, g, e, workspace, need)) return W4A4_E_OVERLAP;
  g.a = xq; g.sa = xs;
  g.workspace = workspace;
  w4a4::launch_w8a8_gemm_act(g, e, as_stream(stream));
  return launched();
}

w4a4_status_t w8a8_linear_act(const void* x, int32_t x_dtype, int64_t M, int64_t K, int64_t ldx,
                              const int8_t* wq, const float* ws, const float* bias, int32_t act, int32_t gated,
                              const void* residual, int64_t ldr, int64_t N, void* workspace, int64_t workspace_bytes,
                              void* y, int32_t y_dtype, int64_t ldy, void* stream) {
  if (!act_extents_ok(M, N, K, gated) || ldx < K || !act_ok(act)) return W4A4_E_SHAPE;
  if (!x_dtype_ok(x_dtype) || !x_dtype_ok(y_dtype)) return W4A4_E_DTYPE;
  if (ldx % 8) return W4A4_E_ALIGN;
  if (M == 0 || N == 0) return W4A4_OK;
  if (ldy < N || (residual && ldr < N)) return W4A4_E_SHAPE;
  if (!x) return W4A4_E_NULL;
  if (!aligned(x, 16)) return W4A4_E_ALIGN;
  w4a4::W8GemmArgs g;
  w4a4::W8Epilogue e;
  const w4a4_status_t st = act_call(wq, ws, bias, act, gated, residual, ldr, M, N, K, workspace, y, y_dtype, ldy, g, e);
  if (st != W4A4_OK) return st;
  const int64_t need = w8a8_linear_act_workspace(M, N, K, gated, e.wide);
  if (workspace_bytes < need) return W4A4_E_SHAPE;
  if (need > 0 && !workspace) return W4A4_E_NULL;
  if (act_meets(Rows{x, M, 2 * ldx, 2 * K}, nullptr, g, e, workspace, need)) return W4A4_E_OVERLAP;
  const int bf16 = x_dtype == W4A4_Y_BF16;
  if (w4a4::w8a8_one_launch(M, g.N, K)) {
    w4a4::launch_w8a8_small_act(g, e, x, bf16, ldx, as_stream(stream));
    return launched();
  }
  int8_t* xq = static_cast<int8_t*>(workspace);
  float* xs = reinterpret_cast<float*>(xq + align256(M * K));
  w4a4::launch_w8a8_quant(x, bf16, M, K, ldx, xq, xs, as_stream(stream));
  g.a = xq; g.sa = xs;
  g.workspace = xq + align256(M * K) + align256(4 * M);
  w4a4::launch_w8a8_gemm_act(g, e, as_stream(stream));
  return launched();
}

w4a4_status_t moe_route(const void* logits, int32_t dtype, int64_t T, int64_t E, int64_t ldl, int64_t k,
                        int32_t renormalize, int32_t* ids, float* weights, void* stream) {
  if (!y_dtype_ok(dtype)) return W4A4_E_DTYPE;
  if (T < 0 || T >= kMaxW8Rows || E <= 0 || E > w4a4::kMoeMaxExperts || ldl < E || k <= 0 || k > w4a4::kRouteMaxK)
    return W4A4_E_SHAPE;
  if (T == 0) return W4A4_OK;
  if (!logits || !ids || !weights) return W4A4_E_NULL;
  if (!aligned(logits, dtype == W4A4_Y_F32 ? 4 : 2) || !aligned(ids, 4) || !aligned(weights, 4)) return W4A4_E_ALIGN;
  const int64_t size = dtype == W4A4_Y_F32 ? 4 : 2;
  const Rows rl{logits, T, size * ldl, size * E}, ri = flat(ids, 4 * T * k), rw = flat(weights, 4 * T * k);
  if (meets_any(ri, rl, rw) || meet(rw, rl)) return W4A4_E_OVERLAP;
  w4a4::launch_moe_route(logits, dtype, T, E, ldl, (int)k, renormalize != 0, ids, weights, as_stream(stream));
  return launched();
}

static bool moe_extents_ok(int64_t T, int64_t k, int64_t E, int64_t H, int64_t I) {
  return T >= 0 && k > 0 && T <= w4a4::kMoeMaxPairs && k <= w4a4::kMoeMaxPairs && T * k <= w4a4::kMoeMaxPairs &&
         E > 0 && E <= w4a4::kMoeMaxExperts && H > 0 && H % 16 == 0 && H <= kMaxW8K && I > 0 && I % 16 == 0 &&
         I <= kMaxW8K;
}

int64_t w8a8_moe_workspace(int64_t T, int64_t k, int64_t E, int64_t H, int64_t I) {
  if (!moe_extents_ok(T, k, E, H, I)) return -1;
  return T == 0 ? 0 : w4a4::moe_workspace(T, k, E, H, I);
}

w4a4_status_t w8a8_moe(const int8_t* xq, const float* xs, const int32_t* ids, const float* weights, int64_t T, int64_t k,
                       const int8_t* w13, const float* s13, const int8_t* w2, const float* s2,
                       int64_t E, int64_t H, int64_t I, int32_t act, void* workspace, int64_t workspace_bytes,
                       void* y, int32_t y_dtype, int64_t ldy, void* stream) {
  if (!moe_extents_ok(T, k, E, H, I) || !act_ok(act)) return W4A4_E_SHAPE;
  if (!x_dtype_ok(y_dtype)) return W4A4_E_DTYPE;
  if (T == 0) return W4A4_OK;
  const int64_t need = w8a8_moe_workspace(T, k, E, H, I);
  if (ldy < H || workspace_bytes < need) return W4A4_E_SHAPE;
  if (!xq || !xs || !ids || !weights || !w13 || !s13 || !w2 || !s2 || !y || !workspace) return W4A4_E_NULL;
  if (!aligned(xq, 16) || !aligned(w13, 16) || !aligned(w2, 16) || !aligned(workspace, 16) || !aligned(xs, 4) ||
      !aligned(ids, 4) || !aligned(weights, 4) || !aligned(s13, 4) || !aligned(s2, 4) || !aligned(y, 2))
    return W4A4_E_ALIGN;
  // y is written while the last launch still reads the others
  const Rows ry{y, T, 2 * ldy, 2 * H}, space = flat(workspace, need), ri = flat(ids, 4 * T * k), rf = flat(weights, 4 * T * k);
  const Rows r2 = flat(w2, E * H * I), rs2 = flat(s2, 4 * E * H);
  if (meets_any(ry, ri, rf, r2, rs2, space) ||
      meets_any(space, flat(xq, T * H), flat(xs, 4 * T), ri, rf, flat(w13, 2 * E * I * H), flat(s13, 8 * E * I), r2, rs2))
    return W4A4_E_OVERLAP;
  w4a4::MoeArgs a = {};
  a.xq = xq; a.xs = xs; a.ids = ids; a.weights = weights;
  a.w13 = w13; a.s13 = s13; a.w2 = w2; a.s2 = s2;
  a.T = (int)T; a.k = (int)k; a.E = (int)E; a.H = (int)H; a.I = (int)I;
  a.act = act;
  a.y = y; a.ydtype = y_dtype; a.ldy = ldy;
  a.workspace = workspace;
  w4a4::launch_w8a8_moe(a, as_stream(stream));
  return launched();
}

}  // extern "C"
