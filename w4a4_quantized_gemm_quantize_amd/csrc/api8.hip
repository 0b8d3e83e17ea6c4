// C ABI of the 8-bit operators (w8a8_*, include/w4a4.h; kv8_*, include/kv8.h):
// argument validation, then the launches of one call.
#include <hip/hip_runtime.h>
#include <stdint.h>

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

}  // extern "C"
