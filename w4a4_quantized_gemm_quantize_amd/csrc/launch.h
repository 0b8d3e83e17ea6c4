// Internal launchers behind the C ABI. Arguments are validated by the caller
// (api.hip); these only pick a kernel configuration and enqueue it.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace w4a4 {

void launch_int4_quant(const void* x, int64_t M, int64_t K, int64_t ldx, int group,
                       uint8_t* q, float* s, hipStream_t stream);

// mode 0: MXFP4 codes of x; 1: [Q(x) | Q(x - deq Q(x))] along K (width 2K);
// 2: [Q(x) | Q(x)] (width 2K); 3: as 1 with the second scale tied to the
// first (first exponent: nothing clips; second: the first minus 2)
void launch_mxfp4_quant(const void* x, int64_t rows, int64_t K, int64_t ldx,
                        uint8_t* q, uint8_t* e8m0, int mode, hipStream_t stream);

// Window [m0, m0+mc) x [n0, n0+nc); for the plain GEMM the window is the whole
// output and partials == nullptr.
struct GemmArgs {
  const uint8_t* a;
  const void* sa;      // float* (INT4) or uint8_t* (MXFP4, NVFP4)
  const uint8_t* w;
  const void* sw;
  int ga, gw;          // INT4 group sizes (unused for MXFP4)
  int64_t M, N, K;
  void* y;
  int ydtype;
  int64_t ldy;
  int64_t m0, mc, n0, nc;
  int32_t* partials;
};

void launch_w4a4_gemm(const GemmArgs& a, hipStream_t stream);

// K split of the tiled W4A4 GEMM: `splits` workgroups per output tile, each
// over `stages_per_split` 128-k stages (whole groups), fp32 partial outputs in
// a workspace [splits][M][N], summed in split order into y.
struct SplitPlan {
  int splits;
  int stages_per_split;
};
// requested <= 0: enough splits to fill the chip when the tile grid does not
SplitPlan plan_w4a4_splitk(int64_t M, int64_t N, int64_t K, int ga, int gw, int requested);
void launch_w4a4_gemm_splitk(const GemmArgs& a, const SplitPlan& plan, float* workspace, hipStream_t stream);
void launch_mxfp4_gemm(const GemmArgs& a, hipStream_t stream);

// Fused decode path: activation quantization in the few-token GEMM (one
// launch). Supported when M <= 32, the activation group is 64/128/256/512 and
// the workgroup's LDS copy of the quantized activations fits kLinearSmallLds.
constexpr int64_t kLinearSmallLds = 64 * 1024;
bool linear_small_supported(int64_t M, int64_t N, int64_t K, int64_t ga, int64_t gw);
void launch_w4a4_linear_small(const void* x, int64_t M, int64_t K, int64_t ldx, int ga, const uint8_t* wq,
                              const float* ws, int gw, int64_t N, void* y, int ydtype, int64_t ldy,
                              hipStream_t stream);

// NVFP4: *gscale = fl32(max|x| / 2688) (0 for rows == 0)
void launch_nvfp4_global_scale(const void* x, int64_t rows, int64_t K, int64_t ldx, float* gscale,
                               hipStream_t stream);
void launch_nvfp4_quant(const void* x, int64_t rows, int64_t K, int64_t ldx, const float* gscale,
                        uint8_t* q, uint8_t* scales, hipStream_t stream);
// a.sa / a.sw: E4M3 panel scales; ga, gw: device pointers to the global scales
// (unused by the partials export)
void launch_nvfp4_gemm(const GemmArgs& a, const float* ga, const float* gw, hipStream_t stream);

// Storage conversions (layout.hip). count: device int32 receiving the number
// of -8 codes (none may be NULL: not counted).
void launch_repack_int4(const uint8_t* nibbles, int64_t rows, int64_t K, uint8_t* packed, int32_t* count,
                        hipStream_t stream);
void launch_unpack_int4(const uint8_t* packed, int64_t rows, int64_t K, uint8_t* nibbles, hipStream_t stream);
void launch_transpose_f32(const float* in, int64_t rows, int64_t cols, float* out, hipStream_t stream);
// fmt 0: E8M0 (blocks of 32), 1: E4M3 (blocks of 16); nb = blocks per row
void launch_scale_panels(int fmt, bool to_panels, const uint8_t* in, int64_t rows, int64_t nb, uint8_t* out,
                         hipStream_t stream);

// ---- 8-bit linear layers (w8a8.hip). bf16: x is bf16, else fp16.
void launch_w8a8_quant(const void* x, int bf16, int64_t M, int64_t K, int64_t ldx, int8_t* q, float* s,
                       hipStream_t stream);

struct W8GemmArgs {
  const int8_t* a;
  const float* sa;
  const int8_t* w;
  const float* sw;
  const float* bias;   // or nullptr
  int64_t M, N, K;
  void* y;
  int ydtype;          // 0 fp32, 1 fp16, 2 bf16
  int64_t ldy;
  void* workspace;     // w8a8_workspace(M, N, K) bytes
};
int64_t w8a8_workspace(int64_t M, int64_t N, int64_t K);
void launch_w8a8_gemm(const W8GemmArgs& a, hipStream_t stream);
// A linear layer of few tokens in one launch that quantizes them itself: where
// it is taken, and the launch (a.a and a.sa are not used).
bool w8a8_one_launch(int64_t M, int64_t N, int64_t K);
void launch_w8a8_small(const W8GemmArgs& a, const void* x, int bf16, int64_t ldx, hipStream_t stream);

// ---- INT8 key/value cache (kv8_cache.hip, kv8_attention.hip)
struct KvPool {
  int8_t* k;           // [num_pages][heads][page][dim]
  int8_t* v;           // [num_pages][heads][dim][page]
  float* ks;           // [num_pages][heads]
  float* vs;
  int num_pages, heads, page, dim, log_page;
};

struct KvBatch {
  const int32_t* table;   // [B][table_ld] pages of each sequence
  int64_t table_ld;
  const int32_t* cu;      // [B + 1] first token of each sequence in the packed tensors
  const int32_t* lens;    // [B] positions in the cache, the new tokens included
  int B, T, max_new, max_len;
};

struct KvNew {
  const void* k;
  const void* v;
  int64_t k_tok, k_head, v_tok, v_head;   // strides in elements
  int bf16;
};
void launch_kv8_append(const KvPool& c, const KvBatch& b, const KvNew& x, hipStream_t stream);
void launch_kv8_gather(const KvPool& c, const KvBatch& b, void* k, void* v, int ydt, hipStream_t stream);

struct KvQuery {
  const void* q;
  int64_t q_tok, q_head;                  // strides in elements
  int bf16, heads;                        // query heads: a multiple of the cache's
  float scale;
  int causal, window;                     // window 0: none
  void* y;                                // [T][heads][dim]
  int ydtype;
  float* lse;                             // [T][heads] or nullptr
};
int64_t kv8_attention_workspace(const KvPool& c, const KvBatch& b, const KvQuery& q);
void launch_kv8_attention(const KvPool& c, const KvBatch& b, const KvQuery& q, void* workspace, hipStream_t stream);

}  // namespace w4a4
