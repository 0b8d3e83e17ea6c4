// INT8 key/value cache for gfx950: storing new tokens into its pages and
// reading tokens back as values.
//
// A page holds P positions of one sequence. Per kv head h it has
//   K codes [P][D] and V codes [D][P]  (V with the positions contiguous: the
//   attention kernel then reads both operands of its two products straight
//   from the cache, 16 bytes per lane), and one fp32 scale each.
// Storing (per page and head, K and V alike), with s_old the stored scale if
// the page already holds positions of the sequence, else 0:
//   s = max(s_old, fl32(max|new| / 127))
//   old codes  q <- rne(fl32(q fl32(s_old / s)))   if s > s_old
//   new codes  rne(fl32(x / s)), s = 0 -> 0
// One workgroup owns one (page, head), so nothing else reads or writes it.
#include <algorithm>

#include "kv8_common.h"

namespace w4a4 {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float block_max(float v, float* buf) {
  v = group_max<64>(v);
  __syncthreads();                        // buf may still be read from the last call
  if ((threadIdx.x & 63) == 0) buf[threadIdx.x >> 6] = v;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) v = fmaxf(v, buf[w]);
  return v;
}

__device__ __forceinline__ int8_t code_of(float x, float s) {
  return s > 0.0f ? (int8_t)rintf(x / s) : (int8_t)0;
}
__device__ __forceinline__ int8_t rescaled(int8_t q, float r) { return (int8_t)rintf((float)q * r); }

__global__ __launch_bounds__(kThreads) void k_kv8_append(KvPool c, KvBatch b, KvNew x) {
  __shared__ float buf[kThreads / 64];
  const int seq = blockIdx.z, h = blockIdx.y;
  const Seq s = sequence(b, seq);
  const int p0 = s.len - s.n;                       // position of the first new token (< 0: it is not stored)
  const int first = max(p0, 0);
  const int j = (first >> c.log_page) + blockIdx.x;
  const int P = c.page, D = c.dim;
  const int lo = max(first - j * P, 0), hi = min(s.len - j * P, P);   // new slots of the page
  if (s.n == 0 || hi <= lo) return;
  const int pg = page_of(b, c, seq, j * P);
  if (pg < 0) return;
  const int64_t t = s.t0 + (j * P - p0);            // token of slot 0
  const int64_t base = ((int64_t)pg * c.heads + h) * P * D;
  const int tid = threadIdx.x;

  // K: a thread takes one dimension of a slot
  const uint16_t* kx = static_cast<const uint16_t*>(x.k) + h * x.k_head;
  float a = 0.0f;
  for (int i = lo * D + tid; i < hi * D; i += kThreads) a = fmaxf(a, fabsf(f32_of(kx[(t + i / D) * x.k_tok + i % D], x.bf16)));
  a = block_max(a, buf);
  float* sp = c.ks + (int64_t)pg * c.heads + h;
  float s_new = a / 127.0f, s_old = lo > 0 ? *sp : 0.0f;
  float sc = fmaxf(s_old, s_new);
  int8_t* kq = c.k + base;
  for (int i = lo * D + tid; i < hi * D; i += kThreads) kq[i] = code_of(f32_of(kx[(t + i / D) * x.k_tok + i % D], x.bf16), sc);
  if (sc > s_old && lo > 0) {
    const float r = s_old / sc;
    for (int i = tid; i < lo * D; i += kThreads) kq[i] = rescaled(kq[i], r);
  }
  __syncthreads();                                  // every thread has read *sp
  if (tid == 0) *sp = sc;

  // V: the same with the slots contiguous
  const uint16_t* vx = static_cast<const uint16_t*>(x.v) + h * x.v_head;
  a = 0.0f;
  for (int i = lo * D + tid; i < hi * D; i += kThreads) a = fmaxf(a, fabsf(f32_of(vx[(t + i / D) * x.v_tok + i % D], x.bf16)));
  a = block_max(a, buf);
  sp = c.vs + (int64_t)pg * c.heads + h;
  s_new = a / 127.0f;
  s_old = lo > 0 ? *sp : 0.0f;
  sc = fmaxf(s_old, s_new);
  int8_t* vq = c.v + base;
  for (int i = lo * D + tid; i < hi * D; i += kThreads)
    vq[(i % D) * P + i / D] = code_of(f32_of(vx[(t + i / D) * x.v_tok + i % D], x.bf16), sc);
  if (sc > s_old && lo > 0) {
    const float r = s_old / sc;
    for (int i = tid; i < lo * D; i += kThreads) {
      const int at = (i % D) * P + i / D;
      vq[at] = rescaled(vq[at], r);
    }
  }
  __syncthreads();
  if (tid == 0) *sp = sc;
}

// One workgroup reads the last n positions of a sequence that lie in one page.
__global__ __launch_bounds__(kThreads) void k_kv8_gather(KvPool c, KvBatch b, void* ko, void* vo, int ydt) {
  const int seq = blockIdx.z, h = blockIdx.y;
  const Seq s = sequence(b, seq);
  const int p0 = s.len - s.n;
  const int P = c.page, D = c.dim;
  // tokens before position 0 read as zeros
  if (blockIdx.x == 0) {
    const int none = min(max(-p0, 0), s.n);
    for (int i = threadIdx.x; i < none * D; i += kThreads) {
      const int64_t o = ((int64_t)(s.t0 + i / D) * c.heads + h) * D + i % D;
      store_as(ko, ydt, o, 0.0f);
      store_as(vo, ydt, o, 0.0f);
    }
  }
  const int first = max(p0, 0);
  const int j = (first >> c.log_page) + blockIdx.x;
  const int lo = max(first - j * P, 0), hi = min(s.len - j * P, P);
  if (s.n == 0 || hi <= lo) return;
  const int pg = page_of(b, c, seq, j * P);
  const int64_t t = s.t0 + (j * P - p0);
  const int64_t base = pg < 0 ? 0 : ((int64_t)pg * c.heads + h) * P * D;
  const float ks = pg < 0 ? 0.0f : c.ks[(int64_t)pg * c.heads + h], vs = pg < 0 ? 0.0f : c.vs[(int64_t)pg * c.heads + h];
  for (int i = lo * D + threadIdx.x; i < hi * D; i += kThreads) {
    const int64_t o = ((t + i / D) * c.heads + h) * D + i % D;
    store_as(ko, ydt, o, pg < 0 ? 0.0f : (float)c.k[base + i] * ks);
    store_as(vo, ydt, o, pg < 0 ? 0.0f : (float)c.v[base + (i % D) * P + i / D] * vs);
  }
}

// Pages that a sequence's max_new new tokens can touch.
unsigned page_span(const KvPool& c, const KvBatch& b) {
  const int64_t span = ((int64_t)b.max_new + c.page - 2) / c.page + 1;
  return (unsigned)std::min<int64_t>(span, ((int64_t)b.max_len + c.page - 1) / c.page);
}

}  // namespace

void launch_kv8_append(const KvPool& c, const KvBatch& b, const KvNew& x, hipStream_t stream) {
  const dim3 grid(page_span(c, b), (unsigned)c.heads, (unsigned)b.B);
  hipLaunchKernelGGL(k_kv8_append, grid, dim3(kThreads), 0, stream, c, b, x);
}

void launch_kv8_gather(const KvPool& c, const KvBatch& b, void* k, void* v, int ydt, hipStream_t stream) {
  const dim3 grid(page_span(c, b), (unsigned)c.heads, (unsigned)b.B);
  hipLaunchKernelGGL(k_kv8_gather, grid, dim3(kThreads), 0, stream, c, b, k, v, ydt);
}

}  // namespace w4a4
