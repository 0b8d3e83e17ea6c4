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
// One workgroup owns the K or the V side of one (page, head), so nothing else
// reads or writes it. The new rows are read once, 16 values per piece, and stay
// in registers between the maximum and the codes; V's codes go through LDS in
// position order and leave transposed, 16 positions of a dimension per store.
// Both directions are bound by HBM, 3 bytes per value stored, 3 read back: 24
// ragged prompts of up to 1500 tokens, 8 heads of 128 (91 MB each way) take 24.2
// and 20.1 us, 3.8 and 4.5 TB/s. A decode step's few tokens are bound by the
// chain of loads (lengths, table, scale, codes): 64 tokens 9 and 8 us.
#include <algorithm>

#include "kv8_common.h"
#include "quant8.h"

namespace w4a4 {

namespace {

constexpr int kThreads = 256;

// rne(fl32(q r)) of the four codes of a word (|q r| <= 127): as in codes16, the
// addition of 1.5 2^23 rounds and leaves the code in the low byte. The product
// has to round to fp32 before it (fused, 22 of the 255 codes differ by one for
// s_old / s = 1 / 6).
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float r) {
#pragma clang fp contract(off)
  uint32_t b[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float q = (float)(int)(int8_t)(w >> (8 * i)) * r;
    b[i] = __float_as_uint(q + 12582912.0f);
  }
  return __builtin_amdgcn_perm(b[1], b[0], 0x0C0C0400u) | __builtin_amdgcn_perm(b[3], b[2], 0x04000C0Cu);
}

// 4 x 4 byte transpose: byte j of out[i] is byte i of in[j].
__device__ __forceinline__ void transpose4(const uint32_t in[4], uint32_t out[4]) {
  const uint32_t a0 = __builtin_amdgcn_perm(in[1], in[0], 0x05010400u), a1 = __builtin_amdgcn_perm(in[1], in[0], 0x07030602u);
  const uint32_t b0 = __builtin_amdgcn_perm(in[3], in[2], 0x05010400u), b1 = __builtin_amdgcn_perm(in[3], in[2], 0x07030602u);
  out[0] = __builtin_amdgcn_perm(b0, a0, 0x05040100u);
  out[1] = __builtin_amdgcn_perm(b0, a0, 0x07060302u);
  out[2] = __builtin_amdgcn_perm(b1, a1, 0x05040100u);
  out[3] = __builtin_amdgcn_perm(b1, a1, 0x07060302u);
}

// The new slots of page j of a sequence, and the token of slot 0.
struct Slots {
  int lo, hi;
  int64_t t;
  bool any;
};
__device__ __forceinline__ Slots slots_of(const KvPool& c, const KvBatch& b, const Seq& s, int block, int& j) {
  const int p0 = s.len - s.n, first = max(p0, 0);        // p0 < 0: the first tokens have no position
  j = (first >> c.log_page) + block;
  Slots r;
  r.lo = max(first - j * c.page, 0);
  r.hi = min(s.len - j * c.page, c.page);
  r.t = s.t0 + ((int64_t)j * c.page - p0);
  r.any = s.n > 0 && r.hi > r.lo;
  return r;
}

// LDS row of V codes in position order: D bytes and 4 more, so that the words of
// one column in consecutive rows lie in different banks.
__device__ __forceinline__ int lds_row(int slot, int D) { return slot * (D + 4); }

// NPT pieces per thread cover a page: NPT = ceil(P D / 16 / 256).
template <bool BF, int D, int NPT>
__global__ __launch_bounds__(kThreads) void k_kv8_append(KvPool c, KvBatch b, KvNew x) {
  constexpr int PPT = D / 16;                       // pieces per token
  extern __shared__ __align__(16) uint8_t lds[];    // V codes of the page
  __shared__ float wave_max[kThreads / 64];
  const int seq = blockIdx.z, h = blockIdx.y >> 1;
  const bool is_v = blockIdx.y & 1;
  const Seq s = sequence(b, seq);
  int j;
  const Slots w = slots_of(c, b, s, blockIdx.x, j);
  if (!w.any) return;
  const int P = c.page;
  const int pg = page_of(b, c, seq, j * P);             // on its way while the tokens are loaded
  const int tid = threadIdx.x;
  const uint16_t* src = is_v ? static_cast<const uint16_t*>(x.v) + h * x.v_head : static_cast<const uint16_t*>(x.k) + h * x.k_head;
  const int64_t tok = is_v ? x.v_tok : x.k_tok;
  const int count = (w.hi - w.lo) * PPT;
  uint4 raw[NPT][2];
  uint32_t m = 0;
#pragma unroll
  for (int n = 0; n < NPT; ++n) {
    const int i = tid + kThreads * n;
    raw[n][0] = raw[n][1] = uint4{0, 0, 0, 0};
    if (i < count) {
      const uint4* p = reinterpret_cast<const uint4*>(src + (w.t + w.lo + i / PPT) * tok + i % PPT * 16);
      raw[n][0] = p[0];
      raw[n][1] = p[1];
    }
  }
  if (pg < 0) return;
#pragma unroll
  for (int n = 0; n < NPT; ++n) m = absmax16(raw[n], m);
  float* sp = (is_v ? c.vs : c.ks) + (int64_t)pg * c.heads + h;
  const float s_old = w.lo > 0 ? *sp : 0.0f;
  float a = wave_absmax<BF>(m);
  if ((tid & 63) == 0) wave_max[tid >> 6] = a;
  __syncthreads();                                  // also: every thread has read *sp
#pragma unroll
  for (int i = 0; i < kThreads / 64; ++i) a = max_or_nan(a, wave_max[i]);
  const float sc = max_or_nan(s_old, a / 127.0f);
  const bool grown = w.lo > 0 && sc > s_old;
  const float r = grown ? s_old / sc : 1.0f;
  const float k = scale_guard(sc), sk = sc * k, rs = sc == 0.0f ? 0.0f : 1.0f / sk;
  if (tid == 0) *sp = sc;
  int8_t* q = (is_v ? c.v : c.k) + ((int64_t)pg * c.heads + h) * P * D;
  if (!is_v) {
#pragma unroll
    for (int n = 0; n < NPT; ++n) {
      const int i = tid + kThreads * n;
      if (i < count) *reinterpret_cast<uint4*>(q + w.lo * D + 16 * i) = codes16<BF>(raw[n], k, sk, rs);
    }
    if (grown) {
      for (int i = tid; i < w.lo * PPT; i += kThreads) {
        uint4* p = reinterpret_cast<uint4*>(q + 16 * i);
        const uint4 v = *p;
        *p = uint4{rescale4(v.x, r), rescale4(v.y, r), rescale4(v.z, r), rescale4(v.w, r)};
      }
    }
    return;
  }
#pragma unroll
  for (int n = 0; n < NPT; ++n) {
    const int i = tid + kThreads * n;
    if (i < count) {
      const uint4 v = codes16<BF>(raw[n], k, sk, rs);
      uint32_t* p = reinterpret_cast<uint32_t*>(lds + lds_row(w.lo + i / PPT, D) + i % PPT * 16);
      p[0] = v.x;
      p[1] = v.y;
      p[2] = v.z;
      p[3] = v.w;
    }
  }
  __syncthreads();
  // units of 4 dimensions x 16 slots, for the groups of 16 slots that change
  const int g0 = grown ? 0 : w.lo >> 4, groups = ((w.hi + 15) >> 4) - g0;
  for (int u = tid; u < groups * (D / 4); u += kThreads) {
    const int g = g0 + u % groups, d = u / groups * 4;
    uint32_t col[4][4];                             // [dimension][4 slots]
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t in[4], out[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int slot = 16 * g + 4 * i + e;
        in[e] = slot >= w.lo && slot < w.hi ? *reinterpret_cast<const uint32_t*>(lds + lds_row(slot, D) + d) : 0;
      }
      transpose4(in, out);
#pragma unroll
      for (int e = 0; e < 4; ++e) col[e][i] = out[e];
    }
    const bool whole = 16 * g >= w.lo && 16 * g + 16 <= w.hi;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      uint4* p = reinterpret_cast<uint4*>(q + (d + e) * P + 16 * g);
      uint32_t o[4] = {col[e][0], col[e][1], col[e][2], col[e][3]};
      if (!whole) {
        // slots before the new ones (rescaled) and behind them (as they are) stay
        const uint4 v = *p;
        const uint32_t had[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t fresh = 0, older = 0;            // byte masks
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const int slot = 16 * g + 4 * i + y;
            if (slot >= w.lo && slot < w.hi) fresh |= 0xFFu << (8 * y);
            if (slot < w.lo) older |= 0xFFu << (8 * y);
          }
          const uint32_t aged = grown ? rescale4(had[i], r) : had[i];
          o[i] = (o[i] & fresh) | (aged & older) | (had[i] & ~(fresh | older));
        }
      }
      *p = uint4{o[0], o[1], o[2], o[3]};
    }
  }
}

// 16 values of a piece, code * scale, as the output type.
template <int YT>
__device__ __forceinline__ void store16(void* y, int64_t at, const uint4& v, float s) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  float f[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) f[i] = (float)(int)(int8_t)(w[i >> 2] >> (8 * (i & 3))) * s;
  if constexpr (YT == 0) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(y) + at);
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = float4{f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]};
  } else {
    uint4* p = reinterpret_cast<uint4*>(static_cast<uint16_t*>(y) + at);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t o[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        o[e] = u16_of(f[8 * i + 2 * e], YT == 2) | (uint32_t)u16_of(f[8 * i + 2 * e + 1], YT == 2) << 16;
      p[i] = uint4{o[0], o[1], o[2], o[3]};
    }
  }
}

// One workgroup reads the K or the V side of the last n positions of a sequence
// that lie in one page.
template <int D, int YT>
__global__ __launch_bounds__(kThreads) void k_kv8_gather(KvPool c, KvBatch b, void* ko, void* vo) {
  constexpr int PPT = D / 16;
  extern __shared__ __align__(16) uint8_t lds[];
  const int seq = blockIdx.z, h = blockIdx.y >> 1;
  const bool is_v = blockIdx.y & 1;
  const Seq s = sequence(b, seq);
  const int tid = threadIdx.x, P = c.page;
  void* y = is_v ? vo : ko;
  auto row = [&](int64_t t) { return (t * c.heads + h) * D; };
  if (blockIdx.x == 0) {                            // tokens before position 0 read as zeros
    const int none = max(s.n - s.len, 0);
    for (int i = tid; i < none * PPT; i += kThreads)
      store16<YT>(y, row(s.t0 + i / PPT) + i % PPT * 16, uint4{0, 0, 0, 0}, 0.0f);
  }
  int j;
  const Slots w = slots_of(c, b, s, blockIdx.x, j);
  if (!w.any) return;
  const int count = (w.hi - w.lo) * PPT;
  const int pg = page_of(b, c, seq, j * P);
  if (pg < 0) {                                     // no page of the pool: zeros
    for (int i = tid; i < count; i += kThreads)
      store16<YT>(y, row(w.t + w.lo + i / PPT) + i % PPT * 16, uint4{0, 0, 0, 0}, 0.0f);
    return;
  }
  const float sc = (is_v ? c.vs : c.ks)[(int64_t)pg * c.heads + h];
  const int8_t* q = (is_v ? c.v : c.k) + ((int64_t)pg * c.heads + h) * P * D;
  if (is_v) {
    const int g0 = w.lo >> 4, groups = ((w.hi + 15) >> 4) - g0;
    for (int u = tid; u < groups * (D / 4); u += kThreads) {
      const int g = g0 + u % groups, d = u / groups * 4;
      uint4 v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = *reinterpret_cast<const uint4*>(q + (d + e) * P + 16 * g);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t in[4] = {(&v[0].x)[i], (&v[1].x)[i], (&v[2].x)[i], (&v[3].x)[i]};
        uint32_t out[4];
        transpose4(in, out);
#pragma unroll
        for (int e = 0; e < 4; ++e) *reinterpret_cast<uint32_t*>(lds + lds_row(16 * g + 4 * i + e, D) + d) = out[e];
      }
    }
    __syncthreads();
  }
  for (int i = tid; i < count; i += kThreads) {
    const int slot = w.lo + i / PPT, d = i % PPT * 16;
    uint4 v;
    if (is_v) {
      const uint32_t* p = reinterpret_cast<const uint32_t*>(lds + lds_row(slot, D) + d);
      v = uint4{p[0], p[1], p[2], p[3]};
    } else {
      v = *reinterpret_cast<const uint4*>(q + slot * D + d);
    }
    store16<YT>(y, row(w.t + slot) + d, v, sc);
  }
}

// Pages that a sequence's max_new new tokens can touch; 1 at least, whose
// workgroups read tokens without a position.
unsigned page_span(const KvPool& c, const KvBatch& b) {
  const int64_t span = ((int64_t)b.max_new + c.page - 2) / c.page + 1;
  return (unsigned)std::max<int64_t>(1, std::min<int64_t>(span, ((int64_t)b.max_len + c.page - 1) / c.page));
}

unsigned lds_bytes(const KvPool& c) { return (unsigned)(c.page * (c.dim + 4)); }   // <= 66560

template <bool BF, int D>
void append_for(const KvPool& c, const KvBatch& b, const KvNew& x, hipStream_t stream) {
  const dim3 grid(page_span(c, b), (unsigned)(2 * c.heads), (unsigned)b.B);
  // a decode step's few tokens need no more pieces than they have
  const int64_t rows = std::min<int64_t>(c.page, b.max_new);
  const int64_t npt = (rows * D / 16 + kThreads - 1) / kThreads;
#define KV8_APPEND(NPT) hipLaunchKernelGGL((k_kv8_append<BF, D, NPT>), grid, dim3(kThreads), lds_bytes(c), stream, c, b, x)
  if (npt <= 1) KV8_APPEND(1);
  else if (npt <= 2) KV8_APPEND(2);
  else if (npt <= 4) KV8_APPEND(4);
  else if (npt <= 8) KV8_APPEND(8);
  else KV8_APPEND(16);
#undef KV8_APPEND
}

template <int D>
void gather_for(const KvPool& c, const KvBatch& b, void* k, void* v, int ydt, hipStream_t stream) {
  const dim3 grid(page_span(c, b), (unsigned)(2 * c.heads), (unsigned)b.B);
#define KV8_GATHER(YT) hipLaunchKernelGGL((k_kv8_gather<D, YT>), grid, dim3(kThreads), lds_bytes(c), stream, c, b, k, v)
  if (ydt == 0) KV8_GATHER(0);
  else if (ydt == 1) KV8_GATHER(1);
  else KV8_GATHER(2);
#undef KV8_GATHER
}

}  // namespace

void launch_kv8_append(const KvPool& c, const KvBatch& b, const KvNew& x, hipStream_t stream) {
  switch (c.dim) {
    case 64: x.bf16 ? append_for<true, 64>(c, b, x, stream) : append_for<false, 64>(c, b, x, stream); return;
    case 128: x.bf16 ? append_for<true, 128>(c, b, x, stream) : append_for<false, 128>(c, b, x, stream); return;
    case 192: x.bf16 ? append_for<true, 192>(c, b, x, stream) : append_for<false, 192>(c, b, x, stream); return;
    default: x.bf16 ? append_for<true, 256>(c, b, x, stream) : append_for<false, 256>(c, b, x, stream); return;
  }
}

void launch_kv8_gather(const KvPool& c, const KvBatch& b, void* k, void* v, int ydt, hipStream_t stream) {
  switch (c.dim) {
    case 64: gather_for<64>(c, b, k, v, ydt, stream); return;
    case 128: gather_for<128>(c, b, k, v, ydt, stream); return;
    case 192: gather_for<192>(c, b, k, v, ydt, stream); return;
    default: gather_for<256>(c, b, k, v, ydt, stream); return;
  }
}

}  // namespace w4a4
