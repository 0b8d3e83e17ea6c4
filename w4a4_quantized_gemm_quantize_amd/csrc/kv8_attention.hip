// Attention over the INT8 key/value cache for gfx950.
//
// Query token i of the last n of a sequence of L positions sits at pos =
// L - n + i and sees the positions j < L, with causal also j <= pos, with a
// window w also j > pos - w:
//   s_j = scale ks[page(j)] (q . kq_j),  o = sum_j softmax(s)_j vs[page(j)] vq_j
// One pass with a running maximum and sum; no visible position: o = 0 and
// lse = -inf.
//
// Both products run on the fp16 matrix cores with fp32 accumulation. The codes
// are exact in fp16; a page's scale is a factor of the score, or of the
// weight, so no code is ever rounded. bf16 queries are brought to fp16 with a
// power of two per row (the largest element to [2^14, 2^15): elements down to
// 2^-29 of it stay exact, smaller ones are off by 2^-40 of it). The weights
// p_j vs_j enter the second product as fp16(2^b p_j vs_j / vref), vref the
// largest page scale met so far, b = 15 with few query rows and 9 with many: a
// relative rounding of at most 2^-11 for weights down to 2^(-14 - b) of the
// largest one, below that an absolute one of 2^(-25 - b) vref.
//
// Layout. S^T = K Q^T and O^T = V^T P^T with v_mfma_f32_16x16x32_f16: the rows
// of the first product are 64 positions in four tiles, row 4 g + i of tile t
// being position 16 g + 4 t + i (g = lane / 16), so a lane ends up with the
// scores of 16 consecutive positions (of one page) of query row lane % 16.
// Those are the k indices that the second product wants in that lane: the
// weights go from one product's result to the other's operand without
// leaving their lane, and V^T's rows are read as 16 consecutive bytes.
#include <algorithm>
#include <type_traits>

#include "kv8_common.h"
#include "quant8.h"

namespace w4a4 {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNone = -3.0e38f;          // running maximum of a row that has seen nothing
constexpr float kTinyScale = 0x1p-120f, kTinyLog = -120.0f;
// Scores (in log2 units) up to this size keep their factor in the weight's exponent,
// one fma; the maximum that is taken from it there has rounded, so the largest
// score's exponent is that rounding, not 0. Up to 2^10 it is 2^-14 at most, under
// the weights' own 2^-11. Past 2^25 it would be 2 and more, and a weight no fp16:
// larger scores are rounded first.
constexpr float kFusedScores = 1024.0f;
// k_kv8_prefill: weights up to 2^kSlack (the running maximum may lag so far)
// enter fp16 times 2^kBias: at most 2^15
constexpr float kBias = 9.0f, kSlack = 6.0f;

// Four codes as fp16: 1024 + (code + 128) is the bit pattern 0x6400 | byte.
__device__ __forceinline__ void widen4(uint32_t w, h2& a, h2& b) {
  const uint32_t u = w ^ 0x80808080u;
  const h2 bias = {(_Float16)1152.0f, (_Float16)1152.0f};
  a = __builtin_bit_cast(h2, __builtin_amdgcn_perm(0x64646464u, u, 0x04010400u)) - bias;
  b = __builtin_bit_cast(h2, __builtin_amdgcn_perm(0x64646464u, u, 0x04030402u)) - bias;
}
__device__ __forceinline__ v8h widen8(uint32_t x, uint32_t y) {
  h2 a, b, c, d;
  widen4(x, a, b);
  widen4(y, c, d);
  return v8h{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

struct AttnParams {
  KvPool c;
  KvBatch b;
  KvQuery q;
  int group;             // query heads per kv head
  unsigned group_magic;  // ceil(2^32 / group), for token_of
  int tile_rows, tiles;  // query rows per workgroup, row tiles of the longest sequence
  int splits;
  int split;             // positions per split (a multiple of 64 times the waves)
  float* part;           // splits' results: [splits][T heads][dim] then [splits][T heads][2]
  int64_t part_rows;     // T heads
};

typedef float v16f __attribute__((ext_vector_type(16)));

// One query row of D elements, a lane holding N pieces of 8: loads, and later the
// fp16 operands. bf16 rows are scaled by a power of two, returned as the factor
// that undoes it; the row's other elements lie FIRST_XOR .. 32 lanes away. A
// negative softmax scale is moved into the queries (flip), so that every factor
// of a score is >= 0.
template <int N, typename Dim>
__device__ __forceinline__ void load_query(const uint16_t* qp, Dim dim, uint4 (&raw)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) raw[i] = *reinterpret_cast<const uint4*>(qp + dim(i));
}
template <int N, int FIRST_XOR>
__device__ __forceinline__ float query_operands(uint4 (&raw)[N], bool bf16, bool flip, v8h (&qf)[N]) {
  const uint32_t sign = flip ? 0x80008000u : 0u;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    raw[i].x ^= sign;
    raw[i].y ^= sign;
    raw[i].z ^= sign;
    raw[i].w ^= sign;
  }
  if (!bf16) {
#pragma unroll
    for (int i = 0; i < N; ++i) qf[i] = __builtin_bit_cast(v8h, raw[i]);
    return 1.0f;
  }
  uint32_t m = 0;
  static_assert(N % 2 == 0, "16 elements at a time");
#pragma unroll
  for (int i = 0; i < N; i += 2) m = absmax16(raw + i, m);
  m = max(m & 0xFFFFu, m >> 16) << 16;
#pragma unroll
  for (int x = FIRST_XOR; x < 64; x *= 2) m = max(m, (uint32_t)__shfl_xor((int)m, x));
  // exponent of the largest element to 14; a row of zeros and subnormals stays as it is
  const int e = (int)(m >> 23), up = min(max(127 + 14 + 127 - e, 1), 254);
  const float mul = e == 0 ? 1.0f : __uint_as_float((uint32_t)up << 23);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      qf[i][2 * k] = (_Float16)(__uint_as_float(w[k] << 16) * mul);
      qf[i][2 * k + 1] = (_Float16)(__uint_as_float(w[k] & 0xFFFF0000u) * mul);
    }
  }
  return 1.0f / mul;
}

// Maximum over a lane and its partner in the other half of the wave.
__device__ __forceinline__ float max_halves(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float lane_value(float x, int lane) {
  return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(x), lane));
}

// log2 of a page scale, subnormal ones too (the instruction takes them as zeros).
__device__ __forceinline__ float log2_scale(float x) {
  const bool tiny = x < 0x1p-126f;
  return __builtin_amdgcn_logf(tiny ? x * 0x1p32f : x) - (tiny ? 32.0f : 0.0f);
}

// Four outputs at a multiple of 4 elements of the 16-byte aligned y.
__device__ __forceinline__ void store4_as(void* y, int ydt, int64_t i, v4f v) {
  if (ydt == 0) {
    *reinterpret_cast<v4f*>(static_cast<float*>(y) + i) = v;
  } else {
    const bool bf = ydt == 2;
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(y) + i) =
        uint2{u16_of(v[0], bf) | (uint32_t)u16_of(v[1], bf) << 16, u16_of(v[2], bf) | (uint32_t)u16_of(v[3], bf) << 16};
  }
}

// A query at position x sees positions below this; at a negative one it sees none.
__device__ __forceinline__ int sees_below(const AttnParams& p, const Seq& s, int x) {
  return p.q.causal ? min(s.len, x + 1) : x < 0 ? 0 : s.len;
}

// Positions the tokens [t0, t1] of a sequence can see: [lo, hi), lo a multiple of
// 64.
struct Range {
  int lo, hi;
};
__device__ __forceinline__ Range token_range(const AttnParams& p, const Seq& s, int t0, int t1) {
  const int p0 = s.len - s.n;
  Range r{0, s.len};
  if (p.q.causal) r.hi = min(s.len, p0 + t1 + 1);
  if (p.q.window > 0) r.lo = max(0, p0 + t0 - p.q.window + 1) & ~63;
  r.hi = max(r.hi, r.lo);
  return r;
}
// The same for a tile of query rows [r0, r1).
__device__ __forceinline__ Range tile_range(const AttnParams& p, const Seq& s, int r0, int r1) {
  return token_range(p, s, r0 / p.group, (r1 - 1) / p.group);
}

// A workgroup's work: row tile `tile` of (sequence, kv head, split), the heads
// innermost: where they are a multiple of 8, the tiles of one head run on one
// XCD (workgroup index mod 8), whose L2 fetches its codes once. (As a grid of
// three dimensions, without the divisions, 131072 positions took 2 % longer.)
struct Work {
  int seq, h, split, tile;
};
__device__ __forceinline__ Work work_of(const AttnParams& p) {
  Work w;
  unsigned x = blockIdx.x;
  w.h = x % p.c.heads;
  x /= p.c.heads;
  w.tile = x % p.tiles;
  x /= p.tiles;
  w.split = x % p.splits;
  w.seq = x / p.splits;
  return w;
}

// r / group for the rows of k_kv8_decode and k_kv8_draft: r (ceil(2^32 / group)
// group - 2^32) < 2^32, since r < 2^16 and group < 2^16.
__device__ __forceinline__ int token_of(const AttnParams& p, int r) {
  return p.group == 1 ? r : (int)__umulhi((unsigned)r, p.group_magic);
}

// The end of a workgroup whose NW waves hold partial results of the same R query
// rows (unnormalized sums, running maximum, sum of weights): the rows' outputs,
// or the split's part for k_kv8_join.
template <int D, int NW, int R>
__device__ __forceinline__ void join_waves(const AttnParams& p, const Seq& s, const Work& wk, int r0, int rows, int nsplit,
                                           const float (&lo_)[NW][R][D + 4], const float (&lm)[NW][R],
                                           const float (&ll)[NW][R]) {
  __syncthreads();
  for (int i = threadIdx.x; i < R * D / 4; i += 64 * NW) {
    const int r = r0 + i / (D / 4), d = i % (D / 4) * 4;
    if (r >= rows) break;
    float M = kNone;
#pragma unroll
    for (int w = 0; w < NW; ++w) M = fmaxf(M, lm[w][r - r0]);
    float L = 0.0f;
    v4f o = {0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float e = __builtin_amdgcn_exp2f(lm[w][r - r0] - M);
      L += ll[w][r - r0] * e;
      o += *reinterpret_cast<const v4f*>(&lo_[w][r - r0][d]) * e;
    }
    const int tok = token_of(p, r);
    const int64_t row = (int64_t)(s.t0 + tok) * p.q.heads + wk.h * p.group + r - tok * p.group;
    if (nsplit == 1) {
      store4_as(p.q.y, p.q.ydtype, row * D + d, L == 0.0f ? v4f{0, 0, 0, 0} : o * (1.0f / L));
      if (p.q.lse && d == 0) p.q.lse[row] = L == 0.0f ? -INFINITY : (M + __builtin_amdgcn_logf(L)) / kLog2e;
    } else {
      const int64_t at = wk.split * p.part_rows + row;
      *reinterpret_cast<v4f*>(p.part + at * D + d) = o;
      if (d == 0) *reinterpret_cast<float2*>(p.part + (int64_t)p.splits * p.part_rows * D + 2 * at) = float2{M, L};
    }
  }
}

// Few query rows per kv head: a workgroup of NW waves takes 16 rows (token,
// query head of the group) of one kv head and a split of the positions; its
// waves take chunks of 64 positions in turn, with no sharing until the end.
// Bound by HBM: 64 ragged rows up to 4096, 8 query heads per kv head, 57 us, 4.8
// TB/s of codes; 131072 positions 43 us and a joining launch. Short contexts by the chain of loads
// (lengths, table, codes) and the launch: 257 positions 7.4 us. Two chunks in
// flight per wave instead of one measured the same (61.2 and 62.6 us for the 64
// rows, 43.5 and 40.0 for 20 of 4096), three waves per SIMD in place of two were
// slower (75).
template <int D, int NW>
__global__ __launch_bounds__(64 * NW)
__attribute__((amdgpu_waves_per_eu(D > 192 ? 1 : 2, D > 192 ? 1 : 2))) void k_kv8_decode(AttnParams p) {
  constexpr int DB = D / 64, DT = D / 16;
  __shared__ __align__(16) float lo_[NW][16][D + 4];
  __shared__ float lm[NW][16], ll[NW][16];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, g = lane >> 4;
  const Work w = work_of(p);
  const int seq = w.seq, h = w.h, tile = w.tile;
  const Seq s = sequence(p.b, seq);
  const int rows = s.n * p.group;
  const int r0 = tile * 16;
  if (r0 >= rows) return;
  const Range rg = token_range(p, s, token_of(p, r0), token_of(p, min(r0 + 16, rows) - 1));
  const int nsplit = max(1, (rg.hi - rg.lo + p.split - 1) / p.split);
  if (w.split >= nsplit) return;
  const int from = rg.lo + w.split * p.split, to = min(rg.hi, from + p.split);

  // query row of this lane's column
  const int r = min(r0 + c, rows - 1);
  const int tok = token_of(p, r), hq = h * p.group + r - tok * p.group;
  const int pos = s.len - s.n + tok;
  auto hi_of = [&](int x) { return sees_below(p, s, x); };
  auto lo_of = [&](int x) { return p.q.window > 0 ? max(0, x - p.q.window + 1) : 0; };
  const int row_hi = hi_of(pos), row_lo = lo_of(pos);
  // positions that every row of the tile sees
  const int all_hi = min(hi_of(s.len - s.n + token_of(p, r0)), to);
  const int all_lo = lo_of(s.len - s.n + token_of(p, min(r0 + 15, rows - 1)));
  const int P = p.c.page;
  const int* const table = p.b.table + seq * p.b.table_ld;
  const uint32_t page_bytes = (uint32_t)p.c.heads * P * D;     // < 2^32
  const int8_t* const k_head = p.c.k + (int64_t)h * P * D;
  const int8_t* const v_head = p.c.v + (int64_t)h * P * D;
  // This lane's pages as a reader of K rows (positions 16 (c / 4) .. of a chunk)
  // and as the owner of scores and V columns (positions 16 g ..): the table's
  // entries as they are, judged when they are used; positions past the last
  // one take its page. Everything of a chunk is loaded while the one before it
  // is worked on: its pages one chunk earlier still, K's codes once the scores
  // have left their registers, V's once the values have.
  int gk, gv;
  auto load_pages = [&](int at) {
    gk = table[min(at + 16 * (c >> 2), to - 1) >> p.c.log_page];
    gv = table[min(at + 16 * g, to - 1) >> p.c.log_page];
  };
  auto page_ok = [&](int id) { return (unsigned)id < (unsigned)p.c.num_pages; };
  uint4 kr[4][DB], vr[DT];
  float ks, vs, ks_next, vs_next;
  bool ok, ok_next;                                    // the page of this lane's scores is one of the pool
  const int8_t* vp;
  auto load_k = [&](int at) {
    const int8_t* kp = k_head + (uint64_t)(uint32_t)(page_ok(gk) ? gk : 0) * page_bytes +
                       (((at + 16 * (c >> 2)) & (P - 1)) + (c & 3)) * D + 16 * g;
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int d = 0; d < DB; ++d) kr[t][d] = *reinterpret_cast<const uint4*>(kp + 4 * t * D + 64 * d);
    ok_next = page_ok(gv);
    const uint32_t page = ok_next ? gv : 0;
    ks_next = p.c.ks[(int64_t)page * p.c.heads + h];
    vs_next = p.c.vs[(int64_t)page * p.c.heads + h];
    vp = v_head + (uint64_t)page * page_bytes + ((at + 16 * g) & (P - 1)) + c * P;
  };
  auto load_v = [&]() {
#pragma unroll
    for (int i = 0; i < DT; ++i) vr[i] = *reinterpret_cast<const uint4*>(vp + 16 * i * P);
  };

  v4f acc[DT];
#pragma unroll
  for (int i = 0; i < DT; ++i) acc[i] = v4f{0, 0, 0, 0};
  float m = kNone, l = 0.0f, vref = kTinyScale;

  uint4 raw[2 * DB];
  const bool work = from + 64 * wave < to;
  if (work) load_pages(from + 64 * wave);
  load_query<2 * DB>(static_cast<const uint16_t*>(p.q.q) + (int64_t)(s.t0 + tok) * p.q.q_tok + hq * p.q.q_head,
                     [&](int i) { return 64 * (i >> 1) + 16 * g + 8 * (i & 1); }, raw);
  if (work) {
    load_k(from + 64 * wave);
    load_pages(from + 64 * (wave + NW));
    load_v();
  }
  v8h qf[2 * DB];
  const float qscale = fabsf(p.q.scale) * kLog2e * query_operands<2 * DB, 16>(raw, p.q.bf16, p.q.scale < 0.0f, qf);
  for (int at = from + 64 * wave; at < to; at += 64 * NW) {
    ks = ks_next;
    vs = vs_next;
    ok = ok_next;
    v4f sc[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      sc[t] = v4f{0, 0, 0, 0};
#pragma unroll
      for (int d = 0; d < DB; ++d) {
        sc[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(widen8(kr[t][d].x, kr[t][d].y), qf[2 * d], sc[t], 0, 0, 0);
        sc[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(widen8(kr[t][d].z, kr[t][d].w), qf[2 * d + 1], sc[t], 0, 0, 0);
      }
    }
    const bool more = at + 64 * NW < to;
    if (more) {
      load_k(at + 64 * NW);
      load_pages(at + 128 * NW);
    }
    float f = ks * qscale;                             // >= 0
    const int first = at + 16 * g;
    float cm = sc[0][0];
    if (at >= all_lo && at + 64 <= all_hi && __all(ok)) {
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) cm = fmaxf(cm, sc[t][i]);
      cm *= f;
      if (__any(fabsf(cm) > kFusedScores)) {
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) sc[t][i] *= f;
        f = 1.0f;
      }
    } else {
      cm = kNone;
      const int lim = ok ? min(row_hi, to) : 0;
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int j = first + 4 * t + i;
          sc[t][i] = j >= row_lo && j < lim ? sc[t][i] * f : -INFINITY;
          cm = fmaxf(cm, sc[t][i]);
        }
      f = 1.0f;
    }
    cm = fmaxf(cm, __shfl_xor(cm, 16));
    cm = max_halves(cm);
    // a block past the last position or of no page: its scale must not count
    const float vs_here = ok && first < to ? vs : 0.0f;
    const float vm = max_halves(fmaxf(vs_here, __shfl_xor(vs_here, 16)));
    const float m2 = fmaxf(m, cm), vref2 = fmaxf(vref, vm);
    const float al = __builtin_amdgcn_exp2f(m - m2);
    const float ao = al * (vref / vref2);
    const float w = vs_here / vref2 * 32768.0f;
    float sum[2] = {l * al, 0.0f};
    v8h pf[2];
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float e = __builtin_amdgcn_exp2f(fmaf(sc[t][i], f, -m2));
        sum[i & 1] += e;
        pf[t >> 1][4 * (t & 1) + i] = (_Float16)(e * w);
      }
    l = sum[0] + sum[1];
    if (__any(m2 != m) || vref2 != vref) {
#pragma unroll
      for (int i = 0; i < DT; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[i][k] *= ao;
    }
    m = m2;
    vref = vref2;
#pragma unroll
    for (int i = 0; i < DT; ++i) {
      acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(widen8(vr[i].x, vr[i].y), pf[0], acc[i], 0, 0, 0);
      acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(widen8(vr[i].z, vr[i].w), pf[1], acc[i], 0, 0, 0);
    }
    if (more) load_v();
  }
  // the lanes of a row hold its positions 16 g .. of each chunk
  l += __shfl_xor(l, 16);
  l += __shfl_xor(l, 32);
  if (g == 0) {
    lm[wave][c] = m;
    ll[wave][c] = l;
  }
  const float back = vref * 0x1p-15f;
#pragma unroll
  for (int i = 0; i < DT; ++i)
#pragma unroll
    for (int k = 0; k < 4; ++k) lo_[wave][c][16 * i + 4 * g + k] = acc[i][k] * back;
  join_waves<D, NW, 16>(p, s, w, r0, rows, nsplit, lo_, lm, ll);
}

// 17 to 128 rows per kv head (drafts being verified, chunks of a few tokens): as
// k_kv8_decode with 32 rows a workgroup, so that a code is widened for twice the
// rows. S^T = K Q^T and O^T = V^T P^T with v_mfma_f32_32x32x16_f16:
// lane l supplies 8 consecutive k of row l % 32 at k offset 8 (l / 32), result
// register i of lane half hi is row 8 (i / 4) + 4 hi + i % 4. A chunk's 64
// positions are two tiles T; that row is position 32 T + 16 hi + i, so a lane
// ends up with the scores of 16 consecutive positions per tile, the k indices
// that the second product wants in it. The dimensions are summed in the order of
// the codes in memory: lane half hi takes dimensions hi D / 2 and up.
//
// Bound by the chain of loads at the start (lengths, table, codes: 4 us of it),
// then by about 5000 cycles a chunk of a wave: its codes' way from memory beside
// 600 vector instructions (320 of them widen codes) and 32 matrix ones. 35 rows
// in a window of 1024, 24 sequences of 4 kv heads: 19 us; 64 rows of 4096, 8
// sequences of 8 kv heads: 34 us in two splits, 47 in one. Eight waves a
// workgroup were slower.
template <int D, int NW>
__global__ __launch_bounds__(64 * NW) __attribute__((amdgpu_waves_per_eu(2, 2))) void k_kv8_draft(AttnParams p) {
  constexpr int KB = D / 32, DT = D / 32;              // 16-byte pieces of a half row of K, 32-dimension tiles of O
  __shared__ __align__(16) float lo_[NW][32][D + 4];
  __shared__ float lm[NW][32], ll[NW][32];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 31, hi = lane >> 5;
  const Work w = work_of(p);
  const int seq = w.seq, h = w.h;
  const Seq s = sequence(p.b, seq);
  const int rows = s.n * p.group;
  const int r0 = w.tile * 32;
  if (r0 >= rows) return;
  const Range rg = token_range(p, s, token_of(p, r0), token_of(p, min(r0 + 32, rows) - 1));
  const int nsplit = max(1, (rg.hi - rg.lo + p.split - 1) / p.split);
  if (w.split >= nsplit) return;
  const int from = rg.lo + w.split * p.split, to = min(rg.hi, from + p.split);

  const int r = min(r0 + c, rows - 1);
  const int tok = token_of(p, r), hq = h * p.group + r - tok * p.group;
  const int pos = s.len - s.n + tok;
  auto hi_of = [&](int x) { return sees_below(p, s, x); };
  auto lo_of = [&](int x) { return p.q.window > 0 ? max(0, x - p.q.window + 1) : 0; };
  const int row_hi = hi_of(pos), row_lo = lo_of(pos);
  const int all_hi = min(hi_of(s.len - s.n + token_of(p, r0)), to);
  const int all_lo = lo_of(s.len - s.n + token_of(p, min(r0 + 31, rows - 1)));
  const int P = p.c.page;
  const int* const table = p.b.table + seq * p.b.table_ld;
  const uint32_t page_bytes = (uint32_t)p.c.heads * P * D;     // < 2^32
  const int8_t* const k_head = p.c.k + (int64_t)h * P * D + hi * (D / 2);
  const int8_t* const v_head = p.c.v + (int64_t)h * P * D + c * P;
  const int kpos = 16 * ((c >> 2) & 1) + 4 * (c >> 3) + (c & 3);   // the position of this lane's K row in a tile
  int gk[2], gv[2];
  auto load_pages = [&](int at) {
#pragma unroll
    for (int T = 0; T < 2; ++T) {
      gk[T] = table[min(at + 32 * T + (kpos & 16), to - 1) >> p.c.log_page];
      gv[T] = table[min(at + 32 * T + 16 * hi, to - 1) >> p.c.log_page];
    }
  };
  auto page_ok = [&](int id) { return (unsigned)id < (unsigned)p.c.num_pages; };
  uint4 kr[2][KB], vr[2][DT];
  float ks[2], vs[2], ks_next[2], vs_next[2];
  bool ok[2], ok_next[2];
  const int8_t* vp[2];
  auto load_k = [&](int at) {
#pragma unroll
    for (int T = 0; T < 2; ++T) {
      const int8_t* kp = k_head + (uint64_t)(uint32_t)(page_ok(gk[T]) ? gk[T] : 0) * page_bytes +
                         ((at + 32 * T + kpos) & (P - 1)) * D;
#pragma unroll
      for (int b = 0; b < KB; ++b) kr[T][b] = *reinterpret_cast<const uint4*>(kp + 16 * b);
      ok_next[T] = page_ok(gv[T]);
      const uint32_t page = ok_next[T] ? gv[T] : 0;
      ks_next[T] = p.c.ks[(int64_t)page * p.c.heads + h];
      vs_next[T] = p.c.vs[(int64_t)page * p.c.heads + h];
      vp[T] = v_head + (uint64_t)page * page_bytes + ((at + 32 * T + 16 * hi) & (P - 1));
    }
  };
  auto load_v = [&]() {
#pragma unroll
    for (int T = 0; T < 2; ++T)
#pragma unroll
      for (int i = 0; i < DT; ++i) vr[T][i] = *reinterpret_cast<const uint4*>(vp[T] + 32 * i * P);
  };

  v16f acc[DT];
#pragma unroll
  for (int i = 0; i < DT; ++i)
#pragma unroll
    for (int k = 0; k < 16; ++k) acc[i][k] = 0.0f;
  float m = kNone, l = 0.0f, vref = kTinyScale;

  uint4 raw[2 * KB];
  const bool work = from + 64 * wave < to;
  if (work) load_pages(from + 64 * wave);
  load_query<2 * KB>(static_cast<const uint16_t*>(p.q.q) + (int64_t)(s.t0 + tok) * p.q.q_tok + hq * p.q.q_head,
                     [&](int i) { return hi * (D / 2) + 8 * i; }, raw);
  if (work) {
    load_k(from + 64 * wave);
    load_pages(from + 64 * (wave + NW));
    load_v();
  }
  v8h qf[2 * KB];
  const float qscale = fabsf(p.q.scale) * kLog2e * query_operands<2 * KB, 32>(raw, p.q.bf16, p.q.scale < 0.0f, qf);
  // The operands stay in LDS, where the wave's result will lie: with them a lane
  // would need more than its 256 registers.
  v8h* const ql = reinterpret_cast<v8h*>(&lo_[wave][0][0]) + lane;
#pragma unroll
  for (int i = 0; i < 2 * KB; ++i) ql[64 * i] = qf[i];
  for (int at = from + 64 * wave; at < to; at += 64 * NW) {
    v16f sc[2];
    int again = 0;
    asm volatile("" : "+v"(again));                    // read them here, not before the loop
    const v8h* const qs = ql + again;
#pragma unroll
    for (int T = 0; T < 2; ++T) {
      ks[T] = ks_next[T];
      vs[T] = vs_next[T];
      ok[T] = ok_next[T];
#pragma unroll
      for (int i = 0; i < 16; ++i) sc[T][i] = 0.0f;
#pragma unroll
      for (int b = 0; b < KB; ++b) {
        sc[T] = __builtin_amdgcn_mfma_f32_32x32x16_f16(widen8(kr[T][b].x, kr[T][b].y), qs[128 * b], sc[T], 0, 0, 0);
        sc[T] = __builtin_amdgcn_mfma_f32_32x32x16_f16(widen8(kr[T][b].z, kr[T][b].w), qs[128 * b + 64], sc[T], 0, 0, 0);
      }
    }
    const bool more = at + 64 * NW < to;
    if (more) {
      load_k(at + 64 * NW);
      load_pages(at + 128 * NW);
    }
    float cm = kNone, f[2] = {ks[0] * qscale, ks[1] * qscale};   // >= 0
    if (at >= all_lo && at + 64 <= all_hi && __all(ok[0] && ok[1])) {
#pragma unroll
      for (int T = 0; T < 2; ++T) {
        float x = sc[T][0];
#pragma unroll
        for (int i = 1; i < 16; ++i) x = fmaxf(x, sc[T][i]);
        cm = T == 0 ? x * f[0] : fmaxf(cm, x * f[1]);   // (NaN queries: not kNone, which is no score)
      }
      if (__any(fabsf(cm) > kFusedScores)) {
#pragma unroll
        for (int T = 0; T < 2; ++T) {
#pragma unroll
          for (int i = 0; i < 16; ++i) sc[T][i] *= f[T];
          f[T] = 1.0f;
        }
      }
    } else {
#pragma unroll
      for (int T = 0; T < 2; ++T) {
        const int first = at + 32 * T + 16 * hi, lim = ok[T] ? min(row_hi, to) : 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          sc[T][i] = first + i >= row_lo && first + i < lim ? sc[T][i] * f[T] : -INFINITY;
          cm = fmaxf(cm, sc[T][i]);
        }
        f[T] = 1.0f;
      }
    }
    cm = max_halves(cm);
    // a block past the last position or of no page: its scale must not count
    const float vs0 = ok[0] && at + 16 * hi < to ? vs[0] : 0.0f, vs1 = ok[1] && at + 32 + 16 * hi < to ? vs[1] : 0.0f;
    const float vm = max_halves(fmaxf(vs0, vs1));
    const float m2 = fmaxf(m, cm), vref2 = fmaxf(vref, vm);
    const float al = __builtin_amdgcn_exp2f(m - m2);
    const float ao = al * (vref / vref2);
    const float unit = 1.0f / vref2;                   // finite: vref2 >= kTinyScale (2^15 over it would not be)
    float sum[2] = {l * al, 0.0f};
    v8h pf[2][2];
#pragma unroll
    for (int T = 0; T < 2; ++T) {
      const float wt = (T ? vs1 : vs0) * unit * 32768.0f;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float e = __builtin_amdgcn_exp2f(fmaf(sc[T][i], f[T], -m2));
        sum[i & 1] += e;
        pf[T][i >> 3][i & 7] = (_Float16)(e * wt);
      }
    }
    l = sum[0] + sum[1];
    if (__any(m2 != m) || vref2 != vref) {
#pragma unroll
      for (int i = 0; i < DT; ++i)
#pragma unroll
        for (int k = 0; k < 16; ++k) acc[i][k] *= ao;
    }
    m = m2;
    vref = vref2;
#pragma unroll
    for (int T = 0; T < 2; ++T)
#pragma unroll
      for (int i = 0; i < DT; ++i) {
        acc[i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(widen8(vr[T][i].x, vr[T][i].y), pf[T][0], acc[i], 0, 0, 0);
        acc[i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(widen8(vr[T][i].z, vr[T][i].w), pf[T][1], acc[i], 0, 0, 0);
      }
    if (more) load_v();
  }
  l += __shfl_xor(l, 32);
  if (hi == 0) {
    lm[wave][c] = m;
    ll[wave][c] = l;
  }
  const float back = vref * 0x1p-15f;
#pragma unroll
  for (int i = 0; i < DT; ++i)
#pragma unroll
    for (int k = 0; k < 4; ++k)
      *reinterpret_cast<v4f*>(&lo_[wave][c][32 * i + 8 * k + 4 * hi]) =
          v4f{acc[i][4 * k] * back, acc[i][4 * k + 1] * back, acc[i][4 * k + 2] * back, acc[i][4 * k + 3] * back};
  join_waves<D, NW, 32>(p, s, w, r0, rows, nsplit, lo_, lm, ll);
}

// Many query rows per kv head: a workgroup of NW waves takes 32 NW / DS rows of
// one kv head and walks over its split of the positions in tiles of 64. The
// tile's codes are loaded 16 per thread and piece one tile ahead, widened to
// fp16 once for all waves and kept in two LDS buffers. A wave owns 32 rows; with
// DS = 2 (wide heads, whose accumulators and queries exceed a wave's 256
// registers) two waves share them, each with the scores and half of O.
//
// S^T = K Q^T and O^T = V^T P^T with v_mfma_f32_32x32x16_f16: row rho of a
// 32-position tile of the first product is position rho with bits 2 and 3
// swapped, so registers 8 v .. 8 v + 7 of lane half hi are the scores of
// positions 16 v + 8 hi .. + 7 of query row lane % 32: the k indices of that
// lane in the second product. A page (>= 16 positions) is uniform over such
// a block of 16, so its scales are scalars: p_j vs_j comes out of one exp2 with
// log2 of the scale in its addend, and the sum of a block's p_j is that of its
// weights over the scale.
//
// LDS rows of K (2 D bytes) and V^T (128 bytes) keep their 16-byte slots
// XOR-swizzled so that 16 consecutive rows hit distinct bank groups.
//
// ONE: a page holds whole tiles, so a tile has one page and one pair of scales,
// fetched through the scalar cache.
//
// Bound by the matrix cores and the vector work beside them (softmax, widening)
// at the clock that the power limit leaves: a step's matrix phase takes 1700 to
// 1950 cycles (1024 of matrix instructions), its vector phase as many, so a tile
// 4200. Four chunks of up to 4096 tokens on as much context, 64 heads over 8 kv
// heads (1214 GFLOP): 1260 us from a cool machine (965 TFLOP/s), 1450 in a row; a
// large fp16 matrix product reaches 1170.
template <typename T>
__device__ __forceinline__ T scalar_load(const T* p) {
  return *(const __attribute__((address_space(4))) T*)p;
}

template <int D, int NW, int DS, bool ONE>
__global__ __launch_bounds__(64 * NW) __attribute__((amdgpu_waves_per_eu(NW / 4, NW / 4)))
void k_kv8_prefill(AttnParams p) {
  constexpr int ST = D / 16, DT = D / 32 / DS;         // k steps of S, the wave's 32-dimension tiles of O
  constexpr int ROWS = 32 * NW / DS;
  constexpr int TW = D > 192 ? 32 : 64, NB = TW / 16;  // positions per tile; the widest heads have no registers for 64
  constexpr int PIECES = TW * D / 16;                  // 16-code pieces of K (or V) per tile
  constexpr int KB = TW * D * 2;                       // bytes of a K (or V) buffer
  constexpr int NP = 2 * PIECES / (64 * NW);           // pieces per thread and tile
  static_assert(NP * 64 * NW == 2 * PIECES && PIECES % 64 == 0, "whole waves load K or V");
  __shared__ __align__(16) uint8_t lk[2][KB];
  __shared__ __align__(16) uint8_t lv[2][KB];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l32 = lane & 31, hi = lane >> 5;
  const Work w = work_of(p);
  // late rows see the most positions: they start first
  const int seq = w.seq, h = w.h, tile = p.tiles - 1 - w.tile;
  const Seq s = sequence(p.b, seq);
  const int rows = s.n * p.group;
  const int r0 = tile * ROWS;
  if (r0 >= rows) return;
  const Range rg = tile_range(p, s, r0, min(r0 + ROWS, rows));
  const int nsplit = max(1, (rg.hi - rg.lo + p.split - 1) / p.split);
  if (w.split >= nsplit) return;
  const int from = rg.lo + w.split * p.split, to = min(rg.hi, from + p.split);

  // this lane's query row, and the positions its wave's rows see
  const int wr0 = r0 + 32 * (wave % (NW / DS)), d0 = wave / (NW / DS) * (D / DS);
  const int r = min(wr0 + l32, rows - 1);
  const int tok = r / p.group, hq = h * p.group + r % p.group;
  auto row_hi = [&](int tk) { return sees_below(p, s, s.len - s.n + tk); };
  auto row_lo = [&](int tk) { return p.q.window > 0 ? max(0, s.len - s.n + tk - p.q.window + 1) : 0; };
  const int my_hi = row_hi(tok), my_lo = row_lo(tok);
  const int tok_a = __builtin_amdgcn_readfirstlane(min(wr0, rows - 1) / p.group);
  const int tok_b = __builtin_amdgcn_readfirstlane(min(wr0 + 31, rows - 1) / p.group);
  const int hi_min = row_hi(tok_a), hi_max = row_hi(tok_b), lo_min = row_lo(tok_a), lo_max = row_lo(tok_b);
  v8h qf[ST];
  float qscale = fabsf(p.q.scale) * kLog2e;
  {
    uint4 raw[ST];
    load_query<ST>(static_cast<const uint16_t*>(p.q.q) + (int64_t)(s.t0 + tok) * p.q.q_tok + hq * p.q.q_head,
                   [&](int i) { return 16 * i + 8 * hi; }, raw);
    qscale *= query_operands<ST, 32>(raw, p.q.bf16, p.q.scale < 0.0f, qf);
  }

  const int P = p.c.page;
  // piece i of this thread: K codes 16 (x % (D / 16)) .. of position x / (D /
  // 16), or V codes of positions 16 (x % NB) .. of dimension x / NB (a wave's
  // pieces are all of one kind)
  auto is_k = [&](int i) {
    return (i + 1) * 64 * NW <= PIECES ? true : i * 64 * NW >= PIECES ? false : i * 64 * NW + 64 * wave < PIECES;
  };
  auto x_of = [&](int i) { return i * 64 * NW + tid - (is_k(i) ? 0 : PIECES); };
  auto pos_of = [&](int i) { return is_k(i) ? x_of(i) / (D / 16) : 16 * (x_of(i) % NB); };
  // Pages: the table's entries as they are, judged when they are used, so that
  // nothing waits for them where they are loaded. Positions past the last one
  // take its page.
  const int* const table = p.b.table + seq * p.b.table_ld;
  const uint32_t page_bytes = (uint32_t)p.c.heads * P * D;     // < 2^32
  const int8_t* const k_head = p.c.k + (int64_t)h * P * D;
  const int8_t* const v_head = p.c.v + (int64_t)h * P * D;
  auto page_at = [&](int pos) { return table[min(pos, to - 1) >> p.c.log_page]; };
  auto page_one = [&](int pos) { return scalar_load(table + (min(pos, to - 1) >> p.c.log_page)); };
  // A step stages the K codes of tile kt and the V codes of the tile before it.
  constexpr int NPG = ONE ? 2 : NP;                    // pages: of K and V, or of each piece
  int pg[NPG];
  uint4 code[NP];
  auto v_tile = [&](int kt) { return max(kt - TW, from); };
  auto tile_of = [&](int i, int kt) { return is_k(i) ? kt : v_tile(kt); };
  auto load_pages = [&](int kt) {
    if constexpr (ONE) {
      pg[0] = page_one(kt);
      pg[1] = page_one(v_tile(kt));
    } else {
#pragma unroll
      for (int i = 0; i < NP; ++i) pg[i] = page_at(tile_of(i, kt) + pos_of(i));
    }
  };
  auto load_codes = [&](int kt) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int x = x_of(i), id = ONE ? __builtin_amdgcn_readfirstlane(pg[is_k(i) ? 0 : 1]) : pg[i];
      const uint32_t page = (unsigned)id < (unsigned)p.c.num_pages ? id : 0;
      const int8_t* src = (is_k(i) ? k_head : v_head) + (uint64_t)page * page_bytes;
      if constexpr (ONE) {
        // the tile's offset in its page, then the piece's in the tile
        const int in = tile_of(i, kt) & (P - 1);
        src += is_k(i) ? in * D : in;
        code[i] = *reinterpret_cast<const uint4*>(src + (uint32_t)(is_k(i) ? 16 * x : x / NB * P + 16 * (x % NB)));
      } else {
        const int in = (tile_of(i, kt) + pos_of(i)) & (P - 1);
        code[i] = *reinterpret_cast<const uint4*>(src + (is_k(i) ? in * D + x % (D / 16) * 16 : x / NB * P + in));
      }
    }
  };
  // Scales of a tile (of this lane's block lane % NB, or of all), loaded while the
  // weights of the tile before it are made, from the page loaded one earlier.
  int pgs, gone, gone_next;
  float ksv, vsv, ks_next, vs_next;
  auto load_scales = [&]() {
    const int id = ONE ? __builtin_amdgcn_readfirstlane(pgs) : pgs;
    gone_next = (unsigned)id >= (unsigned)p.c.num_pages;    // no page of the pool
    const int64_t e = (int64_t)(gone_next ? 0 : id) * p.c.heads + h;
    ks_next = ONE ? scalar_load(p.c.ks + e) : p.c.ks[e];
    vs_next = ONE ? scalar_load(p.c.vs + e) : p.c.vs[e];
  };
  auto scale_pages = [&](int at) { pgs = ONE ? page_one(at) : page_at(at + 16 * (lane % NB)); };
  auto k_slot = [&](int row, int slot) {               // byte offset in a K buffer
    return row * 2 * D + 16 * (slot ^ (D % 128 == 0 ? row & 15 : (row >> 1) & 7));
  };
  auto v_slot = [&](int row, int slot) {               // in a V buffer
    return row * 2 * TW + 16 * (slot ^ (TW == 64 ? (row >> 1) & 7 : (row >> 2) & 3));
  };
  // half j % 2 of piece j / 2 into LDS
  auto write_half = [&](int kt, int j) {
    const int i = j >> 1, x = x_of(i), buf = (tile_of(i, kt) - from) / TW & 1;
    const v8h a = j & 1 ? widen8(code[i].z, code[i].w) : widen8(code[i].x, code[i].y);
    if (is_k(i)) *reinterpret_cast<v8h*>(lk[buf] + k_slot(x / (D / 16), 2 * (x % (D / 16)) + (j & 1))) = a;
    else *reinterpret_cast<v8h*>(lv[buf] + v_slot(x / NB, 2 * (x % NB) + (j & 1))) = a;
  };

  v16f acc[DT];
#pragma unroll
  for (int i = 0; i < DT; ++i)
#pragma unroll
    for (int k = 0; k < 16; ++k) acc[i][k] = 0.0f;
  // running maximum (log2 domain), sum, and log2 of the largest V scale met
  float m = kNone, l = 0.0f, lref = kTinyLog;
  const int krow = (l32 & 0x13) | (l32 & 4) << 1 | (l32 & 8) >> 1;
  v16f sc[TW / 32];
  v8h pf[TW / 32][2];
  auto sees = [&](int at) { return at < to && at < hi_max && at + TW > lo_min; };

  // The matrix work of a step: values of the last tile (VALUES), scores of this
  // one (SCORES), and between its later instructions the staging of the next
  // step's codes. Operand reads run RING ahead of the instructions that use
  // them, in this order; one wave per SIMD does this at a time, so nothing else
  // hides their latency.
  auto matrix_step = [&](int at, auto values_c, auto scores_c) {
    constexpr int NV = decltype(values_c)::value ? DT * NB : 0, NS = decltype(scores_c)::value ? ST * TW / 32 : 0;
    constexpr int RING = D > 128 ? 4 : 6;              // (the wide heads' registers are full)
    const uint8_t* bk = lk[(at - from) / TW & 1];
    const uint8_t* bv = lv[(at - TW - from) / TW & 1];
    auto read = [&](int x) {
      if (x < NV) return *reinterpret_cast<const v8h*>(bv + v_slot(d0 + 32 * (x % DT) + l32, 2 * (x / DT) + hi));
      x -= NV;
      return *reinterpret_cast<const v8h*>(bk + k_slot(32 * (x % (TW / 32)) + krow, 2 * (x / (TW / 32)) + hi));
    };
    // The matrix instructions of the late group, whose waves are the younger
    // ones, would otherwise wait for the early group's vector instructions
    // (2260 cycles a step in place of 1960).
    __builtin_amdgcn_s_setprio(3);
    v8h ring[RING];
#pragma unroll
    for (int x = 0; x < RING; ++x) ring[x] = read(x);
    if constexpr (NS > 0) {
#pragma unroll
      for (int t = 0; t < TW / 32; ++t)
#pragma unroll
        for (int k = 0; k < 16; ++k) sc[t][k] = 0.0f;
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int x = 0; x < NV + NS; ++x) {
      if (x < NV) {
        const int i = x % DT, b = x / DT;
        acc[i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(ring[x % RING], pf[b >> 1][b & 1], acc[i], 0, 0, 0);
      } else {
        const int t = (x - NV) % (TW / 32), u = (x - NV) / (TW / 32);
        sc[t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(ring[x % RING], qf[u], sc[t], 0, 0, 0);
      }
      if (x + RING < NV + NS) ring[x % RING] = read(x + RING);
      constexpr int FIRST = NV + NS - 8 * NP;
      static_assert(NS == 0 || FIRST >= 0, "four instructions per half piece");
      if (NS > 0 && x >= FIRST && (x - FIRST) % 4 == 0) write_half(at + TW, (x - FIRST) / 4);
      __builtin_amdgcn_sched_barrier(0);
    }
    __builtin_amdgcn_s_setprio(0);
  };
  // scores -> weights of the tile at `at`, whose scales this wave holds
  auto weights = [&](int at) {
    // factors of the tile's blocks: of the scores, and log2 of the V scale. A block past the last position or of no page is masked; its scales
    // must not count.
    constexpr int NF = ONE ? 1 : NB;
    float f[NF], lvs[NF];
    int none = 0;
    if constexpr (ONE) {
      f[0] = ksv * qscale;
      lvs[0] = gone ? kTinyLog : log2_scale(vsv);
      none = gone ? (1 << NB) - 1 : 0;
    } else {
      const bool past = at + 16 * (lane % NB) >= to || gone;
      const float lv_ = past ? kTinyLog : log2_scale(vsv);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        f[b] = lane_value(ksv, b) * qscale;
        lvs[b] = lane_value(lv_, b);
        none |= __builtin_amdgcn_readlane(gone, b) << b;
      }
    }
    float lref2 = lref, lmin = lvs[0];
#pragma unroll
    for (int b = 0; b < NF; ++b) {
      lref2 = fmaxf(lref2, lvs[b]);
      lmin = fminf(lmin, lvs[b]);
    }
    float m2;
    // masked positions, scales too far apart for the sum of weights over scale, large
    // scores
    bool rare = at + TW > hi_min || at < lo_max || none || !(lmin >= lref2 - 40.0f);
    float cm = kNone;
    if (!rare) {
#pragma unroll
      for (int g = 0; g < NF; ++g) {                   // scores that share a factor
        float x = sc[g >> 1][8 * (g & 1)];
#pragma unroll
        for (int k = 1; k < 16 * (TW / 32) / NF; ++k) x = fmaxf(x, sc[(8 * g + k) >> 4][(8 * g + k) & 15]);
        cm = g == 0 ? x * f[0] : fmaxf(cm, x * f[g]);   // (NaN queries: not kNone, which is no score)
      }
      rare = __any(fabsf(cm) > kFusedScores);
    }
    if (rare) {
      cm = kNone;
#pragma unroll
      for (int t = 0; t < TW / 32; ++t)
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const int b = 2 * t + (k >> 3), j = at + 16 * b + 8 * hi + (k & 7);
          sc[t][k] = j >= my_lo && j < my_hi && !(none >> b & 1) ? sc[t][k] * f[b % NF] : -INFINITY;
          cm = fmaxf(cm, sc[t][k]);
        }
    }
    // The maximum only has to keep the weights within fp16: it stays where it is
    // until some row passes it by 2^kSlack (rescaling O in most tiles of 8192
    // positions cost 14 % of the time).
    m2 = fmaxf(m, max_halves(cm));
    if (__any(m2 - m > kSlack) || lref2 != lref) {     // (m + kSlack would round where m is large)
      const float al = __builtin_amdgcn_exp2f(m - m2), ao = __builtin_amdgcn_exp2f(m - m2 + (lref - lref2));
      l *= al;
#pragma unroll
      for (int i = 0; i < DT; ++i)
#pragma unroll
        for (int k = 0; k < 16; ++k) acc[i][k] *= ao;
      m = m2;
      lref = lref2;
    }
    if (rare) {
#pragma unroll
      for (int t = 0; t < TW / 32; ++t)
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const int b = 2 * t + (k >> 3);
          const float e = __builtin_amdgcn_exp2f(sc[t][k] - m);
          l += e;
          pf[t][k >> 3][k & 7] = (_Float16)(e * __builtin_amdgcn_exp2f(lvs[b % NF] - lref + kBias));
        }
    } else {
      const float base = kBias - lref - m;
#pragma unroll
      for (int g = 0; g < NF; ++g) {
        const float c = lvs[g] + base;
        float sum[2] = {0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < 16 * (TW / 32) / NF; ++k) {
          const int x = 8 * g + k;
          const float e = __builtin_amdgcn_exp2f(fmaf(sc[x >> 4][x & 15], f[g], c));
          sum[k & 1] += e;
          pf[x >> 4][x >> 3 & 1][x & 7] = (_Float16)e;
        }
        l = fmaf(sum[0] + sum[1], __builtin_amdgcn_exp2f(lref - kBias - lvs[g]), l);
      }
    }
  };

  // Two groups of waves, one wave of each per SIMD, run the same steps half a
  // tile apart: while one group's waves do their matrix work (values of the
  // last tile, scores of this one, staging of the next) the other's turn scores
  // into weights, so the matrix cores and the vector units work at the same
  // time. K is staged a tile ahead of V. A step of the early group reads what both
  // groups staged in the step before; the buffer that is staged into was last
  // read by the late group's step before.
#define PHASE_END()                                                                   \
  {                                                                                   \
    __builtin_amdgcn_s_waitcnt(0xC07F); /* lgkmcnt(0): own LDS accesses are done */   \
    asm volatile("" ::: "memory");                                                    \
    __builtin_amdgcn_sched_barrier(0);                                                \
    __builtin_amdgcn_s_barrier();                                                     \
    __builtin_amdgcn_sched_barrier(0);                                                \
    asm volatile("" ::: "memory");                                                    \
  }
  const bool late = wave >= NW / 2;
  if (from < to) {
    load_pages(from);
    load_codes(from);
#pragma unroll
    for (int j = 0; j < 2 * NP; ++j) write_half(from, j);
    load_pages(from + TW);
    load_codes(from + TW);
    load_pages(from + 2 * TW);
    scale_pages(from);
    load_scales();
    scale_pages(from + TW);
  }
  PHASE_END()
  if (late) PHASE_END()
  for (int at = from; at < to; at += TW) {
    // (a tile that the wave's rows do not see has weights of zero)
    if (at > from) matrix_step(at, std::true_type{}, std::true_type{});
    else matrix_step(at, std::false_type{}, std::true_type{});
    PHASE_END()
    load_codes(at + 2 * TW);
    ksv = ks_next;
    vsv = vs_next;
    gone = gone_next;
    load_scales();
    if constexpr (ONE) {                               // K's page is that of V and of the scales one tile later
      pg[1] = pgs = pg[0];
      pg[0] = page_one(at + 3 * TW);
    } else {
      scale_pages(at + 2 * TW);
      load_pages(at + 3 * TW);
    }
    if (sees(at)) {
      weights(at);
    } else {
#pragma unroll
      for (int b = 0; b < NB; ++b) pf[b >> 1][b & 1] = v8h{};
    }
    PHASE_END()
  }
  if (from < to) matrix_step(from + (to - from + TW - 1) / TW * TW, std::true_type{}, std::false_type{});
  if (!late) PHASE_END()
#undef PHASE_END

  // each half of the wave holds half of a row's sum
  l += __shfl_xor(l, 32);
  if (wr0 + l32 >= rows) return;
  const int64_t row = (int64_t)(s.t0 + tok) * p.q.heads + hq;
  // (exp2 gives no subnormal numbers: where the factor is one, a power of two of it
  // is left for the end)
  const bool tiny = lref < -60.0f;
  const float back = __builtin_amdgcn_exp2f(lref - kBias + (tiny ? 64.0f : 0.0f)), rest = tiny ? 0x1p-64f : 1.0f;
  if (nsplit == 1) {
    const float out = l == 0.0f ? 0.0f : back / l;
#pragma unroll
    for (int i = 0; i < DT; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int64_t o = row * D + d0 + 32 * i + 8 * k + 4 * hi;
        v4f f;
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = l == 0.0f ? 0.0f : acc[i][4 * k + e] * out * rest;
        store4_as(p.q.y, p.q.ydtype, o, f);
      }
    if (p.q.lse && hi == 0 && d0 == 0) p.q.lse[row] = l == 0.0f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) / kLog2e;
  } else {
    const int64_t at = w.split * p.part_rows + row;
#pragma unroll
    for (int i = 0; i < DT; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        *reinterpret_cast<float4*>(p.part + at * D + d0 + 32 * i + 8 * k + 4 * hi) =
            float4{acc[i][4 * k] * back * rest, acc[i][4 * k + 1] * back * rest, acc[i][4 * k + 2] * back * rest,
                   acc[i][4 * k + 3] * back * rest};
    if (hi == 0 && d0 == 0) {
      float* ml = p.part + (int64_t)p.splits * p.part_rows * D + 2 * at;
      ml[0] = m;
      ml[1] = l;
    }
  }
}

// Joins the splits of the query rows, 4 dimensions per thread. FEW splits: D / 4
// threads per row, which read its splits one after the other. Many: a workgroup
// per row, its groups of D / 4 threads taking the splits in turn and meeting in
// LDS. 8 sequences of 64 rows in 2 splits: the call takes 34 us with the first
// form, 38 with the second.
template <int D, bool FEW>
__global__ __launch_bounds__(256) void k_kv8_join(AttnParams p) {
  constexpr int TPS = D / 4, G = 256 / TPS;            // threads per split, groups of them
  constexpr int RPW = FEW ? G : 1, STEP = FEW ? 1 : G;  // rows a workgroup, splits at a time
  __shared__ float so[FEW ? 1 : G][D];
  __shared__ float sm[G], sl[G];
  const int seq = blockIdx.y;
  const Seq s = sequence(p.b, seq);
  const int g = threadIdx.x / TPS, d = threadIdx.x % TPS * 4;
  const int x = blockIdx.x * RPW + (FEW ? g : 0);
  const int h = x % p.c.heads, r = x / p.c.heads;
  if (r >= s.n * p.group || (FEW && g >= G)) return;
  const int r0 = r / p.tile_rows * p.tile_rows;
  const Range rg = tile_range(p, s, r0, min(r0 + p.tile_rows, s.n * p.group));
  const int nsplit = (rg.hi - rg.lo + p.split - 1) / p.split;
  if (nsplit <= 1) return;
  const int64_t t = s.t0 + r / p.group;
  const int head = h * p.group + r % p.group;
  const int64_t row = t * p.q.heads + head;
  const float* ml = p.part + (int64_t)p.splits * p.part_rows * D;
  float M = kNone, L = 0.0f;
  v4f o = {0, 0, 0, 0};
  if (g < G) {
#pragma unroll 4
    for (int i = FEW ? 0 : g; i < nsplit; i += STEP) {
      const int64_t at = i * p.part_rows + row;
      const float2 e = *reinterpret_cast<const float2*>(ml + 2 * at);
      const v4f v = *reinterpret_cast<const v4f*>(p.part + at * D + d);
      const float M2 = fmaxf(M, e.x);
      const float a = __builtin_amdgcn_exp2f(M - M2), b = __builtin_amdgcn_exp2f(e.x - M2);
      L = L * a + e.y * b;
#pragma unroll
      for (int k = 0; k < 4; ++k) o[k] = o[k] * a + v[k] * b;
      M = M2;
    }
  }
  if constexpr (FEW) {
    store4_as(p.q.y, p.q.ydtype, row * D + d, L == 0.0f ? v4f{0, 0, 0, 0} : o * (1.0f / L));
  } else {
    if (g < G) {
      *reinterpret_cast<v4f*>(&so[g][d]) = o;
      if (d == 0) {
        sm[g] = M;
        sl[g] = L;
      }
    }
    __syncthreads();
    if (threadIdx.x >= D) return;
    M = kNone;
#pragma unroll
    for (int i = 0; i < G; ++i) M = fmaxf(M, sm[i]);
    float out = 0.0f;
    L = 0.0f;
#pragma unroll
    for (int i = 0; i < G; ++i) {
      const float e = __builtin_amdgcn_exp2f(sm[i] - M);
      L += sl[i] * e;
      out += so[i][threadIdx.x] * e;
    }
    store_as(p.q.y, p.q.ydtype, row * D + threadIdx.x, L == 0.0f ? 0.0f : out / L);
  }
  if (p.q.lse && (FEW ? d : (int)threadIdx.x) == 0)
    p.q.lse[row] = L == 0.0f ? -INFINITY : (M + __builtin_amdgcn_logf(L)) / kLog2e;
}

constexpr int kWaves = 4;                  // of k_kv8_decode and k_kv8_draft
constexpr int kFewSplits = 8;              // that k_kv8_join reads one after the other

// Which kernel, its query row tiles, and how the positions are split.
//
// Up to 16 rows per kv head: k_kv8_decode. Up to 64, k_kv8_draft (8 sequences,
// 64 rows, 4096 positions, 8 kv heads: 34 us, 42 in the decode kernel; 16 x 64
// rows of 2048, 32 kv heads: 88 and 134). Up to 128 rows as well, where the
// prefill kernel's tiles of 256 rows would leave half of the work empty (8 x 128
// of 2048, 8 kv heads: 28 us, 36 in the prefill kernel; 32 kv heads: 78 and 97),
// except where these tiles fill the chip and end after a few chunks (8 x 128 of
// 512, 32 kv heads: 33 and 30). Above, k_kv8_prefill. Heads of more than 128
// dimensions do not fit k_kv8_draft's registers.
//
// As few splits as fill the chip, since each costs a start, an end and a share
// of the joining launch. One row of 131072 positions, 8 kv heads, in 32 / 64 /
// 128 / 256 / 512 splits (256 .. 4096 workgroups): 50, 51, 55, 63, 82 us; 64 ragged
// rows up to 4096 in 1 / 2 / 4: 58, 69, 79 us. Heads of 64 have half the bytes in
// flight per wave and take twice the workgroups. k_kv8_draft is not split past
// one workgroup a CU: 192 workgroups of 1088 positions take 21 us, 384 of half
// as many 27.
enum Kernel { DECODE, DRAFT, PREFILL };
struct Plan {
  Kernel kernel;
  int tile_rows, tiles, split, splits;
  int64_t blocks;
};
Plan plan(const KvPool& c, const KvBatch& b, const KvQuery& q) {
  Plan pl;
  const int group = q.heads / c.heads;
  const int64_t rows = (int64_t)b.max_new * group;
  const bool full = (int64_t)c.heads * b.B >= 256 && b.max_len <= 512;
  if (c.dim > 128) pl.kernel = rows > 64 ? PREFILL : DECODE;
  else pl.kernel = rows > (full ? 64 : 128) ? PREFILL : rows > 16 ? DRAFT : DECODE;
  pl.tile_rows = pl.kernel == DECODE ? 16 : pl.kernel == DRAFT ? 32 : c.dim <= 128 ? 256 : 128;
  pl.tiles = (int)((rows + pl.tile_rows - 1) / pl.tile_rows);
  int64_t span = b.max_len;
  if (q.window > 0) {
    const int64_t toks = q.causal ? (pl.tile_rows - 1) / group + 2 : b.max_new;
    span = std::min<int64_t>(span, (int64_t)q.window + toks + 64);
  }
  const int64_t work = (int64_t)pl.tiles * c.heads * b.B;
  const int64_t unit = pl.kernel == PREFILL ? 512 : 64 * kWaves;
  const int64_t fill = pl.kernel == PREFILL || (pl.kernel == DECODE && c.dim <= 64) ? 512 : 256;
  const int64_t want = pl.kernel == DRAFT ? std::max<int64_t>(1, fill / work) : (fill + work - 1) / work;
  const int64_t units = (span + unit - 1) / unit;
  // a second launch costs more than two chunks per wave
  const int64_t per = std::max<int64_t>(span <= 512 ? 2 : 1, (units + want - 1) / want);
  pl.split = (int)(per * unit);
  pl.splits = (int)std::max<int64_t>(1, (span + pl.split - 1) / pl.split);
  pl.blocks = (int64_t)c.heads * pl.tiles * pl.splits * b.B;
  return pl;
}

template <int D>
void launch_for(AttnParams p, const Plan& pl, hipStream_t stream) {
  const dim3 grid((unsigned)pl.blocks);
  if (pl.kernel == PREFILL) {
    constexpr int DS = D > 128 ? 2 : 1;
    if (p.c.page >= 64) hipLaunchKernelGGL((k_kv8_prefill<D, 8, DS, true>), grid, dim3(512), 0, stream, p);
    else hipLaunchKernelGGL((k_kv8_prefill<D, 8, DS, false>), grid, dim3(512), 0, stream, p);
  } else if (pl.kernel == DECODE) {
    hipLaunchKernelGGL((k_kv8_decode<D, kWaves>), grid, dim3(64 * kWaves), 0, stream, p);
  } else if constexpr (D <= 128) {
    hipLaunchKernelGGL((k_kv8_draft<D, kWaves>), grid, dim3(64 * kWaves), 0, stream, p);
  }
  if (pl.splits > 1) {
    const int64_t rows = (int64_t)p.b.max_new * p.q.heads, per = pl.splits <= kFewSplits ? 256 / (D / 4) : 1;
    const dim3 jgrid((unsigned)((rows + per - 1) / per), (unsigned)p.b.B);
    if (per > 1) hipLaunchKernelGGL((k_kv8_join<D, true>), jgrid, dim3(256), 0, stream, p);
    else hipLaunchKernelGGL((k_kv8_join<D, false>), jgrid, dim3(256), 0, stream, p);
  }
}

}  // namespace

int64_t kv8_attention_workspace(const KvPool& c, const KvBatch& b, const KvQuery& q) {
  const Plan pl = plan(c, b, q);
  // more threads than a launch can have
  if (pl.blocks >= (int64_t{1} << 32) / 512 || (pl.splits > 1 && (int64_t)b.max_new * q.heads >= (int64_t{1} << 32) / 256))
    return -1;
  return pl.splits > 1 ? (int64_t)pl.splits * b.T * q.heads * (c.dim + 2) * 4 : 0;
}

void launch_kv8_attention(const KvPool& c, const KvBatch& b, const KvQuery& q, void* workspace, hipStream_t stream) {
  const Plan pl = plan(c, b, q);
  AttnParams p;
  p.c = c;
  p.b = b;
  p.q = q;
  p.group = q.heads / c.heads;
  p.group_magic = (unsigned)(((uint64_t{1} << 32) + p.group - 1) / p.group);
  p.tile_rows = pl.tile_rows;
  p.tiles = pl.tiles;
  p.splits = pl.splits;
  p.split = pl.split;
  p.part = static_cast<float*>(workspace);
  p.part_rows = (int64_t)b.T * q.heads;
  switch (c.dim) {
    case 64: launch_for<64>(p, pl, stream); return;
    case 128: launch_for<128>(p, pl, stream); return;
    case 192: launch_for<192>(p, pl, stream); return;
    default: launch_for<256>(p, pl, stream); return;
  }
}

}  // namespace w4a4
