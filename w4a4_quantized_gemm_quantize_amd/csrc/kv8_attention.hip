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
// p_j vs_j enter the second product as fp16(2^15 p_j vs_j / vref), p_j <= 1
// and vref the largest page scale seen so far: a relative rounding of 2^-12
// for weights within 2^-29 of the largest one, below that an absolute one of
// 2^-40 vref.
//
// Layout. S^T = K Q^T and O^T = V^T P^T with v_mfma_f32_16x16x32_f16: the rows
// of the first product are 64 positions in four tiles, row 4 g + i of tile t
// being position 16 g + 4 t + i (g = lane / 16), so a lane ends up with the
// scores of 16 consecutive positions (of one page) of query row lane % 16.
// Those are the k indices that the second product wants in that lane: the
// weights go from one product's result to the other's operand without
// leaving their lane, and V^T's rows are read as 16 consecutive bytes.
#include <algorithm>

#include "kv8_common.h"

namespace w4a4 {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNone = -3.0e38f;          // running maximum of a row that has seen nothing
constexpr float kTinyScale = 0x1p-120f;

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
  int split;             // positions per split (a multiple of 64 times the waves)
  float* part;           // splits' results: [splits][T heads][dim] then [splits][T heads][2]
  int64_t part_rows;     // T heads
};

// Positions a tile of query rows [r0, r1) of a sequence can see: [lo, hi), lo a
// multiple of 64.
struct Range {
  int lo, hi;
};
__device__ __forceinline__ Range tile_range(const AttnParams& p, const Seq& s, int r0, int r1) {
  const int p0 = s.len - s.n;
  Range r{0, s.len};
  if (p.q.causal) r.hi = min(s.len, p0 + (r1 - 1) / p.group + 1);
  if (p.q.window > 0) r.lo = max(0, p0 + r0 / p.group - p.q.window + 1) & ~63;
  r.hi = max(r.hi, r.lo);
  return r;
}

// Few query rows per kv head: a workgroup of NW waves takes 16 rows (token,
// query head of the group) of one kv head and a split of the positions; its
// waves take chunks of 64 positions in turn, with no sharing until the end.
template <int D, int NW>
__global__ __launch_bounds__(64 * NW) void k_kv8_decode(AttnParams p) {
  constexpr int DB = D / 64, DT = D / 16;
  __shared__ float lo_[NW][16][D + 4];
  __shared__ float lm[NW][16], ll[NW][16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = lane & 15, g = lane >> 4;
  const int seq = blockIdx.z;
  const int h = blockIdx.x % p.c.heads, tile = blockIdx.x / p.c.heads;
  const Seq s = sequence(p.b, seq);
  const int rows = s.n * p.group;
  const int r0 = tile * 16;
  if (r0 >= rows) return;
  const Range rg = tile_range(p, s, r0, min(r0 + 16, rows));
  const int nsplit = max(1, (rg.hi - rg.lo + p.split - 1) / p.split);
  if ((int)blockIdx.y >= nsplit) return;
  const int from = rg.lo + blockIdx.y * p.split, to = min(rg.hi, from + p.split);

  // query row of this lane's column
  const int r = min(r0 + c, rows - 1);
  const int tok = r / p.group, hq = h * p.group + r % p.group;
  const int pos = s.len - s.n + tok;
  const int row_hi = p.q.causal ? min(s.len, pos + 1) : s.len;
  const int row_lo = p.q.window > 0 ? max(0, pos - p.q.window + 1) : 0;
  v8h qf[DB][2];
  float qscale = p.q.scale * kLog2e;
  {
    const uint16_t* qp = static_cast<const uint16_t*>(p.q.q) + (int64_t)(s.t0 + tok) * p.q.q_tok + hq * p.q.q_head;
    uint4 raw[DB][2];
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int u = 0; u < 2; ++u) raw[d][u] = *reinterpret_cast<const uint4*>(qp + 64 * d + 16 * g + 8 * u);
    if (!p.q.bf16) {
#pragma unroll
      for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int u = 0; u < 2; ++u) qf[d][u] = __builtin_bit_cast(v8h, raw[d][u]);
    } else {
      uint32_t m = 0;
#pragma unroll
      for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint32_t w[4] = {raw[d][u].x, raw[d][u].y, raw[d][u].z, raw[d][u].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) m = max(m, max((w[i] & 0x7FFFu) << 16, w[i] & 0x7FFF0000u));
        }
      m = max(m, (uint32_t)__shfl_xor((int)m, 16));
      m = max(m, (uint32_t)__shfl_xor((int)m, 32));
      // exponent of the largest element to 14; a row of zeros and subnormals stays as it is
      const int e = (int)(m >> 23), up = min(max(127 + 14 + 127 - e, 1), 254);
      const float mul = e == 0 ? 1.0f : __uint_as_float((uint32_t)up << 23);
      qscale = qscale / mul;
#pragma unroll
      for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint32_t w[4] = {raw[d][u].x, raw[d][u].y, raw[d][u].z, raw[d][u].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            qf[d][u][2 * i] = (_Float16)(__uint_as_float(w[i] << 16) * mul);
            qf[d][u][2 * i + 1] = (_Float16)(__uint_as_float(w[i] & 0xFFFF0000u) * mul);
          }
        }
    }
  }

  const int P = p.c.page;
  v4f acc[DT];
#pragma unroll
  for (int i = 0; i < DT; ++i) acc[i] = v4f{0, 0, 0, 0};
  float m = kNone, l = 0.0f, vref = kTinyScale;

  for (int at = from + 64 * wave; at < to; at += 64 * NW) {
    // this lane's page as a reader of K rows (positions 16 (c / 4) ..) and as
    // the owner of scores and V columns (positions 16 g ..)
    const int pk = at + 16 * (c >> 2), pv = at + 16 * g;
    const int gk = pk < to ? page_of(p.b, p.c, seq, pk) : -1;
    const int gv = pv < to ? page_of(p.b, p.c, seq, pv) : -1;
    const int8_t* kp = p.c.k + ((int64_t)max(gk, 0) * p.c.heads + h) * P * D + (int64_t)(pk & (P - 1)) * D;
    const int8_t* vp = p.c.v + ((int64_t)max(gv, 0) * p.c.heads + h) * P * D + (pv & (P - 1));
    const float ks = gv < 0 ? 0.0f : p.c.ks[(int64_t)gv * p.c.heads + h];
    const float vs = gv < 0 ? 0.0f : p.c.vs[(int64_t)gv * p.c.heads + h];
    uint4 kr[4][DB];
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int d = 0; d < DB; ++d)
        kr[t][d] = *reinterpret_cast<const uint4*>(kp + (4 * t + (c & 3)) * D + 64 * d + 16 * g);
    uint4 vr[DT];
#pragma unroll
    for (int i = 0; i < DT; ++i) vr[i] = *reinterpret_cast<const uint4*>(vp + (16 * i + c) * P);

    v4f sc[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      sc[t] = v4f{0, 0, 0, 0};
#pragma unroll
      for (int d = 0; d < DB; ++d) {
        sc[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(widen8(kr[t][d].x, kr[t][d].y), qf[d][0], sc[t], 0, 0, 0);
        sc[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(widen8(kr[t][d].z, kr[t][d].w), qf[d][1], sc[t], 0, 0, 0);
      }
    }
    const float f = ks * qscale;
    const int first = pv, lim = gv < 0 ? 0 : row_hi;
    float cm = kNone;
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int j = first + 4 * t + i;
        sc[t][i] = j >= row_lo && j < lim ? sc[t][i] * f : -INFINITY;
        cm = fmaxf(cm, sc[t][i]);
      }
    cm = fmaxf(cm, __shfl_xor(cm, 16));
    cm = fmaxf(cm, __shfl_xor(cm, 32));
    float vm = fmaxf(vs, __shfl_xor(vs, 16));
    vm = fmaxf(vm, __shfl_xor(vm, 32));
    const float m2 = fmaxf(m, cm), vref2 = fmaxf(vref, vm);
    const float al = __builtin_amdgcn_exp2f(m - m2);
    const float ao = al * (vref / vref2);
    const float w = vs / vref2 * 32768.0f;
    l *= al;
    v8h pf[2];
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float e = __builtin_amdgcn_exp2f(sc[t][i] - m2);
        l += e;
        pf[t >> 1][4 * (t & 1) + i] = (_Float16)(e * w);
      }
    m = m2;
    vref = vref2;
#pragma unroll
    for (int i = 0; i < DT; ++i) {
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[i][k] *= ao;
      acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(widen8(vr[i].x, vr[i].y), pf[0], acc[i], 0, 0, 0);
      acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(widen8(vr[i].z, vr[i].w), pf[1], acc[i], 0, 0, 0);
    }
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
  __syncthreads();
  for (int i = threadIdx.x; i < 16 * D; i += 64 * NW) {
    const int rr = i / D, d = i % D;
    if (r0 + rr >= rows) continue;
    float M = kNone;
#pragma unroll
    for (int w = 0; w < NW; ++w) M = fmaxf(M, lm[w][rr]);
    float L = 0.0f, o = 0.0f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float e = __builtin_amdgcn_exp2f(lm[w][rr] - M);
      L += ll[w][rr] * e;
      o += lo_[w][rr][d] * e;
    }
    const int64_t t = s.t0 + (r0 + rr) / p.group;
    const int head = h * p.group + (r0 + rr) % p.group;
    if (nsplit == 1) {
      store_as(p.q.y, p.q.ydtype, (t * p.q.heads + head) * D + d, L == 0.0f ? 0.0f : o / L);
      if (p.q.lse && d == 0) p.q.lse[t * p.q.heads + head] = L == 0.0f ? -INFINITY : (M + __builtin_amdgcn_logf(L)) / kLog2e;
    } else {
      const int64_t row = blockIdx.y * p.part_rows + t * p.q.heads + head;
      p.part[row * D + d] = o;
      if (d == 0) {
        float* ml = p.part + (int64_t)gridDim.y * p.part_rows * D + 2 * row;
        ml[0] = M;
        ml[1] = L;
      }
    }
  }
}

// Joins the splits of a query row: one wave per row, lanes over the dimensions.
template <int D>
__global__ __launch_bounds__(256) void k_kv8_join(AttnParams p, int splits) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int seq = blockIdx.z;
  const Seq s = sequence(p.b, seq);
  const int rows = s.n * p.group;                   // of one kv head
  const int x = blockIdx.x * 4 + wave;
  const int h = x % p.c.heads, r = x / p.c.heads;
  if (r >= rows) return;
  const Range rg = tile_range(p, s, r & ~15, min((r & ~15) + 16, rows));
  const int nsplit = (rg.hi - rg.lo + p.split - 1) / p.split;
  if (nsplit <= 1) return;
  const int64_t t = s.t0 + r / p.group;
  const int head = h * p.group + r % p.group;
  const int64_t row = t * p.q.heads + head;
  const float* ml = p.part + (int64_t)splits * p.part_rows * D;
  float M = kNone;
  for (int i = 0; i < nsplit; ++i) M = fmaxf(M, ml[2 * (i * p.part_rows + row)]);
  float L = 0.0f, o[D / 64];
#pragma unroll
  for (int d = 0; d < D / 64; ++d) o[d] = 0.0f;
  for (int i = 0; i < nsplit; ++i) {
    const int64_t at = i * p.part_rows + row;
    const float e = __builtin_amdgcn_exp2f(ml[2 * at] - M);
    L += ml[2 * at + 1] * e;
#pragma unroll
    for (int d = 0; d < D / 64; ++d) o[d] += p.part[at * D + 64 * d + lane] * e;
  }
#pragma unroll
  for (int d = 0; d < D / 64; ++d)
    store_as(p.q.y, p.q.ydtype, row * D + 64 * d + lane, L == 0.0f ? 0.0f : o[d] / L);
  if (p.q.lse && lane == 0) p.q.lse[row] = L == 0.0f ? -INFINITY : (M + __builtin_amdgcn_logf(L)) / kLog2e;
}

constexpr int kWaves = 4;

// Positions a query row tile can see at most, and how they are split: enough
// workgroups to fill the chip, splits of at least 64 positions per wave.
struct Plan {
  int tiles, split, splits;
};
Plan plan(const KvPool& c, const KvBatch& b, const KvQuery& q) {
  Plan pl;
  const int group = q.heads / c.heads;
  pl.tiles = (int)(((int64_t)b.max_new * group + 15) / 16);
  int64_t span = b.max_len;
  if (q.window > 0) span = std::min<int64_t>(span, (int64_t)q.window + (q.causal ? 15 / group + 1 : b.max_len) + 64);
  const int64_t work = (int64_t)pl.tiles * c.heads * b.B;
  const int64_t unit = 64 * kWaves;
  const int64_t want = std::max<int64_t>(1, 1024 / std::max<int64_t>(work, 1));
  int64_t units = (span + unit - 1) / unit;
  const int64_t per = std::max<int64_t>(1, (units + want - 1) / want);
  pl.split = (int)(per * unit);
  pl.splits = (int)std::max<int64_t>(1, (span + pl.split - 1) / pl.split);
  return pl;
}

template <int D>
void launch_for(AttnParams p, const Plan& pl, hipStream_t stream) {
  const dim3 grid((unsigned)(pl.tiles * p.c.heads), (unsigned)pl.splits, (unsigned)p.b.B);
  hipLaunchKernelGGL((k_kv8_decode<D, kWaves>), grid, dim3(64 * kWaves), 0, stream, p);
  if (pl.splits > 1) {
    const int64_t rows = (int64_t)p.b.max_new * p.q.heads;
    hipLaunchKernelGGL((k_kv8_join<D>), dim3((unsigned)((rows + 3) / 4), 1, (unsigned)p.b.B), dim3(256), 0, stream, p,
                       pl.splits);
  }
}

}  // namespace

int64_t kv8_attention_workspace(const KvPool& c, const KvBatch& b, const KvQuery& q) {
  const Plan pl = plan(c, b, q);
  return pl.splits > 1 ? (int64_t)pl.splits * b.T * q.heads * (c.dim + 2) * 4 : 0;
}

void launch_kv8_attention(const KvPool& c, const KvBatch& b, const KvQuery& q, void* workspace, hipStream_t stream) {
  const Plan pl = plan(c, b, q);
  AttnParams p;
  p.c = c;
  p.b = b;
  p.q = q;
  p.group = q.heads / c.heads;
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
