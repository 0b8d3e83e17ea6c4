// Mixture of experts for gfx950: the router, and a layer of INT8 experts for few
// tokens.
//
// Router: per token the k largest logits, the lower index first among equals, and
//   w_j = exp(l_j - m) / sum exp(l - m)   (over all experts, or the k chosen).
//
// Layer: for each pair p = (token t, choice j) with expert e = ids[t][j]
//   g, u = rows 2i and 2i + 1 of  fl32(P) fl32(xs[t] s13[e]),  P = w13[e] xq[t]
//   h[p] = act(g) u                                   (fp32)
//   hq[p], hs[p] = INT8 codes and scale of h[p]       (the rule of quant8.h)
//   y[t] = sum_j weights[t][j] fl32(P') fl32(hs[p] s2[e]),  P' = w2[e] hq[p]
// with exact int32 sums P, P' and the sum over j in order, so results do not vary.
#include <algorithm>

#include "act8.h"
#include "device.h"
#include "launch.h"
#include "quant8.h"

namespace w4a4 {

namespace {

// ---- Router -----------------------------------------------------------------

// A wave's maximum, in every lane.
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t m) {
  m = dpp_max<DPP_HALF_MIRROR>(m);
  m = dpp_max<DPP_QUAD_1032>(m);
  m = dpp_max<DPP_QUAD_2301>(m);
  m = dpp_max<DPP_ROW_MIRROR>(m);
  const auto a = __builtin_amdgcn_permlane16_swap(m, m, false, false);
  m = max(a[0], a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(m, m, false, false);
  return max(b[0], b[1]);
}
__device__ __forceinline__ float wave_add(float v) {
  v += dpp<DPP_HALF_MIRROR>(v);
  v += dpp<DPP_QUAD_1032>(v);
  v += dpp<DPP_QUAD_2301>(v);
  v += dpp<DPP_ROW_MIRROR>(v);
  v += __shfl_xor(v, 16);
  v += __shfl_xor(v, 32);
  return v;
}

// Floats to integers of the same order, minus infinity (and what counts as it) to 0.
__device__ __forceinline__ uint32_t order_key(float v) {
  if (!(v > -__builtin_inff())) return 0;               // NaN too
  const uint32_t b = __float_as_uint(v + 0.0f);         // -0 as +0: they are equal
  return b ^ ((uint32_t)((int)b >> 31) | 0x80000000u);
}

// One wave per token, NL consecutive experts per lane. A choice takes the largest
// key, and of the lanes that hold it the lowest.
template <int DT, int NL>
__global__ __launch_bounds__(256) void k_moe_route(const void* __restrict__ logits, int64_t T, int E, int64_t ldl, int k,
                                                   int renorm, int32_t* __restrict__ ids, float* __restrict__ weights) {
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= T) return;                                   // whole waves
  uint32_t key[NL];
  float v[NL];
#pragma unroll
  for (int i = 0; i < NL; ++i) {
    const int e = lane * NL + i;
    v[i] = -__builtin_inff();
    if (e < E) {
      const int64_t at = t * ldl + e;
      if constexpr (DT == 0) v[i] = static_cast<const float*>(logits)[at];
      else if constexpr (DT == 1) v[i] = (float)static_cast<const _Float16*>(logits)[at];
      else v[i] = __uint_as_float((uint32_t)static_cast<const uint16_t*>(logits)[at] << 16);
      v[i] = v[i] > 3.402823466e38f ? 3.402823466e38f : v[i];
    }
    key[i] = order_key(v[i]);
  }
  auto best = [&]() {
    uint32_t m = key[0];
#pragma unroll
    for (int i = 1; i < NL; ++i) m = max(m, key[i]);
    return m;
  };
  uint32_t top = wave_max_u32(best());
  float vmax = 0.0f, total = 0.0f;
  if (top) {
    vmax = __uint_as_float(top & 0x80000000u ? top ^ 0x80000000u : ~top);
    if (!renorm) {
#pragma unroll
      for (int i = 0; i < NL; ++i) total += key[i] ? expf(v[i] - vmax) : 0.0f;
      total = wave_add(total);
    }
  }
  int my_id = -1;
  float my_w = 0.0f, chosen = 0.0f;
  for (int j = 0; j < k; ++j) {
    if (top) {                                          // else nothing is left: id -1, weight 0
      const uint32_t mine = best();
      const int from = __builtin_ctzll(__ballot(mine == top));
      int at = 0;
#pragma unroll
      for (int i = NL - 1; i >= 0; --i) at = key[i] == top ? i : at;
      at = __builtin_amdgcn_readlane(at, from);
      if (lane == from) {
#pragma unroll
        for (int i = 0; i < NL; ++i) key[i] = i == at ? 0 : key[i];
      }
      const float w = expf(__uint_as_float(top & 0x80000000u ? top ^ 0x80000000u : ~top) - vmax);
      chosen += w;
      if (lane == j) my_id = from * NL + at, my_w = w;
      if (j + 1 < k) top = wave_max_u32(best());
    }
  }
  if (lane < k) {
    const float d = renorm ? chosen : total;
    ids[t * k + lane] = my_id;
    weights[t * k + lane] = my_id < 0 ? 0.0f : my_w / d;
  }
}

// ---- Experts ----------------------------------------------------------------

struct MoeParams {
  const int8_t* a;        // UP: the tokens' codes [T][K]; DOWN: codes of h [P][K] (FUSED: not used)
  const float* sa;        // their scales
  const float* h;         // DOWN, FUSED: [P][K]
  const int32_t* ids;
  const float* weights;
  const int8_t* w;        // [E][N][K]
  const float* sw;        // [E][N]
  int T, k, P, E, K, N, act;
  float* h_out;           // UP: [P][N / 2]
  float* part;            // DOWN in shares: [P][N], a pair's part of its token's output
  void* y;                // DOWN
  int ydtype;
  int64_t ldy;
};

constexpr size_t kLds = 64 * 1024;

// Ints per row of sums: the four row groups of a wave on their own banks.
__host__ __device__ constexpr int sums_ld(int channels) { return channels + 4; }

__host__ __device__ constexpr int max_entries(int P, int E, int rows) { return (P < E ? P : E) + P / rows; }
__host__ __device__ constexpr int code_ld(int K, int span) { return (K + span - 1) / span * span + 16; }

// LDS: sums, ids, counts / first positions, entries, pairs by position and back.
inline size_t moe_lds(int P, int E, int rows, int channels) {
  return (size_t)P * sums_ld(channels) * 4 + P * 4 + E * 4 + (max_entries(P, E, rows) + 1) * 8 + ((P + 1) / 2) * 8 + 32;
}
constexpr int kFusedSpan = 512;    // a chunk of k_w8a8_moe with FUSED
inline size_t fused_lds(int P, int K, int span) { return (size_t)P * code_ld(K, span) + P * 4 + 16; }

// Another lane's value, 0 where there is none or the row is not in MASK.
template <int CTRL, int MASK>
__device__ __forceinline__ uint32_t dpp_from(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, MASK, 0xF, false);
}

// The INT8 codes of a row of fp32 values by one wave, and its scale.
__device__ __forceinline__ float quantize_row(const float* __restrict__ h, int K, int lane, int8_t* codes) {
  constexpr int KEEP = 2;                              // 1024-element pieces that stay in registers
  float v[KEEP][16];
  uint32_t top = 0;
  auto load = [&](float f[16], int k0) {
    const float4* src = reinterpret_cast<const float4*>(h + k0);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float4 q = k0 < K ? src[j] : float4{0, 0, 0, 0};
      f[4 * j] = q.x; f[4 * j + 1] = q.y; f[4 * j + 2] = q.z; f[4 * j + 3] = q.w;
    }
  };
  auto most = [&](const float f[16]) {
#pragma unroll
    for (int j = 0; j < 16; ++j) top = max(top, __float_as_uint(f[j]) & 0x7FFFFFFFu);
  };
#pragma unroll
  for (int i = 0; i < KEEP; ++i) load(v[i], 1024 * i + 16 * lane);
#pragma unroll
  for (int i = 0; i < KEEP; ++i) most(v[i]);
  for (int k0 = 1024 * KEEP + 16 * lane; k0 < K; k0 += 1024) {
    float f[16];
    load(f, k0);
    most(f);
  }
  top = wave_max_u32(top);
  const float s = __uint_as_float(top >= 0x7F800000u ? 0x7FC00000u : top) / 127.0f;
  const float k = scale_guard(s);
  const float sk = s * k;
  const float rs = s == 0.0f ? 0.0f : 1.0f / sk;
#pragma unroll
  for (int i = 0; i < KEEP; ++i) {
    const int k0 = 1024 * i + 16 * lane;
    if (k0 < K) *reinterpret_cast<uint4*>(codes + k0) = codes16f(v[i], k, sk, rs);
  }
  for (int k0 = 1024 * KEEP + 16 * lane; k0 < K; k0 += 1024) {
    float f[16];
    load(f, k0);
    *reinterpret_cast<uint4*>(codes + k0) = codes16f(f, k, sk, rs);
  }
  return s;
}

// A workgroup owns CN channels (UP: CN / 2 gates and their values) of every expert, or
// of a share of the experts that the tokens chose (blockIdx.y). It sorts the pairs
// by expert; an entry is up to ROWS rows of one expert, and the entries' chunks of
// four k-steps are dealt to the waves in contiguous runs of equal length, whatever
// experts they fall in. A wave streams its chunks, the next on its way, and adds an
// entry's int32 sums to those in LDS (exact in any order).
//
// The operands of v_mfma_i32_16x16x64_i8 want 16 rows in 16 neighbouring lanes; loaded
// so, a load touches 64 pieces of 16 bytes, and the cache serves about 0.65 of them a
// clock (counted: 54.5 million in 142 us on 256 CUs). Chunks are therefore loaded in
// whole runs of a row, 256 bytes for 16 lanes, and turned by LDS (64 tokens, 8 of 64
// experts of 4096 x 1376: 240 -> 213 us).
//
// HALF: blocks of 8 rows and 8 channels that use both halves of the instruction's 16, the
// upper ones for the next 64 of k: rows r and r + 8 hold the same token, columns c and
// c + 8 the same channel, so D[r][c] + D[r + 8][c + 8] is the sum: longer runs of a row.
//
// FUSED: h is quantized here, into LDS, by every workgroup.
//
// Bound by HBM, the rows' codes from L2 on top: 64 tokens, 8 of 64 experts of 4096 x 1376,
// 1.04 GB of weights: 207 us, 5.0 TB/s; 13 tokens, 4 of 32 of 3584 x 2368, 0.52 GB: 108 us,
// 4.8 TB/s; the first stage for one token and all 64 experts 123 us, 5.9 TB/s; one token, 8
// of 64 of 2048 x 1024, 50 MB: 18 us, of which 7 are two launches without any expert. Two
// chunks on their way instead of one, or 16 waves, were slower (212 -> 236 us, -> 234).
enum { UP = 0, DOWN = 1 };
template <int STAGE, bool HALF, int RT, int CB, int NW, bool FUSED>
__global__ __launch_bounds__(64 * NW) void k_w8a8_moe(MoeParams p) {
  constexpr int NT = 64 * NW, RB = HALF ? 8 : 16, CN = RB * CB, ROWS = RB * RT, LD = sums_ld(CN);
  constexpr int KS = HALF ? 128 : 64, SPAN = 4 * KS, ROW_LANES = SPAN / 16, ROWS_L = 64 / ROW_LANES;
  constexpr int D = FUSED ? 2 : 1;                                   // chunks on their way
  static_assert(kMoeMaxPairs <= NT && kMoeMaxExperts <= NT, "one a thread");
  extern __shared__ __align__(16) uint8_t lds[];
  __shared__ uint32_t wave_total[NW];
  __shared__ __align__(16) uint8_t stage[NW][4096];
  int* const sums = reinterpret_cast<int*>(lds);                     // [P][LD]
  int* const id_of = sums + p.P * LD;                                // [P]
  int* const first = id_of + p.P;                                    // [E] counts, then first positions
  int2* const entry = reinterpret_cast<int2*>(lds + ((p.P * (LD + 1) + p.E) * 4 + 7) / 8 * 8);
  uint16_t* const pair_of = reinterpret_cast<uint16_t*>(entry + max_entries(p.P, p.E, ROWS) + 1);
  uint16_t* const pos_of = pair_of + (p.P + 1) / 2 * 2;
  int8_t* const codes = reinterpret_cast<int8_t*>(lds) + ((reinterpret_cast<uint8_t*>(pos_of + p.P) - lds) + 15) / 16 * 16;
  const int cld = FUSED ? code_ld(p.K, SPAN) : 0;
  float* const hs = reinterpret_cast<float*>(codes + p.P * cld);     // [P], FUSED
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = lane & 15, g = lane >> 4;
  const int cr = HALF ? c & 7 : c, kl = (HALF ? 64 * (c >> 3) : 0) + 16 * g;
  const int n0 = (int)blockIdx.x * CN, rows_w = min(CN, p.N - n0);

  // The pairs by expert, one a thread (P <= kMoeMaxPairs <= NT, E <= kMoeMaxExperts <= NT).
  int my_id = tid < p.P ? p.ids[tid] : -1, my_rank = 0;
  my_id = my_id >= 0 && my_id < p.E ? my_id : -1;
  for (int i = tid; i < p.E; i += NT) first[i] = 0;
  for (int i = tid; i < p.P * LD; i += NT) sums[i] = 0;
  __syncthreads();
  if (tid < p.P) id_of[tid] = my_id;
  if (my_id >= 0) my_rank = atomicAdd(&first[my_id], 1);
  __syncthreads();
  const int count = tid < p.E ? first[tid] : 0;
  const uint32_t own = (uint32_t)((count + ROWS - 1) / ROWS) << 16 | (uint32_t)count;
  uint32_t upto = own;                                               // entries << 16 | positions, up to this expert
  upto += dpp_from<0x111, 0xF>(upto);                                // row_shr:1, 2, 4, 8: sums within rows of 16
  upto += dpp_from<0x112, 0xF>(upto);
  upto += dpp_from<0x114, 0xF>(upto);
  upto += dpp_from<0x118, 0xF>(upto);
  upto += dpp_from<0x142, 0xA>(upto);                                // row_bcast:15 into rows 1 and 3
  upto += dpp_from<0x143, 0xC>(upto);                                // row_bcast:31 into rows 2 and 3
  if (lane == 63) wave_total[wave] = upto;
  __syncthreads();
  uint32_t all = 0, before = upto - own;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    if (w < wave) before += wave_total[w];
    all += wave_total[w];
  }
  if (tid < p.E) {
    first[tid] = (int)(before & 0xFFFFu);
    for (int i = 0; ROWS * i < count; ++i)
      entry[(before >> 16) + i] = int2{tid | min(ROWS, count - ROWS * i) << 16, (int)(before & 0xFFFFu) + ROWS * i};
  }
  const int entries = __builtin_amdgcn_readfirstlane((int)(all >> 16)), positions = (int)(all & 0xFFFFu);
  if (tid == 0) entry[entries] = int2{0, positions};
  __syncthreads();
  if (my_id >= 0) {
    const int pos = first[my_id] + my_rank;
    pair_of[pos] = (uint16_t)tid;
    pos_of[tid] = (uint16_t)pos;
  }
  __syncthreads();

  // This workgroup's entries, this wave's chunks.
  const int shares = gridDim.y, share = blockIdx.y;
  // A share holds whole experts: workgroups may differ in the order of an expert's rows.
  auto whole = [&](int e) {
    while (e > 0 && e < entries && (entry[e].x & 0xFFFF) == (entry[e - 1].x & 0xFFFF)) ++e;
    return __builtin_amdgcn_readfirstlane(e);
  };
  const int ent0 = whole(entries * share / shares), ent1 = whole(entries * (share + 1) / shares);
  const int nch = (p.K + SPAN - 1) / SPAN;
  const int chunks = (ent1 - ent0) * nch;
  const int ch0 = (int)((int64_t)chunks * wave / NW), ch1 = (int)((int64_t)chunks * (wave + 1) / NW);
  // A block is RB rows of SPAN bytes: 4 loads, of which each covers whole rows (a lane's
  // address in its place of the block: row ROWS_L j + lr, 16-byte piece lp).
  struct Buf {
    v4i w[CB][4];
    v4i a[FUSED ? 1 : RT][4];
  };
  const int lr = lane / ROW_LANES, lp = lane % ROW_LANES;
  // rows of an entry that this lane supplies (dropped ones past its end)
  auto entry_at = [&](int e) {
    const int2 v = entry[e];
    return int2{__builtin_amdgcn_readfirstlane(v.x), __builtin_amdgcn_readfirstlane(v.y)};
  };
  const __amdgpu_buffer_rsrc_t rA = buffer_rsrc(p.a, FUSED ? 0 : (STAGE == UP ? p.T : p.P) * p.K);
  int l_ent = ent0 + (chunks ? ch0 / nch : 0), l_ch = chunks ? ch0 % nch : 0, l_at = ch0;
  __amdgpu_buffer_rsrc_t rW = buffer_rsrc(p.w, 0);
  int off_a[FUSED ? 1 : RT][4], l_n = 0;
  auto enter_load = [&]() {
    const int2 v = entry_at(l_ent);
    const int e = v.x & 0xFFFF, n = v.x >> 16;
    l_n = n;
    rW = buffer_rsrc(p.w + ((int64_t)e * p.N + n0) * p.K, rows_w * p.K);
    if constexpr (!FUSED) {
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int row = RB * r + ROWS_L * j + lr;
          const int pair = pair_of[v.y + min(row, n - 1)];
          off_a[r][j] = row < n ? (STAGE == UP ? pair / p.k : pair) * p.K + 16 * lp : kDroppedOffset;
        }
    }
  };
#pragma unroll
  for (int r = 0; r < (FUSED ? 1 : RT); ++r)
#pragma unroll
    for (int j = 0; j < 4; ++j) off_a[r][j] = kDroppedOffset;
  if (ch0 < ch1) enter_load();
  auto fetch = [&](Buf& b) {
    if (l_at < ch1 && l_ch == nch) {
      l_ch = 0;
      ++l_ent;
      enter_load();
    }
    const int k0 = SPAN * l_ch;
    const int out = l_at < ch1 && k0 + 16 * lp < p.K ? 0 : kDroppedOffset;
#pragma unroll
    for (int cb = 0; cb < CB; ++cb)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        b.w[cb][j] = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(
            rW, ((RB * cb + ROWS_L * j + lr) * p.K + 16 * lp) | out, k0, 0));
    if constexpr (!FUSED) {
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        if (r > 0 && l_n <= RB * r) break;             // a block of rows that the entry does not have
#pragma unroll
        for (int j = 0; j < 4; ++j)
          b.a[r][j] = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(rA, off_a[r][j] | out, k0, 0));
      }
    }
    ++l_ch;
    ++l_at;
  };
  // A block into operands: lane (c, g) of k-step u takes row cr at KS u + kl. Pieces are
  // swizzled by their row, so that 16 lanes meet 16 bank groups both ways. The region is
  // the wave's own, whose LDS operations complete in order.
  int put[4], take[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    auto place = [](int row, int piece) {
      return row * SPAN + 16 * (piece ^ (HALF ? (row & 3) | (row & 4) << 1 : row));
    };
    put[j] = place(ROWS_L * j + lr, lp);
    take[j] = place(cr, (KS * j + kl) / 16);
  }
  uint8_t* const mine = stage[wave];
  auto operands = [&](const v4i raw[4], v4i op[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) *reinterpret_cast<v4i*>(mine + put[j]) = raw[j];
    asm volatile("" ::: "memory");
#pragma unroll
    for (int u = 0; u < 4; ++u) op[u] = *reinterpret_cast<const v4i*>(mine + take[u]);
    asm volatile("" ::: "memory");
  };
  Buf b[D];
#pragma unroll
  for (int d = 0; d < D; ++d) fetch(b[d]);

  if constexpr (FUSED) {
    for (int i = wave; i < p.P; i += NW) {
      if (__builtin_amdgcn_readfirstlane(id_of[i]) < 0) continue;
      const float s = quantize_row(p.h + (int64_t)i * p.K, p.K, lane, codes + i * cld);
      if (lane == 0) hs[i] = s;
    }
    __syncthreads();
  }

  int c_ent = l_ent, c_ch = chunks ? ch0 % nch : 0, c_n = 0, c_pos = 0;
  if (ch0 < ch1) c_ent = ent0 + ch0 / nch;
  const int8_t* row_a[RT];
  v4i acc[RT][CB];
  auto enter = [&]() {
    const int2 v = entry_at(c_ent);
    c_n = v.x >> 16;
    c_pos = v.y;
#pragma unroll
    for (int r = 0; r < RT; ++r) {
#pragma unroll
      for (int cb = 0; cb < CB; ++cb) acc[r][cb] = v4i{0, 0, 0, 0};
      if constexpr (FUSED) row_a[r] = codes + pair_of[c_pos + min(RB * r + cr, c_n - 1)] * cld + kl;
    }
  };
  auto consume = [&](const Buf& b) {
    v4i w[CB][4];
#pragma unroll
    for (int cb = 0; cb < CB; ++cb) operands(b.w[cb], w[cb]);
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      if (RB * r >= c_n) break;
      v4i a[4];
      if constexpr (FUSED) {
#pragma unroll
        for (int u = 0; u < 4; ++u) a[u] = *reinterpret_cast<const v4i*>(row_a[r] + SPAN * c_ch + KS * u);
      } else {
        operands(b.a[r], a);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int cb = 0; cb < CB; ++cb)
          acc[r][cb] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[u], w[cb][u], acc[r][cb], 0, 0, 0);
    }
    if (++c_ch == nch) {
      c_ch = 0;
      return true;
    }
    return false;
  };
  auto flush = [&]() {
#pragma unroll
    for (int r = 0; r < RT; ++r) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = RB * r + 4 * (HALF ? g & 1 : g) + i;
#pragma unroll
        for (int cb = 0; cb < CB; ++cb)
          if (row < c_n && (!HALF || c >> 3 == g >> 1)) atomicAdd(&sums[(c_pos + row) * LD + RB * cb + cr], acc[r][cb][i]);
      }
    }
  };
  if (ch0 < ch1) enter();
  for (int at = ch0; at < ch1;) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      const bool done = consume(b[d]);
      fetch(b[d]);
      ++at;
      if (done || at >= ch1) {
        flush();
        if (at >= ch1) break;
        ++c_ent;
        enter();
      }
    }
  }
  __syncthreads();

  if constexpr (STAGE == UP) {
    const int pos0 = entry[ent0].y, pos1 = entry[ent1].y, I = p.N >> 1;
    for (int o = tid; o < (pos1 - pos0) * (CN / 2); o += NT) {
      const int pos = pos0 + o / (CN / 2), i = o % (CN / 2);
      if (2 * i >= rows_w) continue;
      const int pair = pair_of[pos];
      const float sa = p.sa[pair / p.k];
      const float* sw = p.sw + (int64_t)id_of[pair] * p.N + n0 + 2 * i;
      const float gate = (float)sums[pos * LD + 2 * i] * (sa * sw[0]);
      const float up = (float)sums[pos * LD + 2 * i + 1] * (sa * sw[1]);
      p.h_out[(int64_t)pair * I + (n0 >> 1) + i] = activate(p.act, gate) * up;
    }
  } else {
    // Every pair's part of the output in place of its sums, all loads at once; then
    // the parts of a token in the order of its choices, by k_moe_join where they come
    // from several shares.
    constexpr int AT_ONCE = 4;
    const bool alone = FUSED || shares == 1;             // FUSED has one share
    const int at0 = alone ? 0 : entry[ent0].y * CN, at1 = alone ? positions * CN : entry[ent1].y * CN;
    for (int o = at0 + tid; o < at1; o += AT_ONCE * NT) {
      float f[AT_ONCE], s[AT_ONCE];
#pragma unroll
      for (int i = 0; i < AT_ONCE; ++i) {
        const int at = min(o + i * NT, at1 - 1), pair = pair_of[at / CN];
        s[i] = (FUSED ? hs[pair] : p.sa[pair]) * p.sw[(int64_t)id_of[pair] * p.N + min(n0 + at % CN, p.N - 1)];
        f[i] = p.weights[pair];
      }
#pragma unroll
      for (int i = 0; i < AT_ONCE; ++i) {
        const int at = o + i * NT;
        if (at < at1) {
          int* const v = sums + at / CN * LD + at % CN;
          const float part = f[i] * ((float)*v * s[i]);
          if (alone) *v = __float_as_int(part);
          else if (at % CN < rows_w) p.part[(int64_t)pair_of[at / CN] * p.N + n0 + at % CN] = part;
        }
      }
    }
    if (!alone) return;
    __syncthreads();
    for (int o = tid; o < p.T * CN; o += NT) {
      const int t = o / CN, n = o % CN;
      if (n >= rows_w) continue;
      float sum = 0.0f;
      for (int j = 0; j < p.k; ++j) {
        const int pair = t * p.k + j;
        if (id_of[pair] >= 0) sum += __int_as_float(sums[pos_of[pair] * LD + n]);
      }
      const int64_t at = t * p.ldy + n0 + n;
      if (p.ydtype == 1) static_cast<_Float16*>(p.y)[at] = (_Float16)sum;
      else static_cast<__bf16*>(p.y)[at] = (__bf16)sum;
    }
  }
}

// The parts of a token's output, in the order of its choices: a thread a column.
__global__ __launch_bounds__(256) void k_moe_join(MoeParams p) {
  const int n = (int)blockIdx.x * 256 + (int)threadIdx.x, t = blockIdx.y;
  if (n >= p.N) return;
  float sum = 0.0f;
  for (int j = 0; j < p.k; ++j) {
    const int pair = t * p.k + j, id = p.ids[pair];
    if (id >= 0 && id < p.E) sum += p.part[(int64_t)pair * p.N + n];
  }
  const int64_t at = t * p.ldy + n;
  if (p.ydtype == 1) static_cast<_Float16*>(p.y)[at] = (_Float16)sum;
  else static_cast<__bf16*>(p.y)[at] = (__bf16)sum;
}

// The codes of h for k_w8a8_moe without FUSED, one wave a pair. Pairs without an
// expert have no h.
__global__ __launch_bounds__(256) void k_moe_quant(const float* __restrict__ h, const int32_t* __restrict__ ids, int E,
                                                   int P, int K, int8_t* __restrict__ codes, float* __restrict__ s) {
  const int i = __builtin_amdgcn_readfirstlane((int)blockIdx.x * 4 + ((int)threadIdx.x >> 6)), lane = threadIdx.x & 63;
  if (i >= P || ids[i] < 0 || ids[i] >= E) return;
  const float v = quantize_row(h + (int64_t)i * K, K, lane, codes + (int64_t)i * K);
  if (lane == 0) s[i] = v;
}

int64_t align256(int64_t n) { return (n + 255) & ~int64_t{255}; }

// Stage 0 (UP) or 1 (DOWN) of a layer whose experts have few rows, or more.
template <int STAGE, bool FUSED>
void launch_stage(const MoeParams& p, int shares, bool few_rows, hipStream_t stream) {
#define MOE_STAGE(HALF, RT, CB)                                                                                        \
  {                                                                                                                    \
    constexpr int RB = HALF ? 8 : 16;                                                                                  \
    const dim3 grid((unsigned)((p.N + RB * CB - 1) / (RB * CB)), (unsigned)shares);                                    \
    const size_t lds = moe_lds(p.P, p.E, RB * RT, RB * CB) + (FUSED ? fused_lds(p.P, p.K, kFusedSpan) : 0);            \
    hipLaunchKernelGGL((k_w8a8_moe<STAGE, HALF, RT, CB, 8, FUSED>), grid, dim3(512), (unsigned)lds, stream, p);        \
    return;                                                                                                            \
  }
  if constexpr (FUSED) {
    MOE_STAGE(true, 1, 1)
  } else {
    if (few_rows) MOE_STAGE(STAGE == DOWN, 1, (STAGE == UP ? 1 : 2))
    MOE_STAGE(false, 2, 1)
  }
#undef MOE_STAGE
}

// How a layer is run, from its extents (times in us; sizes T, H, I, E, k).
struct MoePlan {
  // Entries of 16 rows (second stage: 8 rows, two blocks of 8 channels) where an expert
  // has few, of 32 rows where it has more (one and the other in the second stage: 16,
  // 2048, 1024, 64, 8 65.1 and 69.2; 16, 4096, 1376, 64, 8 142 and 151; 13, 3584, 2368, 32, 4
  // 111 and 114; 64, 2048, 1024, 64, 8 126 and 123; 64, 4096, 1376, 64, 8 271 and 262; in the
  // first stage 2 either way).
  bool few_rows;
  // Every workgroup of the second stage quantizes h itself up to 16384 values; above, a
  // launch does (T, I, k with H = 2048: 1, 1024, 8 19.1 in two launches, 21 in three;
  // 16, 1024, 2 21.2 and 20.5; 4, 1024, 8 41.1 and 40.3).
  bool fused;
  // Shares of the experts in the first stage, so that a workgroup streams some 128 KiB
  // of weights: enough of them to fill the chip with few experts, and to end evenly with
  // many (1, 2048, 1024, 64, 8: both stages 20.6 with 256 workgroups, 21.3 with 1024; 13,
  // 3584, 2368, 32, 4: 145 with 296, 115 with 2072); at least about 256 workgroups (with
  // those of 128 KiB alone 21, 560, 192, 32, 4 26.6, now 24.0; 2, 688, 144, 64, 6 15.0 and 12.9;
  // 11, 1952, 160, 60, 1 16.9 and 13.8).
  int up;
  // Shares in the second stage where its channels fill at most 128 workgroups and it
  // reads 8 MB or more: up to 512 of them, each with 96 KiB or more, and a launch that
  // joins their parts (one share and several: 64, 2048, 1408, 64, 6 129.5 and 115.0; 51,
  // 1040, 736, 60, 8 66.8 and 53.9; 39, 528, 1136, 32, 4 38.8 and 30.7; they cost elsewhere:
  // 64, 4096, 1376, 64, 8 212.8 and 220.6; 16, 2880, 1024, 32, 4 58.2 and 61.2; 1, 448, 2848, 60,
  // 6 21.5 and 22.6).
  int down;
};
MoePlan plan_moe(int64_t T, int64_t k, int64_t E, int64_t H, int64_t I) {
  MoePlan m;
  const int64_t P = T * k, used = std::min(P, E), columns = H / 16;
  m.few_rows = T <= 8 || P <= 4 * E;
  m.fused = m.few_rows && P * I <= 16384 && moe_lds((int)P, (int)E, 8, 8) + fused_lds((int)P, (int)I, kFusedSpan) <= kLds;
  const int64_t target = std::clamp<int64_t>(used * 2 * I * H >> 17, 256, 2048);
  m.up = (int)std::max<int64_t>(1, std::min(used, target * 16 / (2 * I)));
  m.down = 1;
  if (!m.fused && columns <= 128 && used * H * I >= 8000000)
    m.down = (int)std::max<int64_t>(1, std::min({used, 512 / columns, used * 16 * I / 98304}));
  return m;
}

}  // namespace

void launch_moe_route(const void* logits, int dtype, int64_t T, int64_t E, int64_t ldl, int k, bool renorm,
                      int32_t* ids, float* weights, hipStream_t stream) {
  const dim3 grid((unsigned)((T + 3) / 4)), block(256);
#define MOE_ROUTE(DT, NL) \
  hipLaunchKernelGGL((k_moe_route<DT, NL>), grid, block, 0, stream, logits, T, (int)E, ldl, k, (int)renorm, ids, weights)
#define MOE_ROUTE_E(DT)                   \
  if (E <= 64) MOE_ROUTE(DT, 1);          \
  else if (E <= 128) MOE_ROUTE(DT, 2);    \
  else if (E <= 256) MOE_ROUTE(DT, 4);    \
  else MOE_ROUTE(DT, 8)
  if (dtype == 0) { MOE_ROUTE_E(0); }
  else if (dtype == 1) { MOE_ROUTE_E(1); }
  else { MOE_ROUTE_E(2); }
#undef MOE_ROUTE_E
#undef MOE_ROUTE
}

int64_t moe_workspace(int64_t T, int64_t k, int64_t E, int64_t H, int64_t I) {
  const int64_t P = T * k;
  return align256(4 * P * I) + align256(P * I) + align256(4 * P) + (plan_moe(T, k, E, H, I).down > 1 ? 4 * P * H : 0);
}

void launch_w8a8_moe(const MoeArgs& a, hipStream_t stream) {
  const int P = a.T * a.k;
  float* const h = static_cast<float*>(a.workspace);
  int8_t* const codes = static_cast<int8_t*>(a.workspace) + align256(4 * (int64_t)P * a.I);
  float* const hs = reinterpret_cast<float*>(codes + align256((int64_t)P * a.I));
  MoeParams p = {};
  p.part = reinterpret_cast<float*>(reinterpret_cast<int8_t*>(hs) + align256(4 * (int64_t)P));
  p.ids = a.ids;
  p.weights = a.weights;
  p.T = a.T; p.k = a.k; p.P = P; p.E = a.E;
  p.act = a.act;
  const MoePlan m = plan_moe(a.T, a.k, a.E, a.H, a.I);

  p.a = a.xq; p.sa = a.xs;
  p.w = a.w13; p.sw = a.s13;
  p.K = a.H; p.N = 2 * a.I;
  p.h_out = h;
  launch_stage<UP, false>(p, m.up, m.few_rows, stream);

  p.K = a.I; p.N = a.H;
  p.w = a.w2; p.sw = a.s2;
  p.y = a.y; p.ydtype = a.ydtype; p.ldy = a.ldy;
  if (m.fused) {
    p.h = h;
    launch_stage<DOWN, true>(p, 1, true, stream);
    return;
  }
  hipLaunchKernelGGL(k_moe_quant, dim3((unsigned)((P + 3) / 4)), dim3(256), 0, stream, h, a.ids, a.E, P, a.I, codes, hs);
  p.a = codes; p.sa = hs;
  launch_stage<DOWN, false>(p, m.down, m.few_rows, stream);
  if (m.down > 1)
    hipLaunchKernelGGL(k_moe_join, dim3((unsigned)((p.N + 255) / 256), (unsigned)a.T), dim3(256), 0, stream, p);
}

}  // namespace w4a4
