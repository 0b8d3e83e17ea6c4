// W8A8 linear layers for gfx950: INT8 quantization with one scale per token
// (weights: per output channel), and the matrix product on the INT8 matrix
// cores.
//
//   a = max_k |x|, s = fl32(a / 127), q = rne(fl32(x / s)) in [-127, 127]
//   (s = NaN, and with it the row of Y, if an x is a NaN or an infinity)
//   P[m,n] = sum_k xq[m,k] wq[n,k]            (int32, exact for K <= 131056)
//   Y[m,n] = fl32(fl32(fl32(P) fl32(xs[m] ws[n])) + bias[n])
//
// The scales do not vary along K, so the whole reduction stays in the matrix
// cores' int32 accumulators and any split of K gives the same bits.
#include <algorithm>

#include "device.h"
#include "launch.h"
#include "quant8.h"

namespace w4a4 {

namespace {

typedef int v16i __attribute__((ext_vector_type(16)));

constexpr int kThreads = 256;
constexpr int kCUs = 256;      // of an MI355X: launch shapes are planned for it

// One row per WPR waves (256 / (64 WPR) rows a workgroup); NC > 0: the row's
// 16-element chunks stay in registers (NC per lane), so X is read once. NC = 0:
// rows of any length, read twice (the second time from cache). Bound by HBM, 3
// bytes per element: 4096 x 8192 17.8 us, 5.7 TB/s; 777 x 18944 11 us; one row of
// 4096 2.1 us, a launch.
template <bool BF, int WPR, int NC>
__global__ __launch_bounds__(kThreads) void k_w8a8_quant(const uint16_t* __restrict__ x, int64_t ldx, int64_t M, int K,
                                                         int8_t* __restrict__ q, float* __restrict__ s) {
  constexpr int RPB = kThreads / 64 / WPR;
  __shared__ float wave_max[kThreads / 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t row = (int64_t)blockIdx.x * RPB + wave / WPR;
  const bool live = row < M;                       // WPR > 1 has one row per block: uniform
  const int t = (wave % WPR) * 64 + lane;
  const int n16 = live ? K >> 4 : 0;
  const uint4* src = reinterpret_cast<const uint4*>(x + (live ? row : 0) * ldx);
  uint4 raw[NC > 0 ? NC : 1][2];
  uint32_t m = 0;
  if constexpr (NC > 0) {
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int i = c * 64 * WPR + t;
      raw[c][0] = raw[c][1] = uint4{0, 0, 0, 0};
      if (i < n16) {
        raw[c][0] = src[2 * i];
        raw[c][1] = src[2 * i + 1];
      }
    }
#pragma unroll
    for (int c = 0; c < NC; ++c) m = absmax16(raw[c], m);
  } else {
    for (int i = t; i < n16; i += 64 * WPR) {
      const uint4 r[2] = {src[2 * i], src[2 * i + 1]};
      m = absmax16(r, m);
    }
  }
  float a = wave_absmax<BF>(m);
  if constexpr (WPR > 1) {
    if (lane == 0) wave_max[wave] = a;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < WPR; ++w) a = max_or_nan(a, wave_max[w]);
  }
  if (!live) return;
  const float sc = a / 127.0f;                     // correctly rounded
  const float k = BF ? scale_guard(sc) : 1.0f;     // fp16 scales are 0 or >= 2^-31
  const float sk = sc * k;
  const float rs = sc == 0.0f ? 0.0f : 1.0f / sk;
  uint4* dst = reinterpret_cast<uint4*>(q + row * K);
  if constexpr (NC > 0) {
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int i = c * 64 * WPR + t;
      if (i < n16) dst[i] = codes16<BF>(raw[c], k, sk, rs);
    }
  } else {
    for (int i = t; i < n16; i += 64 * WPR) {
      const uint4 r[2] = {src[2 * i], src[2 * i + 1]};
      dst[i] = codes16<BF>(r, k, sk, rs);
    }
  }
  if (t == 0) s[row] = sc;
}

template <bool BF>
void launch_quant(const uint16_t* x, int64_t M, int64_t K, int64_t ldx, int8_t* q, float* s, hipStream_t stream) {
#define W8A8_QUANT(WPR, NC)                                                                          \
  hipLaunchKernelGGL((k_w8a8_quant<BF, WPR, NC>), dim3((unsigned)((M + 4 / WPR - 1) / (4 / WPR))),   \
                     dim3(kThreads), 0, stream, x, ldx, M, (int)K, q, s)
  if (K <= 1024) W8A8_QUANT(1, 1);
  else if (K <= 4096) W8A8_QUANT(4, 1);
  else if (K <= 8192) W8A8_QUANT(4, 2);
  else if (K <= 16384) W8A8_QUANT(4, 4);
  else if (K <= 32768) W8A8_QUANT(4, 8);
  else W8A8_QUANT(4, 0);
#undef W8A8_QUANT
}

struct W8Params {
  const uint16_t* x;          // k_w8a8_gemm_small with XT > 0: the tokens themselves
  int64_t ldx;
  const int8_t* a;
  const float* sa;
  const int8_t* w;
  const float* sw;
  const float* bias;          // or nullptr
  int M, N, K;
  void* y;
  int ydtype;
  int64_t ldy;
  int32_t* part;              // [splits][M][N] int32 sums, or nullptr
  int splits;                 // K ranges
  int stages;                 // 128-k stages per range
};

// Y value of an exact sum (the product rounds to fp32 before the bias is added: no
// fma), and its store as ydt (0 fp32, 1 fp16, 2 bf16).
__device__ __forceinline__ float scaled(int p, float sa, float sw, float b) {
#pragma clang fp contract(off)
  return (float)p * (sa * sw) + b;
}
__device__ __forceinline__ uint16_t bf16_rne(float v) {
  return __builtin_bit_cast(uint16_t, (__bf16)v);
}
__device__ __forceinline__ void store_y(void* y, int ydt, int64_t i, float v) {
  if (ydt == 0) static_cast<float*>(y)[i] = v;
  else if (ydt == 1) static_cast<uint16_t*>(y)[i] = __half_as_ushort(__float2half_rn(v));
  else static_cast<uint16_t*>(y)[i] = bf16_rne(v);
}

// ---- Up to 16 tokens: W streamed once from HBM straight into the operands -----
// A workgroup of NW waves owns 16 channels and splits K across its waves
// (contiguous runs of 64-k steps). v_mfma_i32_16x16x64_i8: lane l supplies 16
// consecutive k of row l % 16 at k offset 16 (l / 16), so a step is one 16-byte
// load per operand and lane, with no LDS on the way; RING steps are in flight
// per wave. The waves' int32 sums meet in LDS (exact in any order). K is a
// multiple of 16: the last step's lanes beyond K, and steps beyond a wave's
// run, read zeros of W.
//
// XT 0: the tokens' codes come from memory. XT 1, 2 (fp16, bf16 tokens): every
// workgroup quantizes all of them itself, in pieces of 1024 elements per wave
// (PIECES each, kept in registers), into LDS, while its first W loads are on
// their way; that saves a launch and the wait for it.
//
// Bound by the W stream: one token 4096 -> 128256 86.9 us, 6.0 TB/s of weights;
// 8192 -> 28672 43.7 us, 5.4 TB/s; small ones by the launch and the loads'
// latency (8192 -> 1024, 8 MB: 7.6 us). With more tokens by the L2 traffic of
// their codes, which every workgroup reads again (M / 16 of W's bytes): see the
// plan. RING 8 measured as 4.
template <int XT, int NW, int RING, int PIECES>
__global__ __launch_bounds__(64 * NW) void k_w8a8_gemm_small(W8Params p) {
  constexpr bool BF = XT == 2;
  __shared__ int red[NW - 1][4][64];
  __shared__ float row_scale[16];
  __shared__ uint32_t row_max[16];
  extern __shared__ __align__(16) uint8_t codes[];     // XT > 0: [M][K rounded up to 64]
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, g = lane >> 4;
  const int n0 = (int)blockIdx.x * 16;
  const int steps = (p.K + 63) >> 6;
  const int h0 = (int)((int64_t)steps * wave / NW), h1 = (int)((int64_t)steps * (wave + 1) / NW);
  const int w_rows = min(16, p.N - n0);
  const __amdgpu_buffer_rsrc_t rA = buffer_rsrc(p.a, XT ? 0 : p.M * p.K);
  const __amdgpu_buffer_rsrc_t rW = buffer_rsrc(p.w + (int64_t)n0 * p.K, w_rows * p.K);
  const int offA = c < p.M ? c * p.K + 16 * g : kDroppedOffset;
  const int offW = c < w_rows ? c * p.K + 16 * g : kDroppedOffset;
  struct Step {
    v4i a, w;
  };
  Step ring[RING];
  auto load = [&](Step& st, int h) {
    const int out = h < h1 && 64 * h + 16 * g < p.K ? 0 : kDroppedOffset;
    st.w = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(rW, offW | out, 64 * h, 0));
    if constexpr (XT == 0)
      st.a = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(rA, offA | out, 64 * h, 0));
  };
  const int KP = steps * 64;
  if constexpr (XT > 0) {
    if (threadIdx.x < 16) row_max[threadIdx.x] = 0;
    const int per_row = (p.K + 1023) >> 10, pieces = p.M * per_row;
    uint4 raw[PIECES][2];
    int row[PIECES], k[PIECES];                          // this lane's first element
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      const int at = wave + NW * i;
      row[i] = at < pieces ? at / per_row : 0;
      k[i] = at < pieces ? (at - row[i] * per_row) * 1024 + 16 * lane : p.K;
      const uint4* src = reinterpret_cast<const uint4*>(p.x + row[i] * p.ldx + min(k[i], p.K - 16));
      raw[i][0] = src[0];
      raw[i][1] = src[1];
    }
#pragma unroll
    for (int u = 0; u < RING; ++u) load(ring[u], h0 + u);
    __syncthreads();                                     // row_max is cleared
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      const float a = wave_absmax<BF>(k[i] < p.K ? absmax16(raw[i], 0) : 0);
      if (lane == 0) atomicMax(&row_max[row[i]], __float_as_uint(a));   // as max_or_nan
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      const float sc = __uint_as_float(row_max[row[i]]) / 127.0f;
      const float kk = BF ? scale_guard(sc) : 1.0f;
      const float sk = sc * kk;
      const float rs = sc == 0.0f ? 0.0f : 1.0f / sk;
      if (k[i] < p.K) {
        *reinterpret_cast<uint4*>(codes + row[i] * KP + k[i]) = codes16<BF>(raw[i], kk, sk, rs);
        if (k[i] == 0) row_scale[row[i]] = sc;
      }
    }
    __syncthreads();
  } else {
#pragma unroll
    for (int u = 0; u < RING; ++u) load(ring[u], h0 + u);
  }
  const uint8_t* const la = codes + (c < p.M ? c : 0) * KP + 16 * g;   // rows past M: their sums are not stored
  v4i acc = {0, 0, 0, 0};
  for (int h = h0; h < h1; h += RING) {
#pragma unroll
    for (int u = 0; u < RING; ++u) {
      v4i a = ring[u].a;
      if constexpr (XT > 0) a = *reinterpret_cast<const v4i*>(la + 64 * min(h + u, steps - 1));
      acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(a, ring[u].w, acc, 0, 0, 0);
      load(ring[u], h + u + RING);
    }
  }
  if (wave > 0) {
#pragma unroll
    for (int r = 0; r < 4; ++r) red[wave - 1][r][lane] = acc[r];
  }
  __syncthreads();
  if (wave != 0) return;
  const int n = n0 + c;
  const float sw = n < p.N ? p.sw[n] : 0.0f;
  const float b = p.bias && n < p.N ? p.bias[n] : 0.0f;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    int v = acc[r];
#pragma unroll
    for (int w = 0; w < NW - 1; ++w) v += red[w][r][lane];
    const int m = 4 * g + r;
    if (m < p.M && n < p.N) store_y(p.y, p.ydtype, m * p.ldy + n, scaled(v, XT ? row_scale[m] : p.sa[m], sw, b));
  }
}

// ---- Tiles ------------------------------------------------------------------
typedef __attribute__((address_space(3))) void* lds_vptr;

// Direct buffer -> LDS copy: lane l's 16 bytes land at lds + 16 l.
__device__ __forceinline__ void dma16(__amdgpu_buffer_rsrc_t r, int voff, int soff, uint8_t* lds) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_vptr)lds, 16, voff, soff, 0, 0);
}

// s_waitcnt on vmcnt only (expcnt/lgkmcnt left at their maxima), gfx9 encoding.
template <int N>
__device__ __forceinline__ void wait_vmcnt() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (15 << 8) | ((N >> 4) << 14));
}

// The raster: logical tile t of nblk (consecutive tiles on one XCD, which is
// workgroup index mod 8, so its L2 holds the rows they share), in groups of
// kGroupRows tile rows.
constexpr int kGroupRows = 4;

// What a tile's sums become: fp32, fp16 or bf16 (p.ydtype says which), or the
// int32 sums of one K range for k_w8a8_join.
enum { OUT_F32 = 0, OUT_16 = 1, OUT_RAW = 2 };

// Workgroup tile BM tokens x BN channels, waves in a WM x WN grid of TI x TJ
// blocks of v_mfma_i32_32x32x32_i8 (lane l: 16 consecutive k of row l % 32 at k
// offset 16 (l / 32)). K stages of 128 bytes per row in an S-deep LDS ring
// filled by direct loads; a row's eight 16-byte slots are XOR-swizzled with
// (row >> 1) & 7, so 16 lanes reading one slot of 16 consecutive rows hit 16
// distinct bank groups. The channels are the instruction's first operand: a
// lane then holds runs of 4 consecutive channels of one token. 16-bit outputs
// swap runs between the wave's halves and are stored 16 bytes per lane as well.
//
// Each workgroup takes logical tiles b, b + G, b + 2 G, ... (G workgroups). The
// next tile's first S stages are issued before a tile's outputs are stored, so
// the stores drain under the next tile's matrix work.
//
// Bound by the matrix cores at the clock that the power limit leaves them: 4096
// x 28672 x 8192 764 us, 2.5 POP/s; smaller products by what their last round of
// tiles leaves idle (777 x 3584 x 18944, 196 tiles: 67 us, 1.6 POP/s). WIDE: rows of y take
// 16-byte stores (N, ldy and y aligned); else element stores, one tile per
// workgroup.
template <int BM, int BN, int WM, int WN, int S, int OUT, bool WIDE>
__global__ __launch_bounds__(64 * WM * WN) __attribute__((amdgpu_waves_per_eu(WM * WN / 4, WM * WN / 4)))
void k_w8a8_gemm_tiles(W8Params p) {
  constexpr int RB = 128;                              // bytes (k) per row and stage
  constexpr int NWAVE = WM * WN;
  constexpr int TI = BM / WM / 32, TJ = BN / WN / 32;
  constexpr int NA = BM / 8 / NWAVE, NW = BN / 8 / NWAVE;   // 1 KB loads per wave and stage
  constexpr int W_OFF = BM * RB, STAGE = (BM + BN) * RB;
  constexpr int PER_STAGE = NA + NW;
  constexpr int NSTEP = RB / 32;
  constexpr int LPM = (PER_STAGE + TI * TJ - 1) / (TI * TJ);   // direct loads per matrix instruction
  constexpr int NST = TI * TJ * (OUT == OUT_16 ? 2 : 4);       // stores per wave and tile
  static_assert(NA * 8 * NWAVE == BM && NW * 8 * NWAVE == BN, "tile rows per wave");
  __shared__ __align__(16) uint8_t sm0[STAGE];
  __shared__ __align__(16) uint8_t sm1[STAGE];
  __shared__ __align__(16) uint8_t sm2[S == 3 ? STAGE : 16];
  __shared__ __align__(16) float sas[BM], sws[BN], biases[BN];
  static_assert(BM <= 64 * NWAVE && BN <= 64 * NWAVE, "one row per thread");

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int l32 = lane & 31, lhi = lane >> 5;
  const int tiles_m = (p.M + BM - 1) / BM, tiles_n = (p.N + BN - 1) / BN;
  const int tiles = tiles_m * tiles_n, nblk = tiles * p.splits;
  const int G = gridDim.x;
  // consecutive logical tiles on one XCD (workgroup index mod 8)
  const int xcd = blockIdx.x & 7;
  int t = xcd * (G >> 3) + min(xcd, G & 7) + (blockIdx.x >> 3);

  // A lane's 16-byte slot of a row is the same in all its loads (their rows
  // differ by multiples of 8 NWAVE).
  static_assert(NWAVE % 2 == 0, "slot of a lane");
  const int seg = 16 * ((lane & 7) ^ ((4 * wave + (lane >> 4)) & 7));
  int part, tile_m, tile_n, kspan, nk;
  __amdgpu_buffer_rsrc_t rA, rW;
  int voffA[NA], voffW[NW];
  float sa_t, sw_t, bias_t;
  auto setup = [&](int tt) {
    part = tt / tiles;
    tt -= part * tiles;
    const int grp = tt / (kGroupRows * tiles_n);
    const int first_m = grp * kGroupRows, gsize = min(tiles_m - first_m, kGroupRows);
    const int rem = tt - grp * kGroupRows * tiles_n;
    tile_m = (first_m + rem % gsize) * BM;
    tile_n = rem / gsize * BN;
    const int a_rows = min(BM, p.M - tile_m), w_rows = min(BN, p.N - tile_n);
    rA = buffer_rsrc(p.a + (int64_t)tile_m * p.K, a_rows * p.K);
    rW = buffer_rsrc(p.w + (int64_t)tile_n * p.K, w_rows * p.K);
    // The range's stages, rounded up to a multiple of the ring depth: what lies
    // beyond K is read as zeros (tokens) or as anything (channels).
    const int k0 = part * p.stages * RB;
    kspan = min(p.K - k0, p.stages * RB);
    nk = (kspan + S * RB - 1) / (S * RB) * S;
#pragma unroll
    for (int i = 0; i < NA; ++i)
      voffA[i] = min(8 * (wave + NWAVE * i) + (lane >> 3), a_rows - 1) * p.K + seg + k0;
#pragma unroll
    for (int i = 0; i < NW; ++i)
      voffW[i] = min(8 * (wave + NWAVE * i) + (lane >> 3), w_rows - 1) * p.K + seg + k0;
    // the tile's scales and bias, used in its output
    if constexpr (OUT != OUT_RAW) {
      const int m = tile_m + (int)threadIdx.x, n = tile_n + (int)threadIdx.x;
      sa_t = p.sa[min(m, p.M - 1)];
      sw_t = p.sw[min(n, p.N - 1)];
      bias_t = p.bias ? p.bias[min(n, p.N - 1)] : 0.0f;
    }
  };
// One of the PER_STAGE direct loads of stage KT into slot SM; OUTK holds the
// sign bit where the lane's slot of the stage lies beyond K (see
// kDroppedOffset), else 0.
#define OUT_OF(KT) (seg >= kspan - (KT) * RB ? kDroppedOffset : 0)
#define ISSUE1(KT, SM, X, OUTK)                                                                             \
  {                                                                                                         \
    if ((X) < NA) dma16(rA, voffA[(X) < NA ? (X) : 0] | (OUTK), (KT) * RB, (SM) + (wave + NWAVE * (X)) * 1024); \
    else dma16(rW, voffW[(X) < NA ? 0 : (X) - NA], (KT) * RB, (SM) + W_OFF + (wave + NWAVE * ((X) - NA)) * 1024); \
  }
#define ISSUE(KT, SM)                                                                                       \
  {                                                                                                         \
    const int out_ = OUT_OF(KT);                                                                            \
    _Pragma("unroll") for (int x_ = 0; x_ < PER_STAGE; ++x_) ISSUE1(KT, SM, x_, out_)                       \
  }
  v16i acc[TI][TJ];
#define CLEAR()                                                                                             \
  _Pragma("unroll") for (int i = 0; i < TI; ++i)                                                            \
  _Pragma("unroll") for (int j = 0; j < TJ; ++j)                                                            \
  _Pragma("unroll") for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;

  const int rowA = wm * (BM / WM) + l32, rowW = wn * (BN / WN) + l32;
  int offA[NSTEP], offW[NSTEP];
#pragma unroll
  for (int u = 0; u < NSTEP; ++u) {
    offA[u] = rowA * RB + 16 * ((2 * u + lhi) ^ ((rowA >> 1) & 7));
    offW[u] = W_OFF + rowW * RB + 16 * ((2 * u + lhi) ^ ((rowW >> 1) & 7));
  }
  v4i av[2][TI], wv[2][TJ];
// Operand read X of step U (the TI blocks of tokens, then the TJ of channels).
#define LOAD1(SM, U, B, X)                                                                                  \
  {                                                                                                         \
    if ((X) < TI) av[B][(X) < TI ? (X) : 0] = *reinterpret_cast<const v4i*>((SM) + offA[U] + 32 * RB * (X)); \
    else wv[B][(X) < TI ? 0 : (X) - TI] = *reinterpret_cast<const v4i*>((SM) + offW[U] + 32 * RB * ((X) - TI)); \
  }
#define LOAD_OPS(SM, U, B) \
  _Pragma("unroll") for (int x_ = 0; x_ < TI + TJ; ++x_) LOAD1(SM, U, B, x_)
// Barrier between stages: each wave has waited for its own direct loads of the
// stage, and every wave has finished with the slot about to be refilled. No
// memory fence, which would drain the loads in flight.
#define STAGE_BARRIER()                                                                                     \
  {                                                                                                         \
    __builtin_amdgcn_sched_barrier(0);                                                                      \
    __builtin_amdgcn_s_barrier();                                                                           \
    __builtin_amdgcn_sched_barrier(0);                                                                      \
  }
// Stage KT in slot CUR, its first step's operands in registers. Behind each
// matrix instruction goes one operand read of the next step and, in the last
// step, one direct load of the slot's refill: a wave issues in order, and a
// burst of loads in front of the matrix work would stall it. Before the last
// step's matrix work the stage's slot is read out: there the waves meet and go
// on to the next stage's (slot NXT) first operands, so neither the barrier nor
// those reads leave the matrix cores idle. LEFT: the stages behind the next
// one that may still be in flight then.
#define STAGE_OF(KT, CUR, NXT, MORE, REFILL, LEFT)                                                          \
  {                                                                                                         \
    int out_ = 0;                                                                                           \
    _Pragma("unroll") for (int u_ = 0; u_ < NSTEP; ++u_) {                                                  \
      if (u_ + 1 == NSTEP && (MORE)) {                                                                      \
        __builtin_amdgcn_s_waitcnt(0xC07F); /* lgkmcnt(0): this wave has read the slot out */               \
        wait_vmcnt<(LEFT) * PER_STAGE>();                                                                   \
        STAGE_BARRIER();                                                                                    \
        if (REFILL) out_ = OUT_OF((KT) + S);                                                                \
      }                                                                                                     \
      _Pragma("unroll") for (int x_ = 0; x_ < TI * TJ; ++x_) {                                              \
        acc[x_ / TJ][x_ % TJ] = __builtin_amdgcn_mfma_i32_32x32x32_i8(wv[u_ & 1][x_ % TJ], av[u_ & 1][x_ / TJ], \
                                                                      acc[x_ / TJ][x_ % TJ], 0, 0, 0);      \
        if (u_ + 1 < NSTEP) {                                                                               \
          if (x_ < TI + TJ) LOAD1(CUR, (u_ + 1) % NSTEP, (u_ + 1) & 1, x_);                                 \
        } else if (MORE) {                                                                                  \
          if (x_ < TI + TJ) LOAD1(NXT, 0, 0, x_);                                                           \
          _Pragma("unroll") for (int y_ = x_ * LPM; y_ < x_ * LPM + LPM; ++y_)                              \
            if (y_ < PER_STAGE && (REFILL)) ISSUE1((KT) + S, CUR, y_, out_);                                \
        }                                                                                                   \
        __builtin_amdgcn_sched_barrier(0);                                                                  \
      }                                                                                                     \
    }                                                                                                       \
  }
  static_assert(TI + TJ <= TI * TJ, "one operand read per matrix instruction");
  static_assert(NSTEP % 2 == 0, "operand buffers alternate across stages");
// A tile's first S stages into the ring, which every wave has finished with.
#define FILL_RING()                                                                                         \
  {                                                                                                         \
    ISSUE(0, sm0);                                                                                          \
    ISSUE(1, sm1);                                                                                          \
    if constexpr (S == 3) ISSUE(2, sm2);                                                                    \
  }
// All of a tile's matrix work, its first stage in the ring. The loop holds no
// condition around a load or a wait, so the compiler's own waits on the direct
// loads count exactly as the ones written here.
#define TILE()                                                                                              \
  {                                                                                                         \
    LOAD_OPS(sm0, 0, 0);                                                                                    \
    if constexpr (S == 2) {                                                                                 \
      for (int kt = 0; kt + 2 < nk; kt += 2) {                                                              \
        STAGE_OF(kt, sm0, sm1, true, true, 0)                                                               \
        STAGE_OF(kt + 1, sm1, sm0, true, true, 0)                                                           \
      }                                                                                                     \
      STAGE_OF(nk - 2, sm0, sm1, true, false, 0)                                                            \
      STAGE_OF(nk - 1, sm1, sm0, false, false, 0)                                                           \
    } else {                                                                                                \
      for (int kt = 0; kt + 3 < nk; kt += 3) {                                                              \
        STAGE_OF(kt, sm0, sm1, true, true, 1)                                                               \
        STAGE_OF(kt + 1, sm1, sm2, true, true, 1)                                                           \
        STAGE_OF(kt + 2, sm2, sm0, true, true, 1)                                                           \
      }                                                                                                     \
      STAGE_OF(nk - 3, sm0, sm1, true, false, 1)                                                            \
      STAGE_OF(nk - 2, sm1, sm2, true, false, 0)                                                            \
      STAGE_OF(nk - 1, sm2, sm0, false, false, 0)                                                           \
    }                                                                                                       \
  }

  // Output of the tile at (m0, n0) of K range pt.
  const int esz = OUT == OUT_16 ? 2 : 4;
  auto store_tile = [&](int m0, int n0, int pt) {
    uint8_t* y = OUT == OUT_RAW ? reinterpret_cast<uint8_t*>(p.part + (int64_t)pt * p.M * p.N)
                                : static_cast<uint8_t*>(p.y);
    const int64_t ldy = OUT == OUT_RAW ? p.N : p.ldy;
    // WIDE: y's rows of this tile as one buffer (< 2^31 bytes, checked by the
    // host); a lane outside M x N gets an offset past it
    const int ldb = WIDE ? (int)(ldy * esz) : 0;
    const __amdgpu_buffer_rsrc_t rY = buffer_rsrc(y + (int64_t)m0 * ldy * esz, WIDE ? min(BM, p.M - m0) * ldb : 0);
#pragma unroll
    for (int i = 0; i < TI; ++i) {
      const int row = wm * (BM / WM) + 32 * i + l32;
      const float sa = OUT == OUT_RAW ? 0.0f : sas[row];
#pragma unroll
      for (int j = 0; j < TJ; ++j) {
        const int c0 = wn * (BN / WN) + 32 * j + 4 * lhi;      // channel of register 0
        uint32_t h[4][2];                                      // 16-bit pairs
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          v4u w;
          if constexpr (OUT == OUT_RAW) {
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = (uint32_t)acc[i][j][4 * q + e];
          } else {
            const v4f sw = *reinterpret_cast<const v4f*>(sws + c0 + 8 * q);
            const v4f bv = *reinterpret_cast<const v4f*>(biases + c0 + 8 * q);
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = __float_as_uint(scaled(acc[i][j][4 * q + e], sa, sw[e], bv[e]));
          }
          if constexpr (!WIDE) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int n = n0 + c0 + 8 * q + e;
              if (m0 + row < p.M && n < p.N)
                store_y(y, OUT == OUT_16 ? p.ydtype : 0, (m0 + row) * ldy + n, __uint_as_float(w[e]));
            }
          } else if constexpr (OUT == OUT_16) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float f0 = __uint_as_float(w[2 * e]), f1 = __uint_as_float(w[2 * e + 1]);
              const uint32_t f16 = __half_as_ushort(__float2half_rn(f0)) | (uint32_t)__half_as_ushort(__float2half_rn(f1)) << 16;
              const uint32_t b16 = bf16_rne(f0) | (uint32_t)bf16_rne(f1) << 16;
              h[q][e] = p.ydtype == 1 ? f16 : b16;
            }
          } else {
            const int n = n0 + c0 + 8 * q;
            __builtin_amdgcn_raw_buffer_store_b128(w, rY, n < p.N ? row * ldb + n * 4 : kDroppedOffset, 0, 0);
          }
        }
        if constexpr (WIDE && OUT == OUT_16) {
          // runs q (even) and q + 1: the low half of the wave takes channels
          // 8 q .. 8 q + 7, the high half 8 q + 8 .. 8 q + 15
#pragma unroll
          for (int q = 0; q < 4; q += 2) {
            const auto s0 = __builtin_amdgcn_permlane32_swap(h[q][0], h[q + 1][0], false, false);
            const auto s1 = __builtin_amdgcn_permlane32_swap(h[q][1], h[q + 1][1], false, false);
            const int n = n0 + wn * (BN / WN) + 32 * j + 8 * q + 8 * lhi;
            __builtin_amdgcn_raw_buffer_store_b128(v4u{s0[0], s1[0], s0[1], s1[1]}, rY,
                                                   n < p.N ? row * ldb + n * 2 : kDroppedOffset, 0, 0);
          }
        }
      }
    }
  };
// The tile's scales into LDS, where its output reads them: every wave is past
// the last tile's output (it met the others in this tile's stages).
#define SCALES_TO_LDS()                                                                                     \
  if constexpr (OUT != OUT_RAW) {                                                                           \
    if (threadIdx.x < BM) sas[threadIdx.x] = sa_t;                                                          \
    if (threadIdx.x < BN) sws[threadIdx.x] = sw_t, biases[threadIdx.x] = bias_t;                            \
  }                                                                                                         \
  __syncthreads();

  setup(t);
  FILL_RING()
  wait_vmcnt<(S - 1) * PER_STAGE>();
  STAGE_BARRIER();
  if constexpr (WIDE) {
    const int count = (nblk - t + G - 1) / G;
    for (int it = 1; it < count; ++it) {
      CLEAR()
      TILE()
      SCALES_TO_LDS()                                  // and the ring is free
      const int m0 = tile_m, n0 = tile_n, pt = part;
      t += G;
      setup(t);
      FILL_RING()
      store_tile(m0, n0, pt);
      // stage 0 is in: at most the later stages and the stores behind it are out
      // (memory operations complete in order; every store above is issued)
      wait_vmcnt<((S - 1) * PER_STAGE + NST < 63 ? (S - 1) * PER_STAGE + NST : 63)>();
      STAGE_BARRIER();
    }
  }
  CLEAR()
  TILE()
  SCALES_TO_LDS()
  store_tile(tile_m, tile_n, part);
#undef SCALES_TO_LDS
#undef TILE
#undef FILL_RING
#undef STAGE_OF
#undef STAGE_BARRIER
#undef LOAD_OPS
#undef LOAD1
#undef CLEAR
#undef ISSUE
#undef ISSUE1
#undef OUT_OF
}

// Adds the K splits' int32 sums and scales them. They come from the caches: 16 x
// 8192 outputs in four ranges 4.4 us.
__global__ __launch_bounds__(kThreads) void k_w8a8_join(W8Params p, int splits) {
  const int64_t total = (int64_t)p.M * p.N;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < total; i += (int64_t)gridDim.x * kThreads) {
    int v = 0;
    for (int s = 0; s < splits; ++s) v += p.part[s * total + i];
    const int64_t m = i / p.N;
    const int n = (int)(i - m * p.N);
    store_y(p.y, p.ydtype, m * p.ldy + n, scaled(v, p.sa[m], p.sw[n], p.bias ? p.bias[n] : 0.0f));
  }
}

// splits > 1: only for tiles whose OUT_RAW form is built (SPLIT).
template <int BM, int BN, int WM, int WN, int S, bool SPLIT>
void launch_tiles(W8Params p, int splits, hipStream_t stream) {
  const int64_t tiles = (int64_t)((p.M + BM - 1) / BM) * ((p.N + BN - 1) / BN);
  const int nk = (p.K + 127) / 128;
  p.stages = (nk + splits - 1) / splits;
  p.splits = splits = (nk + p.stages - 1) / p.stages;
  const int64_t blocks = tiles * splits;
  const dim3 grid((unsigned)std::min<int64_t>(blocks, kCUs)), block(64 * WM * WN);
  const int64_t ldb = (splits > 1 ? p.N : p.ldy) * (splits > 1 || p.ydtype == 0 ? 4 : 2);
  const int cols = splits > 1 || p.ydtype == 0 ? 4 : 8;
  const bool wide = p.N % cols == 0 && ldb % 16 == 0 && BM * ldb < (int64_t{1} << 31) &&
                    (reinterpret_cast<uintptr_t>(splits > 1 ? static_cast<void*>(p.part) : p.y) & 15) == 0;
  const dim3 each((unsigned)blocks);                   // the element-store form: one tile per workgroup
#define W8A8_TILES(OUT)                                                                                         \
  if (wide) hipLaunchKernelGGL((k_w8a8_gemm_tiles<BM, BN, WM, WN, S, OUT, true>), grid, block, 0, stream, p);   \
  else hipLaunchKernelGGL((k_w8a8_gemm_tiles<BM, BN, WM, WN, S, OUT, false>), each, block, 0, stream, p)
  if constexpr (SPLIT) {
    if (splits > 1) {
      W8A8_TILES(OUT_RAW);
      const int64_t jb = std::min<int64_t>(((int64_t)p.M * p.N + kThreads - 1) / kThreads, 8192);
      hipLaunchKernelGGL(k_w8a8_join, dim3((unsigned)jb), dim3(kThreads), 0, stream, p, splits);
      return;
    }
  }
  if (p.ydtype == 0) {
    W8A8_TILES(OUT_F32);
  } else {
    W8A8_TILES(OUT_16);
  }
#undef W8A8_TILES
}

// Which kernel, and into how many K ranges.
//
// Up to 16 tokens the W stream decides (k_w8a8_gemm_small), but that kernel's
// workgroups each read all tokens' codes: with more than 8 tokens and W above
// 64 MiB 128-channel tiles take over, which read them 8 times less often (16 x
// 28672 x 8192: 53.5 us, 60 in the small kernel; 16 x 8192 x 28672: 47 and 54;
// 16 x 18944 x 3584: 19.5 and 22.4; below, 16 x 8192 x 8192: 21.8 and 20.1; all
// with W from HBM).
//
// Above 16 tokens, the tile whose estimated time is least: rounds of tiles over
// the CUs times (stages x the tile's time per 128-k stage + its start and
// output). The times (us: 256 x 256 tiles 1.15 a stage, 256 x 128 0.8, 128 x 128
// 0.5) are fitted to measured shapes, tokens x channels x K, among them those named
// here, where the choice is the fastest; us of the three in turn: 4096 x 4096 x 4096 62.6, 70.7, 80.9; 1024 x 8192 x 28672 229, 224,
// 290; 512 x 8192 x 8192 74, 55.2, 43.4. 128 x 128 tiles may also split K, which
// costs a launch and 8 bytes per output and range through the caches (64 x 8192
// x 8192: 35.6 us whole, 25.5 in two ranges, 21.2 in four; 512 x 4096 x 11008:
// 53.8, 41.7, 50.1; 256 x 11008 x 4096: 24.1, 41.5, 44.7).
enum { TILE_SMALL = 0, TILE_256 = 1, TILE_256_128 = 2, TILE_128 = 3 };
struct W8Plan {
  int tile, splits;
};
W8Plan plan_w8a8(int64_t M, int64_t N, int64_t K) {
  if (M <= 8 || (M <= 16 && N * K <= (int64_t{1} << 26))) return W8Plan{TILE_SMALL, 1};
  const int64_t nk = (K + 127) / 128;
  W8Plan best{TILE_256, 1};
  double best_us = 1e30;
  auto consider = [&](int tile, int64_t bm, int64_t bn, double stage, double start, int splits) {
    const int64_t tiles = ((M + bm - 1) / bm) * ((N + bn - 1) / bn);
    const int64_t rounds = (tiles * splits + kCUs - 1) / kCUs;
    double us = rounds * (((nk + splits - 1) / splits) * stage + start);
    if (splits > 1) us += 4.0 + 8.0 * splits * M * N / 2.5e6;
    if (us < best_us) {
      best_us = us;
      best = W8Plan{tile, splits};
    }
  };
  consider(TILE_256, 256, 256, 1.15, 3.0, 1);
  consider(TILE_256_128, 256, 128, 0.8, 2.5, 1);
  for (int splits = 1; splits <= 16 && splits * 2 <= nk; splits *= 2)
    consider(TILE_128, 128, 128, 0.5, 2.0, splits);
  return best;
}

}  // namespace

void launch_w8a8_quant(const void* x, int bf16, int64_t M, int64_t K, int64_t ldx, int8_t* q, float* s,
                       hipStream_t stream) {
  const uint16_t* xp = static_cast<const uint16_t*>(x);
  if (bf16) launch_quant<true>(xp, M, K, ldx, q, s, stream);
  else launch_quant<false>(xp, M, K, ldx, q, s, stream);
}

namespace {

W8Params params(const W8GemmArgs& a) {
  W8Params p = {};
  p.a = a.a;
  p.sa = a.sa;
  p.w = a.w;
  p.sw = a.sw;
  p.bias = a.bias;
  p.M = (int)a.M;
  p.N = (int)a.N;
  p.K = (int)a.K;
  p.y = a.y;
  p.ydtype = a.ydtype;
  p.ldy = a.ldy;
  p.splits = 1;
  return p;
}

// 4 waves a workgroup where its count fills the CUs twice over, else 8 (one
// token, W from HBM, us: 8192 x 8192 14.0 with 4 and 15.1 with 8, 4096 x 11008
// 13.4 and 11.1, 1024 x 8192 9.2 and 6.8).
bool four_waves(int64_t N) { return N >= 32 * kCUs; }

template <int XT, int PIECES>
void launch_small(const W8Params& p, hipStream_t stream) {
  const dim3 grid((unsigned)((p.N + 15) / 16));
  const unsigned lds = XT ? (unsigned)(p.M * ((p.K + 63) / 64 * 64)) : 0;
  if (four_waves(p.N)) hipLaunchKernelGGL((k_w8a8_gemm_small<XT, 4, 4, PIECES>), grid, dim3(256), lds, stream, p);
  else hipLaunchKernelGGL((k_w8a8_gemm_small<XT, 8, 4, PIECES>), grid, dim3(512), lds, stream, p);
}

// Pieces of 1024 elements per wave that a workgroup of k_w8a8_gemm_small has to
// quantize for all tokens.
int64_t pieces_per_wave(int64_t M, int64_t N, int64_t K) {
  const int64_t nw = four_waves(N) ? 4 : 8;
  return (M * ((K + 1023) / 1024) + nw - 1) / nw;
}

}  // namespace

void launch_w8a8_gemm(const W8GemmArgs& a, hipStream_t stream) {
  W8Params p = params(a);
  const W8Plan pl = plan_w8a8(a.M, a.N, a.K);
  switch (pl.tile) {
    case TILE_SMALL: launch_small<0, 0>(p, stream); return;
    case TILE_256: launch_tiles<256, 256, 2, 4, 2, false>(p, 1, stream); return;
    case TILE_256_128: launch_tiles<256, 128, 4, 2, 3, false>(p, 1, stream); return;
    default:
      if (pl.splits > 1) p.part = static_cast<int32_t*>(a.workspace);
      launch_tiles<128, 128, 2, 2, 3, true>(p, pl.splits, stream);
      return;
  }
}

// Every workgroup quantizes all tokens, so it pays up to 4 pieces a wave (W
// from HBM, us, one launch and two): 1 x 11008 x 4096 10.6 and 14.2, 1 x 28672 x
// 8192 43.7 and 47.5, 4 x 11008 x 4096 (4 pieces) 13.0 and 16.3, 8 x 4096 x 4096
// (4) 10.1 and 9.8; with 7 and 8 pieces 1 x 8192 x 28672 47.0 and 46.7, 8 x 8192
// x 4096 14.9 and 13.6.
bool w8a8_one_launch(int64_t M, int64_t N, int64_t K) {
  return plan_w8a8(M, N, K).tile == TILE_SMALL && pieces_per_wave(M, N, K) <= 4;
}

void launch_w8a8_small(const W8GemmArgs& a, const void* x, int bf16, int64_t ldx, hipStream_t stream) {
  W8Params p = params(a);
  p.x = static_cast<const uint16_t*>(x);
  p.ldx = ldx;
  const int64_t pieces = pieces_per_wave(a.M, a.N, a.K);
#define W8A8_SMALL(PIECES) bf16 ? launch_small<2, PIECES>(p, stream) : launch_small<1, PIECES>(p, stream)
  if (pieces <= 1) W8A8_SMALL(1);
  else if (pieces <= 2) W8A8_SMALL(2);
  else W8A8_SMALL(4);
#undef W8A8_SMALL
}

int64_t w8a8_workspace(int64_t M, int64_t N, int64_t K) {
  const W8Plan pl = plan_w8a8(M, N, K);
  return pl.splits > 1 ? (int64_t)pl.splits * M * N * 4 : 0;
}

}  // namespace w4a4
