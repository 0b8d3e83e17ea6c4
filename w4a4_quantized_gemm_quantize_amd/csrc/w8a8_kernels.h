// Kernels of the INT8 products (w8a8_gemm, w8a8_linear and their forms with an
// epilogue): the streaming kernel for up to 16 tokens, the tiled one, and the
// choice between them. Each source that includes this instantiates what it launches.
#pragma once

#include <algorithm>

#include "act8.h"
#include "device.h"
#include "launch.h"
#include "quant8.h"

namespace w4a4 {

namespace {

typedef int v16i __attribute__((ext_vector_type(16)));

constexpr int kThreads = 256;
constexpr int kCUs = 256;      // of an MI355X: launch shapes are planned for it

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
  int32_t* part;              // [splits][M][part_ld] int32 sums, or nullptr
  int part_ld;
  int splits;                 // K ranges
  int stages;                 // 128-k stages per range
  int act;                    // forms with an epilogue: ACT_*, and the residual [M][ldr] or nullptr
  const uint16_t* res;
  int64_t ldr;
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

// 16-bit values of type ydt (1 fp16, 2 bf16), and back.
__device__ __forceinline__ float load16(const uint16_t* r, int ydt, int64_t i) {
  return ydt == 1 ? (float)__builtin_bit_cast(_Float16, r[i]) : __uint_as_float((uint32_t)r[i] << 16);
}

// What becomes of a product: itself; act(v) + residual; or, of interleaved
// channels 2n and 2n + 1, act(v[2n]) v[2n + 1] + residual. The forms with an
// epilogue write fp16 or bf16, rounded once.
enum { EPI_PLAIN = 0, EPI_ACT = 1, EPI_GATED = 2 };

// ---- Up to 16 tokens: W streamed once from HBM into the operands ---------------
// A workgroup of NW waves owns 16 channels and splits K across its waves
// (contiguous runs of blocks of four 64-k steps, the next block on its way). The
// waves' int32 sums meet in LDS (exact in any order). K is a multiple of 16: lanes
// beyond K, and steps beyond a wave's run, read zeros of W.
//
// v_mfma_i32_16x16x64_i8: lane l supplies 16 consecutive k of row l % 16 at k offset
// 16 (l / 16), so 16 neighbouring lanes want 16 rows; loaded so, a load touches 64
// pieces of 16 bytes, and the cache serves about 0.65 of them a clock. Blocks are
// loaded in whole runs of a row, 256 bytes for 16 lanes, and turned by LDS (us, W from
// HBM, tokens x channels x K, loads straight into the operands and these: 16 x 8192 x 8192
// 20.5 and 15.7; 8 x 28672 x 8192 54 and 45; 16 x 4096 x 11008 17.9 and 13.9; 8 x 11008 x 4096 14.3
// and 11.7; one token 4096 x 11008 12.4 and 12.1, 1024 x 8192 7.4 and 6.8).
//
// XT 0: the tokens' codes come from memory. XT 1, 2 (fp16, bf16 tokens): every
// workgroup quantizes all of them itself, in pieces of 1024 elements per wave
// (PIECES each, kept in registers), into LDS, while its first W loads are on
// their way; that saves a launch and the wait for it. Its time is mostly latency, so
// where the blocks' LDS keeps workgroups from a CU that it could hold, W is loaded
// straight into the operands (TURN false), a step's refill behind its use.
//
// Bound by the W stream: one token 4096 -> 128256 86.9 us, 6.0 TB/s of weights;
// 8192 -> 28672 42.3 us, 5.6 TB/s; small ones by the launch and the loads' latency
// (8192 -> 1024, 8 MB: 6.8 us).
template <int XT, int NW, int PIECES, int EPI, bool TURN>
__global__ __launch_bounds__(64 * NW) void k_w8a8_gemm_small(W8Params p) {
  constexpr bool BF = XT == 2;
  static_assert(TURN || XT > 0, "codes from memory are turned");
  __shared__ float row_scale[16];
  __shared__ __align__(16) uint8_t turn[NW][TURN ? 4096 : 1024];   // a wave's block, then its sums
  __shared__ uint32_t row_max[16];
  extern __shared__ __align__(16) uint8_t codes[];     // XT > 0: [M][K rounded up to 64]
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, g = lane >> 4;
  const int n0 = (int)blockIdx.x * 16;
  const int steps = (p.K + 63) >> 6, blocks = (steps + 3) >> 2;
  const int h0 = (int)((int64_t)blocks * wave / NW) * 4, h1 = min((int)((int64_t)blocks * (wave + 1) / NW) * 4, steps);
  const int w_rows = min(16, p.N - n0);
  const __amdgpu_buffer_rsrc_t rA = buffer_rsrc(p.a, XT ? 0 : p.M * p.K);
  const __amdgpu_buffer_rsrc_t rW = buffer_rsrc(p.w + (int64_t)n0 * p.K, w_rows * p.K);
  // load j of a block: row 4 j + lane / 16, 16 bytes of its 256; or the operand of step j
  const int run_row = TURN ? lane >> 4 : c, run_k = 16 * (TURN ? lane & 15 : g);
  v4i next_w[4], next_a[XT ? 1 : 4];
  auto load1 = [&](int h, int j) {
    const int row = TURN ? 4 * j + run_row : run_row, at = TURN ? h : h + j;
    const int out = at < h1 && 64 * at + run_k < p.K ? 0 : kDroppedOffset;
    next_w[j] = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(
        rW, (row < w_rows ? row * p.K + run_k : kDroppedOffset) | out, 64 * at, 0));
    if constexpr (XT == 0)
      next_a[j] = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(
          rA, (row < p.M ? row * p.K + run_k : kDroppedOffset) | out, 64 * at, 0));
  };
  auto load = [&](int h) {
#pragma unroll
    for (int j = 0; j < 4; ++j) load1(h, j);
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
    load(h0);
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
    load(h0);
  }
  const uint8_t* const la = codes + (c < p.M ? c : 0) * KP + 16 * g;   // rows past M: their sums are not stored
  // The region is the wave's own, whose LDS operations complete in order; 16-byte
  // pieces are swizzled by their row, so that 16 lanes meet 16 bank groups both ways.
  uint8_t* const mine = turn[wave];
  int put[4], take[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    put[j] = (4 * j + run_row) * 256 + 16 * ((lane & 15) ^ (4 * j + run_row));
    take[j] = c * 256 + 16 * ((4 * j + g) ^ c);
  }
  auto operands = [&](const v4i* from, v4i to[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) *reinterpret_cast<v4i*>(mine + put[j]) = from[j];
    asm volatile("" ::: "memory");
#pragma unroll
    for (int u = 0; u < 4; ++u) to[u] = *reinterpret_cast<const v4i*>(mine + take[u]);
    asm volatile("" ::: "memory");
  };
  v4i acc = {0, 0, 0, 0};
  for (int h = h0; h < h1; h += 4) {
    v4i w[4], a[4];
    if constexpr (TURN) operands(next_w, w);
    if constexpr (XT == 0) {
      operands(next_a, a);
    } else {
#pragma unroll
      for (int u = 0; u < 4; ++u) a[u] = *reinterpret_cast<const v4i*>(la + 64 * min(h + u, steps - 1));
    }
    if constexpr (TURN) load(h + 4);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if constexpr (!TURN) {
        w[u] = next_w[u];
        load1(h + 4, u);
      }
      acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[u], w[u], acc, 0, 0, 0);
    }
  }
  if (wave > 0) {
#pragma unroll
    for (int r = 0; r < 4; ++r) reinterpret_cast<int*>(mine)[64 * r + lane] = acc[r];
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
    for (int w = 1; w < NW; ++w) v += reinterpret_cast<const int*>(turn[w])[64 * r + lane];
    const int m = 4 * g + r;
    if constexpr (EPI == EPI_PLAIN) {
      if (m < p.M && n < p.N) store_y(p.y, p.ydtype, m * p.ldy + n, scaled(v, XT ? row_scale[m] : p.sa[m], sw, b));
    } else {
      float f = scaled(v, m < p.M ? (XT ? row_scale[m] : p.sa[m]) : 0.0f, sw, b);
      const float up = dpp<DPP_QUAD_1032>(f);              // gated: the channel next to an even one
      const int at = EPI == EPI_GATED ? n >> 1 : n;
      f = activate(p.act, f);
      if constexpr (EPI == EPI_GATED) f *= up;
      if (m < p.M && n < p.N && (EPI == EPI_ACT || !(c & 1))) {
        store_y(p.y, p.ydtype, m * p.ldy + at, plus(f, p.res ? load16(p.res, p.ydtype, m * p.ldr + at) : 0.0f));
      }
    }
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
// EPI: an epilogue follows (OUT_16 and WIDE only), ACT says which kind of
// activation it has, BF that the outputs are bf16 (else fp16). Its residual is fetched ahead of the next tile's stages, in the
// layout of the stores, and takes their lane exchange the other way round.
enum { KIND_LINEAR = 0, KIND_SIGMOID = 1, KIND_ERF = 2 };
template <int BM, int BN, int WM, int WN, int S, int OUT, bool WIDE, int EPI = EPI_PLAIN, int ACT = KIND_LINEAR, bool BF = false>
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
  constexpr int NRUN = EPI == EPI_GATED ? 1 : 2;               // 16-byte stores per block of 16-bit outputs
  constexpr int NST = TI * TJ * (OUT == OUT_16 ? NRUN : 4);    // stores per wave and tile
  static_assert(EPI == EPI_PLAIN || (OUT == OUT_16 && WIDE), "epilogues write wide 16-bit rows");
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

  // First of the 8 outputs that this lane's 16-byte store u of column block j holds.
  auto out_channel = [&](int n0, int j, int u) {
    const int c = n0 + wn * (BN / WN) + 32 * j;
    return EPI == EPI_GATED ? (c >> 1) + 8 * lhi : c + 16 * u + 8 * lhi;
  };
  // The residual of the tile at (m0, n0), as its stores lie. Columns past the output's
  // are read from the next row (they are not stored), never past the last row's end.
  // The second half of many block rows is fetched where the first one's registers are free.
  constexpr int EARLY = TI * TJ * NRUN > 12 ? TI / 2 : TI;
  v4u resv[EPI != EPI_PLAIN ? TI : 1][EPI != EPI_PLAIN ? TJ : 1][NRUN];
  auto fetch_residual = [&](int m0, int n0, int i0, int i1) {
    if constexpr (EPI != EPI_PLAIN) {
      const int c = (n0 + wn * (BN / WN)) / (EPI == EPI_GATED ? 2 : 1);
      const int outs = EPI == EPI_GATED ? p.N >> 1 : p.N;
      const int ldb = (int)(p.ldr * 2);
      const __amdgpu_buffer_rsrc_t rR = buffer_rsrc(
          p.res + (int64_t)m0 * p.ldr + c, p.res ? max((min(BM, p.M - m0) - 1) * ldb + (outs - c) * 2, 0) : 0);
      int voff = (wm * (BM / WM) + l32) * ldb + 16 * lhi;
      asm volatile("" : "+v"(voff));                 // not kept across the matrix work, where registers are short
#pragma unroll
      for (int i = i0; i < i1; ++i)
#pragma unroll
        for (int j = 0; j < TJ; ++j)
#pragma unroll
          for (int u = 0; u < NRUN; ++u)
            resv[i][j][u] = __builtin_bit_cast(v4u, __builtin_amdgcn_raw_buffer_load_b128(
                rR, voff + 32 * i * ldb + 32 * (NRUN * j + u), 0, 0));
    }
  };

  // Output of the tile at (m0, n0) of K range pt.
  const int esz = OUT == OUT_16 ? 2 : 4;
  const float act_a = ACT == KIND_SIGMOID ? sigmoid_a(p.act) : p.act == ACT_RELU ? 0.0f : -__builtin_inff();
  const float act_b = sigmoid_b(p.act);
  auto pair16 = [&](float lo, float hi) -> uint32_t {
    if constexpr (BF) return bf16_rne(lo) | (uint32_t)bf16_rne(hi) << 16;
    return __half_as_ushort(__float2half_rn(lo)) | (uint32_t)__half_as_ushort(__float2half_rn(hi)) << 16;
  };
  auto store_tile = [&](int m0, int n0, int pt) {
    uint8_t* y = OUT == OUT_RAW ? reinterpret_cast<uint8_t*>(p.part + (int64_t)pt * p.M * p.part_ld)
                                : static_cast<uint8_t*>(p.y);
    const int64_t ldy = OUT == OUT_RAW ? p.part_ld : p.ldy;
    // WIDE: y's rows of this tile as one buffer (< 2^31 bytes, checked by the
    // host); a lane outside M x N gets an offset past it
    const int ldb = WIDE ? (int)(ldy * esz) : 0;
    const __amdgpu_buffer_rsrc_t rY = buffer_rsrc(y + (int64_t)m0 * ldy * esz, WIDE ? min(BM, p.M - m0) * ldb : 0);
#pragma unroll
    for (int i = 0; i < TI; ++i) {
      const int row = wm * (BM / WM) + 32 * i + l32;
      const float sa = OUT == OUT_RAW ? 0.0f : sas[row];
      if constexpr (EPI != EPI_PLAIN && EARLY < TI) {
        __builtin_amdgcn_sched_barrier(0);
        if (i > 0 && i + EARLY - 1 < TI) fetch_residual(m0, n0, i + EARLY - 1, i + EARLY);
      }
#pragma unroll
      for (int j = 0; j < TJ; ++j) {
        if constexpr (EPI != EPI_PLAIN) __builtin_amdgcn_sched_barrier(0);   // one block's temporaries at a time
        const int c0 = wn * (BN / WN) + 32 * j + 4 * lhi;      // channel of register 0
        uint32_t h[4][2];                                      // 16-bit pairs
        uint32_t res_run[4][2];                                // the residual of this lane's runs
        if constexpr (EPI == EPI_ACT) {
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const v4u d = resv[i][j][u];
            const auto s0 = __builtin_amdgcn_permlane32_swap(d[0], d[2], false, false);
            const auto s1 = __builtin_amdgcn_permlane32_swap(d[1], d[3], false, false);
            res_run[2 * u][0] = s0[0], res_run[2 * u + 1][0] = s0[1];
            res_run[2 * u][1] = s1[0], res_run[2 * u + 1][1] = s1[1];
          }
        } else if constexpr (EPI == EPI_GATED) {
          const v4u d = resv[i][j][0];
          const auto s0 = __builtin_amdgcn_permlane32_swap(d[0], d[1], false, false);
          const auto s1 = __builtin_amdgcn_permlane32_swap(d[2], d[3], false, false);
          res_run[0][0] = s0[0], res_run[2][0] = s0[1], res_run[1][0] = s1[0], res_run[3][0] = s1[1];
        }
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
          if constexpr (EPI != EPI_PLAIN) {
            float f[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              f[e] = __uint_as_float(w[e]);
              if (EPI == EPI_ACT || e % 2 == 0) {
                if constexpr (ACT == KIND_SIGMOID) f[e] = sigmoid_act(f[e], act_a, act_b);
                else if constexpr (ACT == KIND_ERF) f[e] = gelu_act(f[e]);
                else f[e] = f[e] < act_a ? 0.0f : f[e];
              }
            }
            if constexpr (EPI == EPI_GATED) {
              const uint32_t r = res_run[q][0];
              h[q][0] = pair16(plus(f[0] * f[1], lo_f32<BF>(r)), plus(f[2] * f[3], hi_f32<BF>(r)));
            } else {
#pragma unroll
              for (int e = 0; e < 2; ++e)
                h[q][e] = pair16(plus(f[2 * e], lo_f32<BF>(res_run[q][e])), plus(f[2 * e + 1], hi_f32<BF>(res_run[q][e])));
            }
          } else if constexpr (!WIDE) {
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
        if constexpr (EPI == EPI_GATED) {
          const auto s0 = __builtin_amdgcn_permlane32_swap(h[0][0], h[2][0], false, false);
          const auto s1 = __builtin_amdgcn_permlane32_swap(h[1][0], h[3][0], false, false);
          const int n = out_channel(n0, j, 0);
          __builtin_amdgcn_raw_buffer_store_b128(v4u{s0[0], s0[1], s1[0], s1[1]}, rY,
                                                 n < (p.N >> 1) ? row * ldb + n * 2 : kDroppedOffset, 0, 0);
        } else if constexpr (WIDE && OUT == OUT_16) {
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
      fetch_residual(m0, n0, 0, EARLY);
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
  fetch_residual(tile_m, tile_n, 0, EARLY);
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

// Which kernel, and into how many K ranges.
//
// Up to 16 tokens the W stream decides (k_w8a8_gemm_small; us there and in tiles, W
// from HBM: 16 x 28672 x 8192 48 and 57, 16 x 8192 x 28672 47.5 both, 16 x 18944 x 3584
// 16.9 and 20.0, 9 x the same 16.2 and 19.6, 16 x 4096 x 14336 15.5 and 22.4). Of 9 to 16
// tokens, few channels of long K go to tiles: 128 workgroups or fewer leave CUs idle
// while tiles split K (16 x 2048 x 53248 37.6 and 31.5, 16 x 1024 x 98304 63.8 and 35.9, 9 x
// the same 54.0 and 34.7, 9 x 2048 x 36864 27.8 and 24.1, 16 x 640 x 40960 26.9 and 19.8;
// shorter or wider: 16 x 2048 x 28672 21.7 and 22.5, 9 x 2304 x 40960 28.8 and 31.1, 16 x 1024
// x 16384 12.2 and 15.0). Some wide and long ones would gain in tiles, those that one round
// fills to 7/8, but their neighbours lose more (16 x 14336 x 20480 66.9 and 57.8, 28672 x
// 14336 83.5 and 74.8; 28672 x 11008 65.6 and 75.4, 27648 x 20480 119 and 128).
//
// Above 16 tokens and for those, the tile whose estimated time is least: rounds of tiles over
// the CUs times (stages x the tile's time per 128-k stage + its start and
// output). The times (us: 256 x 256 tiles 1.6 a stage, 256 x 128 0.95, 128 x 128
// 0.55) are fitted to measured shapes, tokens x channels x K, among them those named
// here, where the choice is the fastest; us of the three in turn: 4096 x 4096 x 4096
// 62.6, 70.7, 80.9; 1024 x 8192 x 28672 229, 224, 290; 512 x 8192 x 8192 74, 55.2,
// 43.4; 777 x 18944 x 3584 96.3, 84.2, 84.9; 2048 x 4096 x 11008 121, 88, 109. 128 x
// 128 tiles may also split K, which costs a launch and 8 bytes per output and range
// through the caches (64 x 8192 x 8192: 35.6 us whole, 25.5 in two ranges, 21.2 in
// four; 512 x 4096 x 11008: 53.8, 41.7, 50.1; 256 x 11008 x 4096: 24.1, 41.5, 44.7).
enum { TILE_SMALL = 0, TILE_256 = 1, TILE_256_128 = 2, TILE_128 = 3 };
struct W8Plan {
  int tile, splits;
  double us;              // the estimate
};
constexpr int64_t kFewChannels = 8 * kCUs, kLongK = 32768;
W8Plan plan_w8a8(int64_t M, int64_t N, int64_t K) {
  if (M <= 8 || (M <= 16 && (N > kFewChannels || K <= kLongK))) return W8Plan{TILE_SMALL, 1, 4.0 + N * K / 5.2e6};
  const int64_t nk = (K + 127) / 128;
  W8Plan best{TILE_256, 1, 1e30};
  auto consider = [&](int tile, int64_t bm, int64_t bn, double stage, double start, int splits) {
    const int64_t tiles = ((M + bm - 1) / bm) * ((N + bn - 1) / bn);
    const int64_t rounds = (tiles * splits + kCUs - 1) / kCUs;
    double us = rounds * (((nk + splits - 1) / splits) * stage + start);
    if (splits > 1) us += 4.0 + 8.0 * splits * M * N / 2.5e6;
    if (us < best.us) best = W8Plan{tile, splits, us};
  };
  consider(TILE_256, 256, 256, 1.6, 4.0, 1);
  consider(TILE_256_128, 256, 128, 0.95, 3.0, 1);
  for (int splits = 1; splits <= 16 && splits * 2 <= nk; splits *= 2)
    consider(TILE_128, 128, 128, 0.55, 2.5, splits);
  return best;
}

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
  p.part_ld = p.N;
  return p;
}

// 4 or 8 waves a workgroup. With 16 channels each, more than one a CU are better of 4 (W
// from HBM, us, 4 waves and 8: 9 x 6144 x 8192 13.4 and 14.7, 16 x 5120 x 27648 39.9 and
// 42.9, one token 6144 x 8192 12.3 and 13.8, 16 x 8192 x 8192 15.8 and 16.7; 16 x 4096 x 8192
// 11.6 and 10.0, one token 1024 x 8192 9.8 and 7.2), but for up to 4 tokens of the widest
// and longest W, which more loads in flight stream faster (one token 28672 x 8192 45.9
// and 42.2, 14336 x 8192 26.6 and 25.4, 28672 x 14336 79.9 and 75.2; 8 x 14336 x 8192 26.8 and
// 27.0, 16 x 14336 x 8192 27.9 and 29.0, one token 11008 x 8192 19.4 and 19.9).
bool four_waves(int64_t M, int64_t N, int64_t K) {
  return N > 16 * kCUs && !(M <= 4 && N >= 56 * kCUs && K >= 8192);
}
// Where a workgroup quantizes the tokens too, 8 waves up to twice as many channels (one
// token 5120 x 4096 7.4 with 8 and 7.8 with 4, 6144 x 28672 36.9 and 41.4).
bool four_waves_quantizing(int64_t N) { return N >= 32 * kCUs; }

// Whether the blocks of a quantizing workgroup of 4 waves may take LDS: 8 fit a CU, or
// all that there are (tokens x channels x K, us, turned and straight: 1 x 11008 x 4096 10.4
// and 11.1, 3 x 18944 x 4096 17.4 and 19.6, 4 x 18944 x 3584 16.7 and 18.4, 1 x 128256 x 512
// 17.6 and 18.9; where fewer fit, 4 x 18944 x 4096 21.0 and 20.2, 2 x 18944 x 8192 33.9 and
// 32.5, 8 x 28672 x 1024 12.3 and 10.7, 1 x 28672 x 8192 45.2 and 43.5).
bool turns_blocks(int64_t M, int64_t N, int64_t K) {
  const int64_t lds = 4 * 4096 + 128 + M * ((K + 63) / 64 * 64), fit = 160 * 1024 / lds;
  return fit >= 8 || (N + 15) / 16 <= fit * kCUs;
}

template <int XT, int PIECES, int EPI = EPI_PLAIN>
void launch_small(const W8Params& p, hipStream_t stream) {
  const dim3 grid((unsigned)((p.N + 15) / 16));
  const unsigned lds = XT ? (unsigned)(p.M * ((p.K + 63) / 64 * 64)) : 0;
#define W8A8_STREAM(NW, TURN) \
  hipLaunchKernelGGL((k_w8a8_gemm_small<XT, NW, PIECES, EPI, TURN>), grid, dim3(64 * NW), lds, stream, p)
  if constexpr (XT == 0) {
    if (four_waves(p.M, p.N, p.K)) W8A8_STREAM(4, true);
    else W8A8_STREAM(8, true);
  } else {
    if (!four_waves_quantizing(p.N)) W8A8_STREAM(8, true);
    else if (turns_blocks(p.M, p.N, p.K)) W8A8_STREAM(4, true);
    else W8A8_STREAM(4, false);
  }
#undef W8A8_STREAM
}

// Pieces of 1024 elements per wave that a workgroup of k_w8a8_gemm_small has to
// quantize for all tokens.
int64_t pieces_per_wave(int64_t M, int64_t N, int64_t K) {
  const int64_t nw = four_waves_quantizing(N) ? 4 : 8;
  return (M * ((K + 1023) / 1024) + nw - 1) / nw;
}

}  // namespace

}  // namespace w4a4
