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
#include "w8a8_kernels.h"

namespace w4a4 {

namespace {

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

}  // namespace

void launch_w8a8_quant(const void* x, int bf16, int64_t M, int64_t K, int64_t ldx, int8_t* q, float* s,
                       hipStream_t stream) {
  const uint16_t* xp = static_cast<const uint16_t*>(x);
  if (bf16) launch_quant<true>(xp, M, K, ldx, q, s, stream);
  else launch_quant<false>(xp, M, K, ldx, q, s, stream);
}

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

// Every workgroup quantizes all tokens, so it pays up to 4 pieces a wave and, of 4 waves,
// up to 8 tokens (tokens x channels x K, W from HBM, us, one launch and two: 1 x 11008 x 4096
// 10.4 and 13.4, 1 x 28672 x 8192 42.8 and 45.1, 4 x 11008 x 4096 (4 pieces) 13.0 and 14.2, 8 x
// 4096 x 4096 (4) 9.2 and 9.3, 8 x 28672 x 1024 (2) 10.7 and 11.6; with 8 pieces 8 x 11008 x
// 4096 17.6 and 14.6; 16 tokens in 4 waves, 16 x 11008 x 1024 9.4 and 7.9,
// 16 x 128256 x 1024 57.9 and 36.3, 16 x 28672 x 128 13.5 and 7.7; in 8, 16 x 4096 x 1024 5.6 and 6.4).
bool w8a8_one_launch(int64_t M, int64_t N, int64_t K) {
  return plan_w8a8(M, N, K).tile == TILE_SMALL && pieces_per_wave(M, N, K) <= 4 && (M <= 8 || !four_waves_quantizing(N));
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
