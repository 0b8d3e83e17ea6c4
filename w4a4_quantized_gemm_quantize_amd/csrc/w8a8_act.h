// W8A8 products with an epilogue for gfx950: bias, activation (or the gate of two
// interleaved halves) and residual on the exact sums, rounded once to 16 bits.
//
//   v[m,n] = fl32(fl32(fl32(P) fl32(xs[m] ws[n])) + bias[n])
//   Y[m,n] = act(v[m,n]) + R[m,n],  or gated  act(v[m,2n]) v[m,2n+1] + R[m,n]
//
// The products are those of w8a8.hip, K split where its plan splits.
#pragma once

#include "w8a8_kernels.h"

namespace w4a4 {

namespace {

// Adds the K ranges' int32 sums and finishes them: a thread one output of every
// gridDim.y-th row.
template <int EPI>
__global__ __launch_bounds__(kThreads) void k_w8a8_join_act(W8Params p, int splits) {
  constexpr int C = EPI == EPI_GATED ? 2 : 1;              // channels of an output
  const int n = (int)blockIdx.x * kThreads + (int)threadIdx.x;
  if (C * n >= p.N) return;
  const int64_t plane = (int64_t)p.M * p.part_ld;
  float sw[C], b[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    sw[c] = p.sw[C * n + c];
    b[c] = p.bias ? p.bias[C * n + c] : 0.0f;
  }
  for (int64_t m = blockIdx.y; m < p.M; m += gridDim.y) {
    int v[C];
#pragma unroll
    for (int c = 0; c < C; ++c) v[c] = 0;
    const int32_t* at = p.part + m * p.part_ld + C * n;
    for (int s = 0; s < splits; ++s, at += plane) {
#pragma unroll
      for (int c = 0; c < C; ++c) v[c] += at[c];
    }
    const float sa = p.sa[m];
    float f[C];
#pragma unroll
    for (int c = 0; c < C; ++c) f[c] = scaled(v[c], sa, sw[c], b[c]);
    float y = activate(p.act, f[0]);
    if constexpr (EPI == EPI_GATED) y *= f[1];
    store_y(p.y, p.ydtype, m * p.ldy + n, plus(y, p.res ? load16(p.res, p.ydtype, m * p.ldr + n) : 0.0f));
  }
}

template <int BM, int BN, int WM, int WN, int S, int EPI>
void launch_tiles_act(W8Params p, hipStream_t stream) {
  const int64_t tiles = (int64_t)((p.M + BM - 1) / BM) * ((p.N + BN - 1) / BN);
  p.stages = (p.K + 127) / 128;
  const dim3 grid((unsigned)std::min<int64_t>(tiles, kCUs)), block(64 * WM * WN);
#define W8A8_ACT(KIND)                                                                                                   \
  if (p.ydtype == 1)                                                                                                     \
    hipLaunchKernelGGL((k_w8a8_gemm_tiles<BM, BN, WM, WN, S, OUT_16, true, EPI, KIND, false>), grid, block, 0, stream, p); \
  else                                                                                                                   \
    hipLaunchKernelGGL((k_w8a8_gemm_tiles<BM, BN, WM, WN, S, OUT_16, true, EPI, KIND, true>), grid, block, 0, stream, p)
  if (p.act == ACT_GELU) {
    W8A8_ACT(KIND_ERF);
  } else if (p.act == ACT_SILU || p.act == ACT_GELU_TANH) {
    W8A8_ACT(KIND_SIGMOID);
  } else {
    W8A8_ACT(KIND_LINEAR);
  }
#undef W8A8_ACT
}

// Ints per row of sums: whole 16-byte stores whatever the width.
int64_t sums_ld(int64_t N) { return (N + 3) & ~int64_t{3}; }

// int32 sums of `splits` K ranges into the workspace, then the join.
template <int EPI>
void launch_raw(W8Params p, int splits, hipStream_t stream) {
  const int64_t tiles = (int64_t)((p.M + 127) / 128) * ((p.N + 127) / 128);
  const int nk = (p.K + 127) / 128;
  p.stages = (nk + splits - 1) / splits;
  p.splits = splits = (nk + p.stages - 1) / p.stages;
  const int64_t blocks = tiles * splits;
  p.part_ld = (int)sums_ld(p.N);
  hipLaunchKernelGGL((k_w8a8_gemm_tiles<128, 128, 2, 2, 3, OUT_RAW, true>), dim3((unsigned)std::min<int64_t>(blocks, kCUs)),
                     dim3(256), 0, stream, p);
  const int64_t cols = (p.N / (EPI == EPI_GATED ? 2 : 1) + kThreads - 1) / kThreads;
  const int64_t rows = std::min<int64_t>(p.M, std::max<int64_t>(1, 8192 / cols));
  hipLaunchKernelGGL(k_w8a8_join_act<EPI>, dim3((unsigned)cols, (unsigned)rows), dim3(kThreads), 0, stream, p, splits);
}

W8Params act_params(const W8GemmArgs& g, const W8Epilogue& e) {
  W8Params p = params(g);
  p.act = e.act;
  p.res = static_cast<const uint16_t*>(e.residual);
  p.ldr = e.ldr;
  return p;
}

// Tiles that write outputs themselves need rows that take 16-byte stores; other
// rows, of odd widths or strides, go through the int32 sums, as K ranges do (written
// element by element instead: 4000 x 4084 x 1024 84.6 us for 73.2, 797 x 142 x 736 with
// a residual 31.6 for 15.8). Where
// few tokens follow a multiple of 256, they may take a launch of their own, so that
// they cost no further row of tiles (777 x 18944 x 3584 with GELU, us: 112.0, 96.6 and 99.6 in
// 256 x 256, 256 x 128 and 128 x 128 tiles, 63.7 + 18.9 as 768 and 9 tokens).
struct ActPlan {
  int64_t first;          // tokens of the first launch, all or a multiple of 256
  W8Plan plan, rest;
};
// K ranges for rows that go through the sums in any case: rounds of tiles, and the
// sums written and read (tokens x K x channels: 1210 x 2528 x 748 with SiLU and a
// residual 28.0 us in one range, 24.8 split; 797 x 736 x 142 12.5 and 11.4).
W8Plan plan_sums(int64_t M, int64_t N, int64_t K) {
  const int64_t nk = (K + 127) / 128, tiles = ((M + 127) / 128) * ((N + 127) / 128);
  W8Plan best{TILE_128, 1, 1e30};
  for (int splits = 1; splits <= 16 && (splits == 1 || splits * 2 <= nk); splits *= 2) {
    const double us = (tiles * splits + kCUs - 1) / kCUs * ((nk + splits - 1) / splits * 0.55 + 2.5) +
                      8.0 * splits * M * N / 2.5e6;
    if (us < best.us) best = W8Plan{TILE_128, splits, us};
  }
  return best;
}
ActPlan plan_act(int64_t M, int64_t N, int64_t K, bool wide) {
  ActPlan a = {M, plan_w8a8(M, N, K), {}};
  if (a.plan.tile == TILE_SMALL) return a;
  if (!wide) {
    a.plan = plan_sums(M, N, K);
    return a;
  }
  const int64_t m = M / 256 * 256;
  if (m > 0 && m < M) {
    const W8Plan x = plan_w8a8(m, N, K), y = plan_w8a8(M - m, N, K);
    if (x.us + y.us + 2.0 < 0.9 * a.plan.us) a = ActPlan{m, x, y};   // clear of the estimates' errors
  }
  return a;
}
bool sums_in_workspace(const W8Plan& pl, bool wide) { return pl.tile != TILE_SMALL && (pl.splits > 1 || !wide); }

template <int EPI>
void launch_plan(const W8Params& p, const W8Plan& pl, bool wide, hipStream_t stream) {
  if (pl.tile == TILE_SMALL) launch_small<0, 0, EPI>(p, stream);
  else if (sums_in_workspace(pl, wide)) launch_raw<EPI>(p, pl.splits, stream);
  else if (pl.tile == TILE_256) launch_tiles_act<256, 256, 2, 4, 2, EPI>(p, stream);
  else if (pl.tile == TILE_256_128) launch_tiles_act<256, 128, 4, 2, 3, EPI>(p, stream);
  else launch_tiles_act<128, 128, 2, 2, 3, EPI>(p, stream);
}

template <int EPI>
void launch_gemm_act(const W8GemmArgs& g, const W8Epilogue& e, hipStream_t stream) {
  W8Params p = act_params(g, e);
  p.part = static_cast<int32_t*>(g.workspace);
  const ActPlan a = plan_act(g.M, g.N, g.K, e.wide);
  p.M = (int)a.first;
  launch_plan<EPI>(p, a.plan, e.wide, stream);
  if (a.first == g.M) return;
  p.M = (int)(g.M - a.first);
  p.a += a.first * g.K;
  p.sa += a.first;
  p.y = static_cast<uint16_t*>(p.y) + a.first * p.ldy;
  if (p.res) p.res += a.first * p.ldr;
  launch_plan<EPI>(p, a.rest, e.wide, stream);
}

template <int EPI>
void launch_small_act(const W8GemmArgs& g, const W8Epilogue& e, const void* x, int bf16, int64_t ldx,
                      hipStream_t stream) {
  W8Params p = act_params(g, e);
  p.x = static_cast<const uint16_t*>(x);
  p.ldx = ldx;
  const int64_t pieces = pieces_per_wave(g.M, g.N, g.K);
#define W8A8_SMALL(PIECES) bf16 ? launch_small<2, PIECES, EPI>(p, stream) : launch_small<1, PIECES, EPI>(p, stream)
  if (pieces <= 1) W8A8_SMALL(1);
  else if (pieces <= 2) W8A8_SMALL(2);
  else W8A8_SMALL(4);
#undef W8A8_SMALL
}

}  // namespace

}  // namespace w4a4
