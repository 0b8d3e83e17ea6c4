// RMS norm with INT8 output for gfx950: the residual's addition, the norm and the
// quantization of a W8A8 layer's input in one pass.
//
//   h = rne16(fl32(x + r))  (h = x without a residual),  t = fl32(h g),
//   rstd = 1 / sqrt(mean h^2 + eps),  a = max |t|,
//   q = rne(fl32(t / fl32(a / 127))) within -127 .. 127,  s = fl32(fl32(a rstd) / 127),
//   y = rne16(fl32(t rstd))
//
// q s stands for t rstd. The factor rstd > 0 is common to the row, so it leaves
// the codes as they are: sum and maximum come out of one pass and one reduction,
// and the codes depend on no rounding of a sum. h is rounded before the norm
// because that is what the residual stream holds afterwards. Sums are fp32: a lane's
// chunks of 16 squares, at most 4 of them in one chain, more with the rounding of each
// addition carried along (a row of 2^24 equal values was off by 6e-5 in one chain of 2^15
// squares a lane), then a tree. A row with a NaN or an infinity (in h or t) has scale NaN.
//
// Bound by HBM: 4096 x 8192 bf16 with a residual, 7 bytes per element, 42 to 48 us from card
// to card, 4.9 to 5.6 TB/s (a copy by PyTorch 5.3); without, 3 bytes, 24 to 27 us, 3.8 to 4.2
// TB/s (w8a8_quantize_act, which has no weights to read, 20.7 in the same loop); one row of 4096 2.7 us, a launch. Tried: weights
// kept in registers over several rows with the next row on its way 45.5 and 24.2 us, rows of
// 28672 slower (24.1 -> 27.3), not kept; non-temporal stores 46.9 and 20.0, but what reads
// the codes next pays more (the norm and a reader of the codes 122.8 -> 152.8).
#include "device.h"
#include "launch.h"
#include "quant8.h"

namespace w4a4 {

namespace {

template <bool BF>
__device__ __forceinline__ uint16_t to16(float v) {
  if constexpr (BF) return __builtin_bit_cast(uint16_t, (__bf16)v);
  return __builtin_bit_cast(uint16_t, (_Float16)v);
}
template <bool BF>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  return to16<BF>(lo) | (uint32_t)to16<BF>(hi) << 16;
}

// 16 weights at element i (W32: fp32, else of x's type).
template <bool BF, bool W32>
__device__ __forceinline__ void weights16(const void* w, int i, float g[16]) {
  if constexpr (W32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(w) + i);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float4 v = p[j];
      g[4 * j] = v.x; g[4 * j + 1] = v.y; g[4 * j + 2] = v.z; g[4 * j + 3] = v.w;
    }
  } else {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(w) + i);
    const uint4 a = p[0], b = p[1];
    const uint32_t u[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      g[2 * j] = lo_f32<BF>(u[j]);
      g[2 * j + 1] = hi_f32<BF>(u[j]);
    }
  }
}

constexpr int64_t kNormRows = int64_t{1} << 22;

struct NormParams {
  const uint16_t* x;
  const uint16_t* r;      // residual, or nullptr
  const void* w;
  uint16_t* h;            // the sum x + r (may be x or r itself); r != nullptr only
  uint16_t* y;            // the normed tokens, or nullptr
  int8_t* q;
  float* s;
  int64_t ldx, ldr, ldh, ldy, M;
  int K;
  float eps;
};

__device__ __forceinline__ float wave_sum(float v) {
  v += dpp<DPP_HALF_MIRROR>(v);
  v += dpp<DPP_QUAD_1032>(v);
  v += dpp<DPP_QUAD_2301>(v);
  v += dpp<DPP_ROW_MIRROR>(v);
  v += __shfl_xor(v, 16);
  v += __shfl_xor(v, 32);
  return v;
}
__device__ __forceinline__ uint32_t wave_max_bits(uint32_t m) {
  m = dpp_max<DPP_HALF_MIRROR>(m);
  m = dpp_max<DPP_QUAD_1032>(m);
  m = dpp_max<DPP_QUAD_2301>(m);
  m = dpp_max<DPP_ROW_MIRROR>(m);
  m = max(m, (uint32_t)__shfl_xor((int)m, 16));
  return max(m, (uint32_t)__shfl_xor((int)m, 32));
}

// One row per NW / RPB waves, RPB rows a workgroup of NW waves. NC > 0: the row's
// 16-element chunks stay in registers, NC a lane. NC = 0: rows of any length, read
// twice (the second time from cache).
template <bool BF, bool W32, bool RES, int NW, int RPB, int NC>
__global__ __launch_bounds__(64 * NW) void k_w8a8_rmsnorm(NormParams p) {
  constexpr int WPR = NW / RPB;
  __shared__ float sums[2][NW];
  __shared__ uint32_t maxs[NW];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t row = (int64_t)blockIdx.x * RPB + wave / WPR;
  const bool live = row < p.M;                     // WPR > 1 has one row per block: uniform
  const int t0 = (wave % WPR) * 64 + lane;
  const int n16 = live ? p.K >> 4 : 0;
  const uint4* x = reinterpret_cast<const uint4*>(p.x + (live ? row : 0) * p.ldx);
  const uint4* r = RES ? reinterpret_cast<const uint4*>(p.r + (live ? row : 0) * p.ldr) : nullptr;
  uint4* h = RES ? reinterpret_cast<uint4*>(p.h + (live ? row : 0) * p.ldh) : nullptr;

  auto add = [&](uint4 v[2], const uint4 u[2]) {   // v = rne16(v + u)
    uint32_t a[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
    const uint32_t b[8] = {u[0].x, u[0].y, u[0].z, u[0].w, u[1].x, u[1].y, u[1].z, u[1].w};
#pragma unroll
    for (int j = 0; j < 8; ++j) a[j] = pack16<BF>(lo_f32<BF>(a[j]) + lo_f32<BF>(b[j]), hi_f32<BF>(a[j]) + hi_f32<BF>(b[j]));
    v[0] = uint4{a[0], a[1], a[2], a[3]};
    v[1] = uint4{a[4], a[5], a[6], a[7]};
  };
  auto terms = [&](const uint4 v[2], const float g[16], float t[16]) {
    const uint32_t a[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      t[2 * j] = lo_f32<BF>(a[j]) * g[2 * j];
      t[2 * j + 1] = hi_f32<BF>(a[j]) * g[2 * j + 1];
    }
  };
  auto squares = [&](const uint4 v[2], float k, float sum) {
    const uint32_t a[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float lo = lo_f32<BF>(a[j]) * k, hi = hi_f32<BF>(a[j]) * k;
      sum = fmaf(lo, lo, sum);
      sum = fmaf(hi, hi, sum);
    }
    return sum;
  };

  // sum + part, where a lane sums many parts: `lost` is what the sums so far rounded away
  auto carry = [](float sum, float part, float& lost) {
    const float add = part - lost, s = sum + add;
    lost = s < __builtin_inff() ? s - sum - add : 0.0f;   // an infinite sum stays one
    return s;
  };

  uint4 raw[NC > 0 ? NC : 1][2];
  float sum = 0.0f, lost = 0.0f;
  uint32_t top = 0;
  auto first = [&](const uint4 v[2], int i) {
    float g[16], t[16];
    weights16<BF, W32>(p.w, 16 * i, g);
    terms(v, g, t);
    sum = NC > 0 ? squares(v, 1.0f, sum) : carry(sum, squares(v, 1.0f, 0.0f), lost);
#pragma unroll
    for (int j = 0; j < 16; ++j) top = max(top, __float_as_uint(t[j]) & 0x7FFFFFFFu);
  };
  if constexpr (NC > 0) {
    uint4 other[NC][2];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int i = c * 64 * WPR + t0;
      raw[c][0] = raw[c][1] = other[c][0] = other[c][1] = uint4{0, 0, 0, 0};
      if (i < n16) {
        raw[c][0] = x[2 * i];
        raw[c][1] = x[2 * i + 1];
        if constexpr (RES) {
          other[c][0] = r[2 * i];
          other[c][1] = r[2 * i + 1];
        }
      }
    }
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int i = c * 64 * WPR + t0;
      if (i < n16) {
        if constexpr (RES) {
          add(raw[c], other[c]);
          h[2 * i] = raw[c][0];
          h[2 * i + 1] = raw[c][1];
        }
        first(raw[c], i);
      }
    }
  } else {
    for (int i = t0; i < n16; i += 64 * WPR) {
      uint4 v[2] = {x[2 * i], x[2 * i + 1]};
      if constexpr (RES) {
        const uint4 u[2] = {r[2 * i], r[2 * i + 1]};
        add(v, u);
        h[2 * i] = v[0];
        h[2 * i + 1] = v[1];
      }
      first(v, i);
    }
  }
  // the row of h, read again by the lanes that wrote it
  const uint4* again = RES ? h : x;

  sum = wave_sum(sum);
  top = wave_max_bits(top);
  if constexpr (WPR > 1) {
    if (lane == 0) sums[0][wave] = sum, maxs[wave] = top;
    __syncthreads();
    sum = 0.0f;
#pragma unroll
    for (int w = 0; w < WPR; ++w) sum += sums[0][w], top = max(top, maxs[w]);
  }
  float rstd;
  if (BF && sum == __builtin_inff() && top < 0x7F800000u) {
    // squares past fp32's range: once more on 2^-80 h (of no use for fp16)
    float small = 0.0f;
    if constexpr (NC > 0) {
#pragma unroll
      for (int c = 0; c < NC; ++c) small = squares(raw[c], 0x1p-80f, small);   // chunks past the row are zeros
    } else {
      lost = 0.0f;
      for (int i = t0; i < n16; i += 64 * WPR) {
        const uint4 v[2] = {again[2 * i], again[2 * i + 1]};
        small = carry(small, squares(v, 0x1p-80f, 0.0f), lost);
      }
    }
    small = wave_sum(small);
    if constexpr (WPR > 1) {                       // the branch is the row's, so the block's
      if (lane == 0) sums[1][wave] = small;
      __syncthreads();
      small = 0.0f;
#pragma unroll
      for (int w = 0; w < WPR; ++w) small += sums[1][w];
    }
    rstd = 1.0f / sqrtf(small / (float)p.K) * 0x1p-80f;
  } else {
    rstd = 1.0f / sqrtf(sum / (float)p.K + p.eps);
  }
  if (!live) return;
  const float a = __uint_as_float(top >= 0x7F800000u ? 0x7FC00000u : top);
  const float st = a / 127.0f;
  const float k = scale_guard(st);
  const float sk = st * k;
  const float rs = st == 0.0f ? 0.0f : 1.0f / sk;
  uint4* dst = reinterpret_cast<uint4*>(p.q + row * p.K);
  uint4* y = p.y ? reinterpret_cast<uint4*>(p.y + row * p.ldy) : nullptr;
  auto second = [&](const uint4 v[2], int i) {
    float g[16], t[16];
    weights16<BF, W32>(p.w, 16 * i, g);
    terms(v, g, t);
    dst[i] = codes16f(t, k, sk, rs);
    if (y) {
      uint32_t o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = pack16<BF>(t[2 * j] * rstd, t[2 * j + 1] * rstd);
      y[2 * i] = uint4{o[0], o[1], o[2], o[3]};
      y[2 * i + 1] = uint4{o[4], o[5], o[6], o[7]};
    }
  };
  if constexpr (NC > 0) {
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int i = c * 64 * WPR + t0;
      if (i < n16) second(raw[c], i);
    }
  } else {
    for (int i = t0; i < n16; i += 64 * WPR) {
      const uint4 v[2] = {again[2 * i], again[2 * i + 1]};
      second(v, i);
    }
  }
  if (t0 == 0) p.s[row] = a == 0.0f ? 0.0f : a * rstd / 127.0f;
}

template <bool BF, bool W32, bool RES>
void launch_norm(const NormParams& p, hipStream_t stream) {
#define W8A8_NORM(NW, RPB, NC)                                                                       \
  hipLaunchKernelGGL((k_w8a8_rmsnorm<BF, W32, RES, NW, RPB, NC>), dim3((unsigned)((p.M + RPB - 1) / RPB)), \
                     dim3(64 * NW), 0, stream, p)
  // waves a row, chunks a lane (4096 x 8192 with a residual: 2 waves 53.6 us, 4 51.4, 8 47.7)
  if (p.K <= 1024) W8A8_NORM(4, 4, 1);
  else if (p.K <= 4096) W8A8_NORM(4, 1, 1);
  else if (p.K <= 8192) W8A8_NORM(8, 1, 1);
  else if (p.K <= 16384) W8A8_NORM(8, 1, 2);
  else if (p.K <= 32768) W8A8_NORM(8, 1, 4);
  else W8A8_NORM(8, 1, 0);
#undef W8A8_NORM
}

}  // namespace

void launch_w8a8_rmsnorm(const W8NormArgs& a, hipStream_t stream) {
  NormParams p;
  p.x = static_cast<const uint16_t*>(a.x);
  p.r = static_cast<const uint16_t*>(a.residual);
  p.w = a.weight;
  p.h = static_cast<uint16_t*>(a.h);
  p.y = static_cast<uint16_t*>(a.y);
  p.q = a.q;
  p.s = a.s;
  p.ldx = a.ldx; p.ldr = a.ldr; p.ldh = a.ldh; p.ldy = a.ldy;
  p.K = (int)a.K;
  p.eps = a.eps;
#define W8A8_NORM_OF(BF)                                                               \
  if (a.weight_f32) {                                                                  \
    if (p.r) launch_norm<BF, true, true>(p, stream); else launch_norm<BF, true, false>(p, stream);   \
  } else {                                                                             \
    if (p.r) launch_norm<BF, false, true>(p, stream); else launch_norm<BF, false, false>(p, stream); \
  }
  // up to 2^22 rows a launch, so that its threads stay under 2^32
  for (int64_t left = a.M; left > 0; left -= p.M) {
    p.M = left < kNormRows ? left : kNormRows;
    if (a.bf16) { W8A8_NORM_OF(true) } else { W8A8_NORM_OF(false) }
    p.x += p.M * p.ldx;
    if (p.r) p.r += p.M * p.ldr, p.h += p.M * p.ldh;
    if (p.y) p.y += p.M * p.ldy;
    p.q += p.M * p.K;
    p.s += p.M;
  }
#undef W8A8_NORM_OF
}

}  // namespace w4a4
