// Device helpers of the INT8 quantizers (w8a8_quantize_act, kv8_append): the rule
// is a = max|x|, s = fl32(a / 127), q = rne(fl32(x / s)); s is NaN where a value
// of the row is a NaN or an infinity.
#pragma once

#include "quant_common.h"

namespace w4a4 {

// The fp32 value of the low / high 16-bit half of w.
template <bool BF>
__device__ __forceinline__ float lo_f32(uint32_t w) {
  if constexpr (BF) return __uint_as_float(w << 16);
  return (float)__builtin_bit_cast(h2, w).x;
}
template <bool BF>
__device__ __forceinline__ float hi_f32(uint32_t w) {
  if constexpr (BF) return __uint_as_float(w & 0xFFFF0000u);
  return (float)__builtin_bit_cast(h2, w).y;
}

// max |x| over the 16 values of two 16-byte words. The magnitude bits of both
// formats order as integers.
__device__ __forceinline__ uint32_t absmax16(const uint4 r[2], uint32_t m) {
  typedef unsigned short us2 __attribute__((ext_vector_type(2)));
  const uint32_t w[8] = {r[0].x, r[0].y, r[0].z, r[0].w, r[1].x, r[1].y, r[1].z, r[1].w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const us2 v = __builtin_bit_cast(us2, w[i] & 0x7FFF7FFFu);
    m = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(us2, m), v));
  }
  return m;
}

// The codes of 16 values. x / s is q0 = x r, e = fma(-q0, s, x),
// fma(e, r, q0) with r = RN(1/s): RN(x/s) (the correction of quant_common.h).
// k scales x (1, or a power of two that keeps a subnormal s out of the
// divisions; s and r are scaled alike). Adding 1.5 2^23 rounds to nearest even
// and leaves the two's-complement code in the low byte.
template <bool BF>
__device__ __forceinline__ uint4 codes16(const uint4 r[2], float k, float s, float rs) {
  const uint32_t w[8] = {r[0].x, r[0].y, r[0].z, r[0].w, r[1].x, r[1].y, r[1].z, r[1].w};
  uint32_t o[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t b[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      b[2 * i] = __float_as_uint(div_rn(lo_f32<BF>(w[2 * j + i]) * k, s, rs) + 12582912.0f);
      b[2 * i + 1] = __float_as_uint(div_rn(hi_f32<BF>(w[2 * j + i]) * k, s, rs) + 12582912.0f);
    }
    const uint32_t p01 = __builtin_amdgcn_perm(b[1], b[0], 0x0C0C0400u);
    const uint32_t p23 = __builtin_amdgcn_perm(b[3], b[2], 0x04000C0Cu);
    o[j] = p01 | p23;
  }
  return uint4{o[0], o[1], o[2], o[3]};
}

// The largest of the wave's absmax16 results, NaN if it is not finite. All of it on
// the bits, which order NaN above infinity above the numbers (a maximum of floats
// drops a NaN and what its lane had found beside it). Every lane must be active.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t m) {
  return max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, CTRL, 0xF, 0xF, false));
}
template <bool BF>
__device__ __forceinline__ float wave_absmax(uint32_t m) {
  m = max(m & 0xFFFFu, m >> 16);
  m = dpp_max<DPP_HALF_MIRROR>(m);
  m = dpp_max<DPP_QUAD_1032>(m);
  m = dpp_max<DPP_QUAD_2301>(m);
  m = dpp_max<DPP_ROW_MIRROR>(m);
  m = max(m, (uint32_t)__shfl_xor((int)m, 16));
  m = max(m, (uint32_t)__shfl_xor((int)m, 32));
  if constexpr (BF) return __uint_as_float((m >= 0x7F80u ? 0x7FC0u : m) << 16);
  return (float)__builtin_bit_cast(_Float16, (uint16_t)(m >= 0x7C00u ? 0x7E00u : m));
}
// Maximum of two such values, and of scales: none below 0, NaN stays.
__device__ __forceinline__ float max_or_nan(float a, float b) {
  return __uint_as_float(max(__float_as_uint(a), __float_as_uint(b)));
}
// The factor k that codes16 needs for s.
__device__ __forceinline__ float scale_guard(float s) { return s < 0x1p-60f ? 0x1p80f : 1.0f; }

}  // namespace w4a4
