// W8A8 linear layers for gfx950: INT8 quantization with one scale per token
// (weights: per output channel), and the matrix product on the INT8 matrix
// cores.
//
//   a = max_k |x|, s = fl32(a / 127), q = rne(fl32(x / s)) in [-127, 127]
//   P[m,n] = sum_k xq[m,k] wq[n,k]            (int32, exact for K <= 131056)
//   Y[m,n] = fl32(fl32(P) fl32(xs[m] ws[n])) + bias[n]
//
// The scales do not vary along K, so the whole reduction stays in the matrix
// cores' int32 accumulators and any split of K gives the same bits.
#include <algorithm>

#include "device.h"
#include "launch.h"
#include "quant_common.h"

namespace w4a4 {

namespace {

typedef int v16i __attribute__((ext_vector_type(16)));

constexpr int kThreads = 256;

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

// One row per WPR waves (256 / (64 WPR) rows a workgroup); NC > 0: the row's
// 16-element chunks stay in registers (NC per lane), so X is read once. NC = 0:
// rows of any length, read twice (the second time from cache).
template <bool BF, int WPR, int NC>
__global__ __launch_bounds__(kThreads) void k_w8a8_quant(const uint16_t* __restrict__ x, int64_t ldx, int64_t M, int K,
                                                         int8_t* __restrict__ q, float* __restrict__ s) {
  constexpr int RPB = kThreads / 64 / WPR;
  __shared__ uint32_t wave_max[kThreads / 64];
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
  const uint32_t mm = max(m & 0xFFFFu, m >> 16);
  float a = group_max<64>(BF ? __uint_as_float(mm << 16) : (float)__builtin_bit_cast(_Float16, (uint16_t)mm));
  if constexpr (WPR > 1) {
    if (lane == 0) wave_max[wave] = __float_as_uint(a);
    __syncthreads();
#pragma unroll
    for (int w = 0; w < WPR; ++w) a = fmaxf(a, __uint_as_float(wave_max[w]));
  }
  if (!live) return;
  const float sc = a / 127.0f;                     // correctly rounded
  const float k = BF && sc < 0x1p-60f ? 0x1p80f : 1.0f;
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
  const int8_t* a;
  const float* sa;
  const int8_t* w;
  const float* sw;
  const float* bias;          // or nullptr
  int M, N, K;
  void* y;
  int ydtype;
  int64_t ldy;
};

// Y value of an exact sum, and its store as ydt (0 fp32, 1 fp16, 2 bf16).
__device__ __forceinline__ float scaled(int p, float sa, float sw, float b) {
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

// ---- Few tokens: W streamed once from HBM straight into the operands --------
// A workgroup of NW waves owns 16 MT rows x 16 TN columns and splits K across
// its waves (contiguous runs of 64-k steps). v_mfma_i32_16x16x64_i8: lane l
// supplies 16 consecutive k of row l % 16 at k offset 16 (l / 16), so a step is
// one 16-byte load per operand and lane, with no LDS on the way; RING steps
// are in flight per wave. The waves' int32 sums meet in LDS (exact in any
// order). K is a multiple of 16: the last step's lanes beyond K read zeros.
template <int MT, int TN, int NW, int RING>
__global__ __launch_bounds__(64 * NW) void k_w8a8_gemm_small(W8Params p) {
  __shared__ int red[NW > 1 ? NW - 1 : 1][MT * TN * 4][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, g = lane >> 4;
  const int n0 = (int)blockIdx.x * 16 * TN, m0 = (int)blockIdx.y * 16 * MT;
  const int64_t K = p.K;
  const int steps = (p.K + 63) >> 6;
  const int h0 = (int)((int64_t)steps * wave / NW), h1 = (int)((int64_t)steps * (wave + 1) / NW);
  const int a_rows = min(16 * MT, p.M - m0), w_rows = min(16 * TN, p.N - n0);
  const __amdgpu_buffer_rsrc_t rA = buffer_rsrc(p.a + m0 * K, a_rows * p.K);
  const __amdgpu_buffer_rsrc_t rW = buffer_rsrc(p.w + n0 * K, w_rows * p.K);
  int offA[MT], offW[TN];
#pragma unroll
  for (int i = 0; i < MT; ++i) offA[i] = 16 * i + c < a_rows ? (16 * i + c) * p.K + 16 * g : kDroppedOffset;
#pragma unroll
  for (int j = 0; j < TN; ++j) offW[j] = 16 * j + c < w_rows ? (16 * j + c) * p.K + 16 * g : kDroppedOffset;
  struct Step {
    v4i a[MT], w[TN];
  };
  auto load = [&](Step& st, int h) {
    const bool in = 64 * h + 16 * g < p.K;
#pragma unroll
    for (int j = 0; j < TN; ++j)
      st.w[j] = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(rW, in ? offW[j] : kDroppedOffset, 64 * h, 0));
#pragma unroll
    for (int i = 0; i < MT; ++i)
      st.a[i] = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(rA, in ? offA[i] : kDroppedOffset, 64 * h, 0));
  };
  v4i acc[MT][TN];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = v4i{0, 0, 0, 0};
  Step ring[RING];
#pragma unroll
  for (int u = 0; u < RING; ++u)
    if (h0 + u < h1) load(ring[u], h0 + u);
  for (int h = h0; h < h1; h += RING) {
#pragma unroll
    for (int u = 0; u < RING; ++u) {
      if (h + u < h1) {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int j = 0; j < TN; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(ring[u].a[i], ring[u].w[j], acc[i][j], 0, 0, 0);
        if (h + u + RING < h1) load(ring[u], h + u + RING);
      }
    }
  }
  if constexpr (NW > 1) {
    if (wave > 0) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
          for (int r = 0; r < 4; ++r) red[wave - 1][(i * TN + j) * 4 + r][lane] = acc[i][j][r];
    }
    __syncthreads();
  }
  // one (row tile, column tile) pair per wave, in turn
  const int base = wave;
  if constexpr (NW > 1) {
    if (wave != 0) return;
  }
  (void)base;
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const int n = n0 + 16 * j + c;
      const float sw = n < p.N ? p.sw[n] : 0.0f;
      const float b = p.bias && n < p.N ? p.bias[n] : 0.0f;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        int v = acc[i][j][r];
        if constexpr (NW > 1) {
#pragma unroll
          for (int w = 0; w < NW - 1; ++w) v += red[w][(i * TN + j) * 4 + r][lane];
        }
        const int m = m0 + 16 * i + 4 * g + r;
        if (m < p.M && n < p.N) store_y(p.y, p.ydtype, m * p.ldy + n, scaled(v, p.sa[m], sw, b));
      }
    }
}

}  // namespace

void launch_w8a8_quant(const void* x, int bf16, int64_t M, int64_t K, int64_t ldx, int8_t* q, float* s,
                       hipStream_t stream) {
  const uint16_t* xp = static_cast<const uint16_t*>(x);
  if (bf16) launch_quant<true>(xp, M, K, ldx, q, s, stream);
  else launch_quant<false>(xp, M, K, ldx, q, s, stream);
}

void launch_w8a8_gemm(const W8GemmArgs& a, hipStream_t stream) {
  W8Params p;
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
  constexpr int MT = 1, TN = 1, NW = 8, RING = 4;
  const dim3 grid((unsigned)((a.N + 16 * TN - 1) / (16 * TN)), (unsigned)((a.M + 16 * MT - 1) / (16 * MT)));
  hipLaunchKernelGGL((k_w8a8_gemm_small<MT, TN, NW, RING>), grid, dim3(64 * NW), 0, stream, p);
}

}  // namespace w4a4
