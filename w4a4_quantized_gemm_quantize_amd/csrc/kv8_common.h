// Arguments and device helpers of the INT8 key/value cache kernels (kv8_*).
#pragma once

#include "device.h"
#include "launch.h"
#include "quant_common.h"

namespace w4a4 {

typedef _Float16 v8h __attribute__((ext_vector_type(8)));

// A sequence of the batch: its n new tokens are tokens t0 .. t0 + n - 1 of the
// packed tensors and the last n of its len cached positions. Device values out
// of range (a cu_seqlens that runs backwards or past T, more new tokens than
// max_new, a length past the table or max_len) are cut, so no access leaves the
// caller's tensors or the workspace, whose size follows from the same bounds.
struct Seq {
  int t0, n, len;
};
__device__ __forceinline__ Seq sequence(const KvBatch& b, int i) {
  const int a = min(max(b.cu[i], 0), b.T), e = min(max(b.cu[i + 1], 0), b.T);
  return Seq{a, min(max(e - a, 0), b.max_new), min(max(b.lens[i], 0), b.max_len)};
}

// The page of a position, or -1 if the table's entry is no page of the pool.
__device__ __forceinline__ int page_of(const KvBatch& b, const KvPool& c, int seq, int pos) {
  const int pg = b.table[seq * b.table_ld + (pos >> c.log_page)];
  return (unsigned)pg < (unsigned)c.num_pages ? pg : -1;
}

__device__ __forceinline__ float f32_of(uint16_t v, bool bf) {
  return bf ? __uint_as_float((uint32_t)v << 16) : (float)__builtin_bit_cast(_Float16, v);
}
__device__ __forceinline__ uint16_t u16_of(float v, bool bf) {
  return bf ? __builtin_bit_cast(uint16_t, (__bf16)v) : __builtin_bit_cast(uint16_t, (_Float16)v);
}
// ydt: 0 fp32, 1 fp16, 2 bf16
__device__ __forceinline__ void store_as(void* y, int ydt, int64_t i, float v) {
  if (ydt == 0) static_cast<float*>(y)[i] = v;
  else static_cast<uint16_t*>(y)[i] = u16_of(v, ydt == 2);
}

}  // namespace w4a4
