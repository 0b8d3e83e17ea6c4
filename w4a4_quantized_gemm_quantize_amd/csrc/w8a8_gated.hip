// The gated products, in a source of their own (each kind builds 18 tile kernels).
#include "w8a8_act.h"

namespace w4a4 {

void launch_w8a8_gemm_gated(const W8GemmArgs& g, const W8Epilogue& e, hipStream_t stream) {
  launch_gemm_act<EPI_GATED>(g, e, stream);
}

void launch_w8a8_small_gated(const W8GemmArgs& g, const W8Epilogue& e, const void* x, int bf16, int64_t ldx,
                             hipStream_t stream) {
  launch_small_act<EPI_GATED>(g, e, x, bf16, ldx, stream);
}

}  // namespace w4a4
