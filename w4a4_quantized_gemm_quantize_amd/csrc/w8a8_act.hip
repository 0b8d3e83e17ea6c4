// The products with an activation, and what both kinds of epilogue share.
#include "w8a8_act.h"

namespace w4a4 {

bool w8a8_wide_rows(int64_t outs, const void* y, int64_t ldy, const void* residual, int64_t ldr) {
  auto fits = [](const void* p, int64_t ld) {
    return ld % 8 == 0 && 256 * ld * 2 < (int64_t{1} << 31) && (reinterpret_cast<uintptr_t>(p) & 15) == 0;
  };
  return outs % 8 == 0 && fits(y, ldy) && (!residual || fits(residual, ldr));
}

int64_t w8a8_act_workspace(int64_t M, int64_t N, int64_t K, bool wide) {
  const ActPlan a = plan_act(M, N, K, wide);
  auto sums = [&](int64_t m, const W8Plan& pl) { return sums_in_workspace(pl, wide) ? (int64_t)pl.splits * m * sums_ld(N) * 4 : 0; };
  const int64_t n = a.first == M ? sums(M, a.plan) : std::max(sums(a.first, a.plan), sums(M - a.first, a.rest));
  return wide ? n : std::max(n, w8a8_act_workspace(M, N, K, true));   // never less for other rows
}

void launch_w8a8_gemm_act(const W8GemmArgs& g, const W8Epilogue& e, hipStream_t stream) {
  if (e.gated) launch_w8a8_gemm_gated(g, e, stream);
  else launch_gemm_act<EPI_ACT>(g, e, stream);
}

void launch_w8a8_small_act(const W8GemmArgs& g, const W8Epilogue& e, const void* x, int bf16, int64_t ldx,
                           hipStream_t stream) {
  if (e.gated) launch_w8a8_small_gated(g, e, x, bf16, ldx, stream);
  else launch_small_act<EPI_ACT>(g, e, x, bf16, ldx, stream);
}

}  // namespace w4a4
