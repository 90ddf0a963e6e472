// mhc_ffn_fwd.cu -- forward kernels of the gated feed-forward block.
#include "mhc_ffn_few.cuh"

namespace mhc {
namespace {

template <bool F16, int kKept>
cudaError_t gate_up(const FfnFwdLaunch& L, cudaStream_t s) {
  EpiGateUp<F16, kKept> e;
  e.a = static_cast<uint16_t*>(L.a_buf);
  e.gate_up = static_cast<uint16_t*>(L.gate_up);
  e.codes = static_cast<uint8_t*>(L.codes);
  e.scales = static_cast<uint8_t*>(L.scales);
  e.T = L.T;
  e.F = L.F;
  e.act = L.act;
  return launch_gemm<true, false, 1>({{L.x, L.wgu, L.gu}}, L.call, e, true, false, s);
}

template <bool F16>
cudaError_t forward(const FfnFwdLaunch& L, cudaStream_t s) {
  const cudaError_t e = L.kept == 0 ? gate_up<F16, 0>(L, s) : L.kept == 1 ? gate_up<F16, 1>(L, s) : gate_up<F16, 2>(L, s);
  if (e != cudaSuccess) return e;
  EpiStore<F16, 1> o;
  o.to[0] = {static_cast<uint16_t*>(L.y), L.T, L.D, L.part};
  const cudaError_t d = launch_gemm<false, false, 1>({{L.a, L.wd, L.down}}, L.call, o, false, true, s);
  return d != cudaSuccess || !L.part ? d : launch_sum<F16>(o.to[0], L.down.slices, L.call.sms, s);
}

template <bool F16, int kKept>
cudaError_t few_gate_up(const FfnFwdLaunch& L, cudaStream_t s) {
  FewGateUp<F16, kKept> e;
  e.a = static_cast<uint16_t*>(L.a_buf);
  e.gate_up = static_cast<uint16_t*>(L.gate_up);
  e.codes = static_cast<uint8_t*>(L.codes);
  e.scales = static_cast<uint8_t*>(L.scales);
  e.F = L.F;
  e.act = L.act;
  return launch_few(L.wgu, L.x, few_shape(L.gu, L.call, L.F, L.T, F16, false, true, false), e, s);
}

template <bool F16>
cudaError_t forward_few(const FfnFwdLaunch& L, cudaStream_t s) {
  const cudaError_t e = L.kept == 0   ? few_gate_up<F16, 0>(L, s)
                        : L.kept == 1 ? few_gate_up<F16, 1>(L, s)
                                      : few_gate_up<F16, 2>(L, s);
  if (e != cudaSuccess) return e;
  FewStore<F16> o;
  o.out = static_cast<uint16_t*>(L.y);
  o.N = L.D;
  return launch_few(L.wd, L.a, few_shape(L.down, L.call, L.D, L.T, F16, false, false, true), o, s);
}

}  // namespace

cudaError_t launch_ffn_forward(const FfnFwdLaunch& L, bool f16, cudaStream_t s) {
  if (L.T <= kFewTokens) return f16 ? forward_few<true>(L, s) : forward_few<false>(L, s);
  return f16 ? forward<true>(L, s) : forward<false>(L, s);
}

}  // namespace mhc
