// mhc_ffn_bwd.cu -- backward kernels of the gated feed-forward block.
#include "mhc_ffn_few.cuh"

namespace mhc {
namespace {

template <bool F16, int kKept>
cudaError_t dgate(const FfnBwdLaunch& L, cudaStream_t s) {
  EpiDgate<F16, kKept> e;
  e.gate_up = static_cast<const uint16_t*>(L.gate_up);
  e.codes = static_cast<const uint8_t*>(L.codes);
  e.scales = static_cast<const uint8_t*>(L.scales);
  e.gg = static_cast<uint16_t*>(L.gg_buf);
  e.a = static_cast<uint16_t*>(L.a_buf);
  e.T = L.T;
  e.F = L.F;
  e.act = L.act;
  return launch_gemm<false>(L.gy_k, L.wd_mn, L.ga, e, L.sms, s);
}

template <bool F16, int kKept>
cudaError_t few_dgate(const FfnBwdLaunch& L, cudaStream_t s) {
  FewDgate<F16, kKept> e;
  e.gate_up = static_cast<const uint16_t*>(L.gate_up);
  e.codes = static_cast<const uint8_t*>(L.codes);
  e.scales = static_cast<const uint8_t*>(L.scales);
  e.gg = static_cast<uint16_t*>(L.gg_buf);
  e.a = static_cast<uint16_t*>(L.a_buf);
  e.F = L.F;
  e.act = L.act;
  return launch_few(L.wd_mn, L.gy_k, few_shape(L.ga, L.F, L.T, F16, true), e, s);
}

template <bool F16>
cudaError_t backward(const FfnBwdLaunch& L, cudaStream_t s) {
  const bool few = L.T <= kFewTokens;
  cudaError_t e = few ? (L.kept == 1 ? few_dgate<F16, 1>(L, s) : few_dgate<F16, 2>(L, s))
                      : (L.kept == 1 ? dgate<F16, 1>(L, s) : dgate<F16, 2>(L, s));
  if (e != cudaSuccess) return e;
  EpiStore<F16> o;
  o.N = L.D;
  if (few) {
    FewStore<F16> f;
    f.out = static_cast<uint16_t*>(L.grad_x);
    f.N = L.D;
    e = launch_few(L.wgu_mn, L.gg_k, few_shape(L.gx, L.D, L.T, F16, true), f, s);
  } else {
    o.out = static_cast<uint16_t*>(L.grad_x);
    o.M = L.T;
    e = launch_gemm<false>(L.gg_k, L.wgu_mn, L.gx, o, L.sms, s);
  }
  if (e != cudaSuccess) return e;
  o.out = static_cast<uint16_t*>(L.grad_w_gate_up);
  o.M = 2 * L.F;
  if ((e = launch_gemm<false>(L.gg_mn, L.x_mn, L.gwgu, o, L.sms, s)) != cudaSuccess) return e;
  o.out = static_cast<uint16_t*>(L.grad_w_down);
  o.M = L.D;
  o.N = L.F;
  return launch_gemm<false>(L.gy_mn, L.a_mn, L.gwd, o, L.sms, s);
}

}  // namespace

cudaError_t launch_ffn_backward(const FfnBwdLaunch& L, bool f16, cudaStream_t s) {
  return f16 ? backward<true>(L, s) : backward<false>(L, s);
}

}  // namespace mhc
