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
  return launch_gemm<false, false, 1>({{L.gy_k, L.wd_mn, L.ga}}, L.call, e, true, false, s);
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
  return launch_few(L.wd_mn, L.gy_k, few_shape(L.ga, L.call, L.F, L.T, F16, true, true, false), e, s);
}

template <bool F16>
cudaError_t backward(const FfnBwdLaunch& L, cudaStream_t s) {
  const bool few = L.T <= kFewTokens;
  cudaError_t e = few ? (L.kept == 1 ? few_dgate<F16, 1>(L, s) : few_dgate<F16, 2>(L, s))
                      : (L.kept == 1 ? dgate<F16, 1>(L, s) : dgate<F16, 2>(L, s));
  if (e != cudaSuccess) return e;
  const GemmOperands gx = {L.gg_k, L.wgu_mn, L.gx}, gwgu = {L.gg_mn, L.x_mn, L.gwgu}, gwd = {L.gy_mn, L.a_mn, L.gwd};
  const StoreTo to_x = {static_cast<uint16_t*>(L.grad_x), L.T, L.D, L.part};
  const StoreTo to_wgu = {static_cast<uint16_t*>(L.grad_w_gate_up), 2 * L.F, L.D, L.part_gu};
  const StoreTo to_wd = {static_cast<uint16_t*>(L.grad_w_down), L.D, L.F, L.part_down};
  if (few) {
    FewStore<F16> f;
    f.out = to_x.out;
    f.N = L.D;
    e = launch_few(L.wgu_mn, L.gg_k, few_shape(L.gx, L.call, L.D, L.T, F16, true, false, false), f, s);
    if (e != cudaSuccess) return e;
    EpiStore<F16, 2> o;
    o.to[0] = to_wgu;
    o.to[1] = to_wd;
    return launch_gemm<false, false, 2>({{gwgu, gwd}}, L.call, o, false, true, s);
  }
  // The three products that follow are independent: one launch, tiles of the
  // deepest first.
  EpiStore<F16, 3> o;
  if (L.gx.kslice >= L.gwgu.kslice) {
    o.to[0] = to_x;
    o.to[1] = to_wgu;
    o.to[2] = to_wd;
    e = launch_gemm<false, true, 3>({{gx, gwgu, gwd}}, L.call, o, false, true, s);
  } else {
    o.to[0] = to_wgu;
    o.to[1] = to_wd;
    o.to[2] = to_x;
    e = launch_gemm<false, true, 3>({{gwgu, gwd, gx}}, L.call, o, false, true, s);
  }
  if (e == cudaSuccess && L.part) e = launch_sum<F16>(to_x, L.gx.slices, L.call.sms, s);
  if (e == cudaSuccess && L.part_gu) e = launch_sum<F16>(to_wgu, L.gwgu.slices, L.call.sms, s);
  if (e == cudaSuccess && L.part_down) e = launch_sum<F16>(to_wd, L.gwd.slices, L.call.sms, s);
  return e;
}

}  // namespace

cudaError_t launch_ffn_backward(const FfnBwdLaunch& L, bool f16, cudaStream_t s) {
  return f16 ? backward<true>(L, s) : backward<false>(L, s);
}

}  // namespace mhc
