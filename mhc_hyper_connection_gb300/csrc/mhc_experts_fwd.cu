// mhc_experts_fwd.cu -- forward kernels of the routed experts.
#include "mhc_experts_gemm.cuh"

namespace mhc {
namespace {

// Rows of x in the plan's order.  The call's first launch: clears its header.
__global__ void __launch_bounds__(256) gather_kernel(uint32_t* header, const PlanView p, long long T, int k, int D,
                                                     const uint16_t* x, uint16_t* xs) {
  pdl_trigger();
  if (blockIdx.x == 0 && threadIdx.x < 8) header[threadIdx.x] = 0u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t segs = (uint32_t)(D + kGatherCols - 1) / kGatherCols, i = blockIdx.x * 8 + warp, n = i / segs;
  const int c0 = (int)(i - n * segs) * kGatherCols + lane * 8;
  if (n < T) {
    const int at = lane < k ? p.places[(size_t)n * k + lane] : -1;
    gather_item(k, at < p.cap_rows ? at : -1, c0, D, x + (size_t)n * D, xs);
  } else if (n < T + p.E) {
    int first, last;
    padding_rows(p, (int)(n - T), &first, &last);
    for (int r = first; r < last; ++r) zero_item(r, c0, D, xs);
  }
}

template <bool F16>
__global__ void __launch_bounds__(256, 4) combine_kernel(const PlanView p, long long T, int k, int D, const float* weights,
                                                      const uint16_t* hi, const uint8_t* lo, int lo_pitch, uint16_t* y) {
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, segs = (D + 255) / 256;
  const long long i = (long long)blockIdx.x * 8 + warp;
  if (i < T * segs)
    combine_item<F16>(i, segs, k, D, p.places, weights, p.cap_rows, hi, lo, lo_pitch, y, lane);
}

template <bool F16, bool kKept, int kAct>
cudaError_t gate_up(const ExpertsFwdLaunch& L, cudaStream_t s) {
  const auto job = experts_job<kRowsGateUp, F16>(L.wgu, L.x, L.plan, L.F, 128, L.D);
  const EpiExpertGateUp<F16, kKept, kAct> e = {static_cast<uint16_t*>(L.a_buf), static_cast<uint16_t*>(L.gate_up), L.F};
  return launch_group(job, grp_call(L.call, 1, false, token_rows(L.lay.width)), e, L.lay.cap_tiles * job.tiles_m, L.call.sms, true, s);
}

template <bool F16>
cudaError_t forward(const ExpertsFwdLaunch& L, cudaStream_t s) {
  cudaError_t e = launch_rows(gather_kernel, (L.T + L.E) * ((L.D + kGatherCols - 1) / kGatherCols), false, s, L.call.header, L.plan,
                              L.T, L.k, L.D, static_cast<const uint16_t*>(L.x_in), static_cast<uint16_t*>(L.xs));
  if (e != cudaSuccess) return e;
  e = L.act == 0 ? (L.gate_up ? gate_up<F16, true, 0>(L, s) : gate_up<F16, false, 0>(L, s))
                 : (L.gate_up ? gate_up<F16, true, 1>(L, s) : gate_up<F16, false, 1>(L, s));
  if (e != cudaSuccess) return e;
  const auto job = experts_job<kRowsK, F16>(L.wd, L.a, L.plan, L.D, kFfnTileM, L.F);
  const EpiRows o = {static_cast<uint16_t*>(L.xs), L.lo, L.D, rows_low_pitch(L.D)};
  e = launch_group(job, grp_call(L.call, 2, true, token_rows(L.lay.width)), o, L.lay.cap_tiles * job.tiles_m, L.call.sms, true, s);
  if (e != cudaSuccess) return e;
  return launch_rows(combine_kernel<F16>, L.T * ((L.D + 255) / 256), true, s, L.plan, L.T, L.k, L.D, L.weights,
                     static_cast<const uint16_t*>(L.xs), static_cast<const uint8_t*>(L.lo), rows_low_pitch(L.D),
                     static_cast<uint16_t*>(L.y));
}

}  // namespace

cudaError_t launch_experts_forward(const ExpertsFwdLaunch& L, bool f16, cudaStream_t s) {
  return f16 ? forward<true>(L, s) : forward<false>(L, s);
}

}  // namespace mhc
