// mhc_experts_bwd.cu -- backward kernels of the routed experts.
#include "mhc_experts_gemm.cuh"

namespace mhc {
namespace {

// Rows of x and grad_y and the weights in the plan's order; zero rows of gg and w a
// where it is padding.  The call's first launch: clears its header.
__global__ void __launch_bounds__(256) gather_backward_kernel(uint32_t* header, const PlanView p, long long T, int k, int D,
                                                              int F, const uint16_t* x, const uint16_t* gy, const float* weights,
                                                              uint16_t* xs, uint16_t* gys, float* w_row, uint16_t* gg,
                                                              uint16_t* wa) {
  pdl_trigger();
  if (blockIdx.x == 0 && threadIdx.x < 8) header[threadIdx.x] = 0u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, widest = max(D, 2 * F);
  const uint32_t segs = (uint32_t)(D + kGatherCols - 1) / kGatherCols, i = blockIdx.x * 8 + warp;
  const uint32_t tokens = (uint32_t)T * segs;
  if (i < tokens) {
    const uint32_t n = i / segs;
    const int seg = (int)(i - n * segs), c0 = seg * kGatherCols + lane * 8;
    int at = lane < k ? p.places[(size_t)n * k + lane] : -1;
    if (at >= p.cap_rows) at = -1;
    if (seg == 0 && at >= 0) w_row[at] = weights[(size_t)n * k + lane];
    gather_item(k, at, c0, D, x + (size_t)n * D, xs);
    gather_item(k, at, c0, D, gy + (size_t)n * D, gys);
  } else {
    const uint32_t pieces = (uint32_t)(widest + kGatherCols - 1) / kGatherCols, n = (i - tokens) / pieces;
    const int seg = (int)(i - tokens - n * pieces), c0 = seg * kGatherCols + lane * 8;
    if (n >= (uint32_t)p.E) return;
    int first, last;
    padding_rows(p, (int)n, &first, &last);
    for (int r = first; r < last; ++r) {
      if (seg == 0 && lane == 0) w_row[r] = 0.0f;
      zero_item(r, c0, D, xs);
      zero_item(r, c0, D, gys);
      zero_item(r, c0, 2 * F, gg);
      zero_item(r, c0, F, wa);
    }
  }
}

// grad_x, and grad_weights from the parts of its sums: rows of the plan's order, one a
// lane; slots without a row get zeros.
template <bool F16>
__global__ void __launch_bounds__(256, 4) combine_backward_kernel(const PlanView p, long long T, int k, int D, int parts,
                                                               long long cap_rows, const uint16_t* hi, const uint8_t* lo, int lo_pitch,
                                                               const float* part,
                                                               uint16_t* grad_x, float* grad_weights) {
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, segs = (D + 255) / 256;
  const int used = min(p.head[1], p.cap_rows);
  const long long groups = (max(used, 0) + 31) / 32;
  const long long i = (long long)blockIdx.x * 8 + warp;
  if (i < T * segs + groups) {
    if (i < groups) {
      const long long r = i * 32 + lane;
      const int slot = r < used ? p.rows[r] : -1;
      if (slot >= 0 && slot < p.slots) {
        float sum = 0.0f;
#pragma unroll 8
        for (int n = 0; n < parts; ++n) sum += part[n * cap_rows + r];
        grad_weights[slot] = sum;
      }
    } else {
      const long long item = i - groups, t = item / segs;
      combine_item<F16>(item, segs, k, D, p.places, nullptr, p.cap_rows, hi, lo, lo_pitch, grad_x, lane);
      if (item == t * segs && lane < k && p.places[t * k + lane] < 0) grad_weights[t * k + lane] = 0.0f;
    }
  }
}

template <bool F16, int kAct>
cudaError_t gate_gradients(const ExpertsBwdLaunch& L, cudaStream_t s) {
  auto job = experts_job<kRowsMn, F16>(L.wd_mn, L.gy, L.plan, L.F, kFfnTileM, L.D);
  job.blocks = L.wd_blocks;
  const EpiExpertDgate<F16, kAct> o = {static_cast<const uint16_t*>(L.gate_up), L.w_row, static_cast<uint16_t*>(L.gg_buf),
                                       static_cast<uint16_t*>(L.wa_buf), L.part, L.F, L.lay.cap_rows};
  return launch_group(job, grp_call(L.call, 1, false, token_rows(L.lay.width)), o, L.lay.cap_tiles * job.tiles_m, L.call.sms, true, s);
}

template <bool F16>
cudaError_t backward(const ExpertsBwdLaunch& L, cudaStream_t s) {
  const int D = L.D, F = L.F, sms = L.call.sms, box = token_rows(L.lay.width);
  const int widest = D > 2 * F ? D : 2 * F;
  const long long gathers = L.T * ((D + kGatherCols - 1) / kGatherCols) + (long long)L.E * ((widest + kGatherCols - 1) / kGatherCols);
  cudaError_t e = launch_rows(gather_backward_kernel, gathers, false, s, L.call.header, L.plan, L.T, L.k, D, F, static_cast<const uint16_t*>(L.x_in), static_cast<const uint16_t*>(L.grad_y), L.weights,
                              static_cast<uint16_t*>(L.xs), static_cast<uint16_t*>(L.gys), L.w_row,
                              static_cast<uint16_t*>(L.gg_buf), static_cast<uint16_t*>(L.wa_buf));
  if (e != cudaSuccess) return e;
  if ((e = L.act == 0 ? gate_gradients<F16, 0>(L, s) : gate_gradients<F16, 1>(L, s)) != cudaSuccess) return e;
  {
    WeightGradJob<F16> job;
    job.a[0] = L.gg_mn;
    job.b[0] = L.xs_mn;
    job.a[1] = L.gy_mn;
    job.b[1] = L.wa_mn;
    job.narrow[0] = L.xs_narrow;
    job.narrow[1] = L.wa_narrow;
    job.counts = L.plan.counts;
    job.starts = L.plan.starts;
    job.E = L.E;
    job.cap_rows = L.plan.cap_rows;
    const int M[2] = {2 * F, D}, N[2] = {D, F};
    for (int i = 0; i < 2; ++i) {
      const int n256 = (N[i] + 255) / 256, w = (N[i] + n256 - 1) / n256;
      job.width[i] = w > 128 ? 256 : w > 64 ? 128 : 64;
      job.tiles_n[i] = (N[i] + job.width[i] - 1) / job.width[i];
      job.area[i] = (M[i] + kFfnTileM - 1) / kFfnTileM * job.tiles_n[i];
      job.by_n[i] = FastDiv((uint32_t)job.tiles_n[i]);
    }
    job.by_expert = FastDiv((uint32_t)(job.area[0] + job.area[1]));
    const EpiWeightGrad<F16> o = {{static_cast<uint16_t*>(L.grad_w_gate_up), static_cast<uint16_t*>(L.grad_w_down)},
                                  {M[0], M[1]}, {N[0], N[1]}, L.room};
    e = launch_group(job, grp_call(L.call, 2, false, 128), o, (long long)L.E * (job.area[0] + job.area[1]), sms, true, s);
    if (e != cudaSuccess) return e;
  }
  // rows of grad_x over those of x and of grad_y
  auto job = experts_job<kRowsMn, F16>(L.wgu_mn, L.gg, L.plan, D, kFfnTileM, 2 * F);
  job.blocks = L.wgu_blocks;
  const EpiRows o = {static_cast<uint16_t*>(L.xs), static_cast<uint8_t*>(L.gys), D, rows_low_pitch(D)};
  e = launch_group(job, grp_call(L.call, 3, true, box), o, L.lay.cap_tiles * job.tiles_m, sms, true, s);
  if (e != cudaSuccess) return e;
  return launch_rows(combine_backward_kernel<F16>, L.T * ((D + 255) / 256) + L.lay.cap_rows / 32 + 1, true, s, L.plan, L.T, L.k,
                     D, (F + 31) / 32, (long long)L.lay.cap_rows, static_cast<const uint16_t*>(L.xs), static_cast<const uint8_t*>(L.gys), rows_low_pitch(D),
                     static_cast<const float*>(L.part),
                     static_cast<uint16_t*>(L.grad_x), L.grad_weights);
}

}  // namespace

cudaError_t launch_experts_backward(const ExpertsBwdLaunch& L, bool f16, cudaStream_t s) {
  return f16 ? backward<true>(L, s) : backward<false>(L, s);
}

}  // namespace mhc
