// mhc_experts_api.cu -- host side of include/mhc_experts.h: argument checks, workspace
// layout and tensor maps.
#include "mhc_experts_gemm.cuh"
#include "mhc_host.cuh"
#include "../../include/mhc_experts.h"

using namespace mhc;

namespace {

size_t up256(size_t v) { return (v + 255) & ~size_t(255); }

mhc_status_t check_sizes(int64_t T, int64_t E, int64_t k, int64_t D, int64_t F) {
  size_t bytes;
  const mhc_status_t st = mhc_expert_plan_size(T, k, E, &bytes);
  if (st != MHC_OK) return st;
  if (D < 8 || D > 16384 || D % 8 != 0)
    return fail(MHC_ERR_PARAM_INVALID, "D must be a multiple of 8 in [8, 16384] (got %lld)", (long long)D);
  if (F < 8 || F > 16384 || F % 8 != 0)
    return fail(MHC_ERR_PARAM_INVALID, "F must be a multiple of 8 in [8, 16384] (got %lld)", (long long)F);
  return MHC_OK;
}

mhc_status_t check_common(int32_t dtype, int32_t act, uint32_t wait_us, int32_t withhold) {
  if (dtype != MHC_DTYPE_BF16 && dtype != MHC_DTYPE_FP16)
    return fail(MHC_ERR_PARAM_INVALID, "dtype must be MHC_DTYPE_BF16 or MHC_DTYPE_FP16 (got %d)", (int)dtype);
  if (act != MHC_FFN_SILU && act != MHC_FFN_GELU)
    return fail(MHC_ERR_PARAM_INVALID, "act must be MHC_FFN_SILU or MHC_FFN_GELU (got %d)", (int)act);
  if (wait_us > 10000000u) return fail(MHC_ERR_PARAM_INVALID, "wait_limit_us must be at most 10 s");
  if (withhold != 0 && withhold != 1) return fail(MHC_ERR_PARAM_INVALID, "withhold_copy must be 0 or 1");
  return MHC_OK;
}

// Tensor of 16-bit elements: extents from the contiguous one on, pitches of the
// others in elements; 128-byte swizzle, zeros outside.
bool map_nd(CUtensorMap* m, const void* base, bool f16, int rank, const uint64_t* dims, const uint64_t* pitch, const uint32_t* box) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t d[5], st[4];
  cuuint32_t b[5], es[5];
  for (int i = 0; i < rank; ++i) {
    d[i] = dims[i];
    b[i] = box[i];
    es[i] = 1;
    if (i) st[i - 1] = pitch[i - 1] * 2;
  }
  return fn(m, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void*>(base), d,
            st, b, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
bool map_rows(CUtensorMap* m, const void* base, bool f16, uint64_t cols, uint64_t rows, uint32_t box_rows) {
  const uint64_t d[2] = {cols, rows}, p[1] = {cols};
  const uint32_t b[2] = {64, box_rows};
  return map_nd(m, base, f16, 2, d, p, b);
}
bool map_tokens(CUtensorMap (&m)[4], const void* base, bool f16, uint64_t cols, uint64_t rows) {
  for (int i = 0; i < 4; ++i)
    if (!map_rows(&m[i], base, f16, cols, rows, 16u << i)) return false;
  return true;
}
// Columns in blocks of 64, a box of two blocks of 64 rows.  Where the columns are no multiple
// of 64 the last block runs into the next row (behind the last row: into what follows): it
// holds columns of the operand whose results are not stored.
bool map_blocks(CUtensorMap* m, const void* base, bool f16, uint64_t cols, uint64_t rows) {
  const uint64_t d[3] = {64, rows, (cols + 63) / 64}, p[2] = {cols, 64};
  const uint32_t b[3] = {64, kFfnBoxMn, 2};
  return map_nd(m, base, f16, 3, d, p, b);
}
// An expert's weights MN-major: in blocks where the columns are a multiple of 64 (*blocks =
// 1), else boxes of 64 columns.
bool map_weights_mn(CUtensorMap* m, int* blocks, const void* base, bool f16, uint64_t cols, uint64_t rows, uint64_t E) {
  *blocks = cols % 64 == 0;
  if (*blocks) {
    const uint64_t d[4] = {64, rows, cols / 64, E}, p[3] = {cols, 64, cols * rows};
    const uint32_t b[4] = {64, kFfnBoxMn, 2, 1};
    return map_nd(m, base, f16, 4, d, p, b);
  }
  const uint64_t d[3] = {cols, rows, E}, p[2] = {cols, cols * rows};
  const uint32_t b[3] = {64, kFfnBoxMn, 1};
  return map_nd(m, base, f16, 3, d, p, b);
}
bool map_weights(CUtensorMap* m, const void* base, bool f16, uint64_t cols, uint64_t rows, uint64_t E, uint32_t box_rows) {
  const uint64_t d[3] = {cols, rows, E}, p[2] = {cols, cols * rows};
  const uint32_t b[3] = {64, box_rows, 1};
  return map_nd(m, base, f16, 3, d, p, b);
}
// w_gate_up with eight rows of the gate and the same eight of up in turn.
bool map_gate_up(CUtensorMap* m, const void* base, bool f16, uint64_t D, uint64_t F, uint64_t E) {
  const uint64_t d[5] = {D, 8, 2, F / 8, E}, p[4] = {D, F * D, 8 * D, 2 * F * D};
  const uint32_t b[5] = {64, 8, 2, 8, 1};
  return map_nd(m, base, f16, 5, d, p, b);
}

struct FwdLayout {
  size_t xs, a, lo, total;
};
FwdLayout fwd_layout(const PlanLayout& p, int64_t D, int64_t F) {
  FwdLayout l;
  l.xs = 256;
  l.a = l.xs + up256((size_t)p.cap_rows * D * 2);
  l.lo = l.a + up256((size_t)p.cap_rows * F * 2);
  l.total = l.lo + up256((size_t)p.cap_rows * rows_low_pitch((int)D));
  return l;
}
struct BwdLayout {
  size_t xs, gys, gg, wa, w_row, part, room, total;
};
// An expert's sums have parts from this many rows on; each CTA then has a room of 128 x
// 256 fp32 sums.  For 152 CTAs whatever the device, so that sizes follow from the call's.
constexpr int64_t kPartRows = (int64_t)kGrpDeepest * kFfnTileK;
constexpr size_t kRoomBytes = (size_t)152 * 128 * 256 * 4;
BwdLayout bwd_layout(const PlanLayout& p, int64_t D, int64_t F) {
  BwdLayout l;
  l.xs = 256;
  l.gys = l.xs + up256((size_t)p.cap_rows * D * 2);
  l.gg = l.gys + up256((size_t)p.cap_rows * D * 2);
  l.wa = l.gg + up256((size_t)p.cap_rows * F * 4);
  l.w_row = l.wa + up256((size_t)p.cap_rows * F * 2);
  l.part = l.w_row + up256((size_t)p.cap_rows * 4);
  l.room = l.part + up256((size_t)p.cap_rows * ((F + 31) / 32) * 4);
  l.total = l.room + (p.slots > kPartRows ? kRoomBytes : 0) + 256;   // map_blocks reads a little past a buffer
  return l;
}

mhc_status_t device(int* sms) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return fail(MHC_ERR_RUNTIME, "no CUDA device");
  const DeviceInfo di = device_info(dev);
  if (!di.ok) return fail(MHC_ERR_RUNTIME, "device %d is not an sm_103 GPU", dev);
  *sms = di.sms;
  return MHC_OK;
}
ExpertsCall call(void* workspace, uint32_t wait_us, int withhold, int sms) {
  ExpertsCall c;
  c.header = static_cast<uint32_t*>(workspace);
  c.wait_ns = wait_us ? (uint64_t)wait_us * 1000u : 2000000000ull;
  c.withhold = withhold;
  c.sms = sms < 152 ? sms : 152;
  return c;
}

}  // namespace

extern "C" {

mhc_status_t mhc_experts_workspace_size(int64_t T, int64_t E, int64_t k, int64_t D, int64_t F, size_t* bytes) {
  clear_error();
  if (!bytes) return fail(MHC_ERR_NULLPTR, "bytes must be non-NULL");
  const mhc_status_t st = check_sizes(T, E, k, D, F);
  if (st != MHC_OK) return st;
  *bytes = T ? fwd_layout(plan_layout(T, k, E), D, F).total : 0;
  return MHC_OK;
}

mhc_status_t mhc_experts_backward_workspace_size(int64_t T, int64_t E, int64_t k, int64_t D, int64_t F, size_t* bytes) {
  clear_error();
  if (!bytes) return fail(MHC_ERR_NULLPTR, "bytes must be non-NULL");
  const mhc_status_t st = check_sizes(T, E, k, D, F);
  if (st != MHC_OK) return st;
  *bytes = T ? bwd_layout(plan_layout(T, k, E), D, F).total : 0;
  return MHC_OK;
}

mhc_status_t mhc_experts_run(const mhc_experts_args* a, void* stream) {
  clear_error();
  if (!a) return fail(MHC_ERR_NULLPTR, "args must be non-NULL");
  const int64_t T = a->T, E = a->E, k = a->k, D = a->D, F = a->F;
  mhc_status_t st = check_sizes(T, E, k, D, F);
  if (st == MHC_OK) st = check_common(a->dtype, a->act, a->wait_limit_us, a->withhold_copy);
  if (st != MHC_OK || T == 0) return st;
  if (!a->x || !a->weights || !a->plan || !a->w_gate_up || !a->w_down || !a->y || !a->workspace)
    return fail(MHC_ERR_NULLPTR, "x, weights, plan, w_gate_up, w_down, y and the workspace are required");
  const void* v16[] = {a->x, a->w_gate_up, a->w_down, a->y, a->gate_up};
  for (const void* p : v16)
    if (!aligned(p, 16)) return fail(MHC_ERR_PARAM_INVALID, "tensors must be 16-byte aligned");
  if (!aligned(a->weights, 4)) return fail(MHC_ERR_PARAM_INVALID, "weights must be 4-byte aligned");
  if (!aligned(a->workspace, 256) || !aligned(a->plan, 256))
    return fail(MHC_ERR_PARAM_INVALID, "workspace and plan must be 256-byte aligned");
  const PlanLayout p = plan_layout(T, k, E);
  const FwdLayout l = fwd_layout(p, D, F);
  if (a->workspace_bytes < l.total)
    return fail(MHC_ERR_PARAM_INVALID, "workspace too small: %zu bytes given, %zu needed", a->workspace_bytes, l.total);
  const size_t xb = (size_t)T * D * 2, wb = (size_t)E * F * D * 2;
  if ((st = check_apart({{"y", a->y, xb}, {"gate_up", a->gate_up, (size_t)p.cap_rows * F * 4}, {"workspace", a->workspace, l.total}},
                        {{"x", a->x, xb},
                         {"weights", a->weights, (size_t)p.slots * 4},
                         {"plan", a->plan, (size_t)p.total * 4},
                         {"w_gate_up", a->w_gate_up, 2 * wb},
                         {"w_down", a->w_down, wb}})) != MHC_OK)
    return st;
  int sms = 0;
  if ((st = device(&sms)) != MHC_OK) return st;
  const bool f16 = a->dtype == MHC_DTYPE_FP16;
  uint8_t* ws = static_cast<uint8_t*>(a->workspace);
  ExpertsFwdLaunch L;
  L.call = call(ws, a->wait_limit_us, a->withhold_copy, sms);
  L.plan = plan_view(p, E, const_cast<void*>(a->plan));
  L.lay = p;
  L.T = T;
  L.E = (int)E;
  L.k = (int)k;
  L.D = (int)D;
  L.F = (int)F;
  L.act = a->act;
  L.x_in = a->x;
  L.weights = a->weights;
  L.xs = ws + l.xs;
  L.a_buf = ws + l.a;
  L.lo = ws + l.lo;
  L.y = a->y;
  L.gate_up = a->gate_up;
  if (!map_gate_up(&L.wgu, a->w_gate_up, f16, D, F, E) || !map_weights(&L.wd, a->w_down, f16, F, D, E, kGemmHalf) ||
      !map_tokens(L.x, L.xs, f16, D, p.cap_rows) || !map_tokens(L.a, L.a_buf, f16, F, p.cap_rows))
    return fail(MHC_ERR_RUNTIME, "encoding a tensor map failed");
  const cudaError_t e = launch_experts_forward(L, f16, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(MHC_ERR_RUNTIME, "experts launch failed: %s", cudaGetErrorString(e));
  return MHC_OK;
}

mhc_status_t mhc_experts_backward_run(const mhc_experts_bwd_args* a, void* stream) {
  clear_error();
  if (!a) return fail(MHC_ERR_NULLPTR, "args must be non-NULL");
  const int64_t T = a->T, E = a->E, k = a->k, D = a->D, F = a->F;
  mhc_status_t st = check_sizes(T, E, k, D, F);
  if (st == MHC_OK) st = check_common(a->dtype, a->act, a->wait_limit_us, a->withhold_copy);
  if (st != MHC_OK) return st;
  if (!a->grad_w_gate_up || !a->grad_w_down) return fail(MHC_ERR_NULLPTR, "both weight gradients are required");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const size_t xb = (size_t)T * D * 2, wb = (size_t)E * F * D * 2;
  if (T == 0) {
    if ((st = check_apart({{"grad_w_gate_up", a->grad_w_gate_up, 2 * wb}, {"grad_w_down", a->grad_w_down, wb}},
                          {{"w_gate_up", a->w_gate_up, 2 * wb}, {"w_down", a->w_down, wb}})) != MHC_OK)
      return st;
    cudaError_t e = cudaMemsetAsync(a->grad_w_gate_up, 0, 2 * wb, s);
    if (e == cudaSuccess) e = cudaMemsetAsync(a->grad_w_down, 0, wb, s);
    if (e != cudaSuccess) return fail(MHC_ERR_RUNTIME, "clearing the weight gradients failed: %s", cudaGetErrorString(e));
    return MHC_OK;
  }
  if (!a->grad_y || !a->x || !a->weights || !a->plan || !a->w_gate_up || !a->w_down || !a->gate_up || !a->grad_x ||
      !a->grad_weights || !a->workspace)
    return fail(MHC_ERR_NULLPTR, "every tensor of the backward and the workspace are required");
  const void* v16[] = {a->grad_y, a->x, a->w_gate_up, a->w_down, a->gate_up, a->grad_x, a->grad_w_gate_up, a->grad_w_down};
  for (const void* p : v16)
    if (!aligned(p, 16)) return fail(MHC_ERR_PARAM_INVALID, "tensors must be 16-byte aligned");
  if (!aligned(a->weights, 4) || !aligned(a->grad_weights, 4))
    return fail(MHC_ERR_PARAM_INVALID, "weights and grad_weights must be 4-byte aligned");
  if (!aligned(a->workspace, 256) || !aligned(a->plan, 256))
    return fail(MHC_ERR_PARAM_INVALID, "workspace and plan must be 256-byte aligned");
  const PlanLayout p = plan_layout(T, k, E);
  const BwdLayout l = bwd_layout(p, D, F);
  if (a->workspace_bytes < l.total)
    return fail(MHC_ERR_PARAM_INVALID, "workspace too small: %zu bytes given, %zu needed", a->workspace_bytes, l.total);
  if ((st = check_apart({{"grad_x", a->grad_x, xb},
                         {"grad_weights", a->grad_weights, (size_t)p.slots * 4},
                         {"grad_w_gate_up", a->grad_w_gate_up, 2 * wb},
                         {"grad_w_down", a->grad_w_down, wb},
                         {"workspace", a->workspace, l.total}},
                        {{"grad_y", a->grad_y, xb},
                         {"x", a->x, xb},
                         {"weights", a->weights, (size_t)p.slots * 4},
                         {"plan", a->plan, (size_t)p.total * 4},
                         {"w_gate_up", a->w_gate_up, 2 * wb},
                         {"w_down", a->w_down, wb},
                         {"gate_up", a->gate_up, (size_t)p.cap_rows * F * 4}})) != MHC_OK)
    return st;
  int sms = 0;
  if ((st = device(&sms)) != MHC_OK) return st;
  const bool f16 = a->dtype == MHC_DTYPE_FP16;
  uint8_t* ws = static_cast<uint8_t*>(a->workspace);
  ExpertsBwdLaunch L;
  L.call = call(ws, a->wait_limit_us, a->withhold_copy, sms);
  L.plan = plan_view(p, E, const_cast<void*>(a->plan));
  L.lay = p;
  L.T = T;
  L.E = (int)E;
  L.k = (int)k;
  L.D = (int)D;
  L.F = (int)F;
  L.act = a->act;
  L.grad_y = a->grad_y;
  L.x_in = a->x;
  L.gate_up = a->gate_up;
  L.weights = a->weights;
  L.xs = ws + l.xs;
  L.gys = ws + l.gys;
  L.gg_buf = ws + l.gg;
  L.wa_buf = ws + l.wa;
  L.grad_x = a->grad_x;
  L.grad_w_gate_up = a->grad_w_gate_up;
  L.grad_w_down = a->grad_w_down;
  L.w_row = reinterpret_cast<float*>(ws + l.w_row);
  L.part = reinterpret_cast<float*>(ws + l.part);
  L.grad_weights = a->grad_weights;
  L.room = reinterpret_cast<float*>(ws + l.room);
  if (!map_weights_mn(&L.wd_mn, &L.wd_blocks, a->w_down, f16, F, D, E) ||
      !map_weights_mn(&L.wgu_mn, &L.wgu_blocks, a->w_gate_up, f16, D, 2 * F, E) || !map_tokens(L.gy, L.gys, f16, D, p.cap_rows) ||
      !map_tokens(L.gg, L.gg_buf, f16, 2 * F, p.cap_rows) || !map_blocks(&L.gg_mn, L.gg_buf, f16, 2 * F, p.cap_rows) ||
      !map_blocks(&L.xs_mn, L.xs, f16, D, p.cap_rows) || !map_blocks(&L.gy_mn, L.gys, f16, D, p.cap_rows) ||
      !map_blocks(&L.wa_mn, L.wa_buf, f16, F, p.cap_rows) || !map_rows(&L.xs_narrow, L.xs, f16, D, p.cap_rows, kFfnBoxMn) ||
      !map_rows(&L.wa_narrow, L.wa_buf, f16, F, p.cap_rows, kFfnBoxMn))
    return fail(MHC_ERR_RUNTIME, "encoding a tensor map failed");
  const cudaError_t e = launch_experts_backward(L, f16, s);
  if (e != cudaSuccess) return fail(MHC_ERR_RUNTIME, "experts backward launch failed: %s", cudaGetErrorString(e));
  return MHC_OK;
}

mhc_status_t mhc_experts_status(const void* workspace, void* stream) { return mhc_ffn_status(workspace, stream); }

}  // extern "C"
