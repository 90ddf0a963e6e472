// mhc_ffn_api.cu -- host side of include/mhc_ffn.h: argument checks, workspace
// layout, tensor maps and the launches' shapes.
#include "mhc_ffn.cuh"
#include "mhc_host.cuh"
#include "../../include/mhc_ckpt.h"
#include "../../include/mhc_ffn.h"

using namespace mhc;

namespace {

size_t up256(size_t v) { return (v + 255) & ~size_t(255); }

mhc_status_t check_sizes(int64_t T, int64_t D, int64_t F) {
  if (T < 0 || T > (int64_t(1) << 24)) return fail(MHC_ERR_PARAM_INVALID, "T must be in [0, 2^24] (got %lld)", (long long)T);
  if (D < 8 || D > (int64_t(1) << 20) || D % 8 != 0)
    return fail(MHC_ERR_PARAM_INVALID, "D must be a multiple of 8 in [8, 2^20] (got %lld)", (long long)D);
  if (F < 8 || F > (int64_t(1) << 20) || F % 8 != 0)
    return fail(MHC_ERR_PARAM_INVALID, "F must be a multiple of 8 in [8, 2^20] (got %lld)", (long long)F);
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

// Tensor [rows, cols] (cols contiguous), planes of it behind one another; box
// of 64 columns x `box_rows` rows; zeros outside.
bool map_2d(CUtensorMap* m, const void* base, bool f16, uint64_t cols, uint64_t rows, uint64_t planes,
            uint32_t box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t d[3] = {cols, rows, planes};
  cuuint64_t st[2] = {cols * 2, planes > 1 ? cols * rows * 2 : cols * 2};
  cuuint32_t b[3] = {64, box_rows, 1};
  cuuint32_t es[3] = {1, 1, 1};
  return fn(m, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), d,
            st, b, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// How a product is cut into tiles: planned for 76 pairs of CTAs whatever the
// device, so that workspace sizes follow from T, D and F alone.
constexpr int64_t kPairs = 76;
struct Cut {
  int tile_n, slices, kslice;
};
int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Chunks of the depth (of 64) that one tile sums at most, where its product can be
// cut.  The tensor core truncates as it adds to its fp32 accumulators: 1e-7 of the
// running sum per sixteen products, all one way.  Terms of one sign measured 4.2e-4
// low at a depth of 65536 and 6.7e-3 at a million (weight gradients; fp16 rounds by
// 4.9e-4 at most); cut at 32768 and joined in fp32 they stay within 2.2e-4.
constexpr int64_t kDeepest = 512;

// Time of joining `slices` sums of M x N, in stages of a wide tile (0.28 us): a
// launch, and each sum written and read once.
double join_cost(int64_t M, int64_t N, int64_t slices) { return slices > 1 ? 10.0 + 8.0 * M * N * slices / 1.9e6 : 0.0; }

// A product that has its launch to itself: tiles 256, 192 or 128 wide and, where
// few tiles meet a deep product (most > 1), slices of the depth, by the estimated
// time of the rounds of tiles.  A stage of a narrow tile takes 0.6 of a wide one's
// time, with an MN-major B 0.7; of a tile 192 wide 0.8, with an MN-major B (which
// comes in blocks of 64, so as much is copied) what a wide one takes: only its
// epilogue is shorter.  Four wide stages are for a tile's start and end.  (T =
// 1021, D = 2048, F = 5512, down: 64 narrow tiles, forward 68 us where 32 wide ones
// took 75.5; T = 256, D = 4096, F = 8192, down in 2 slices: forward 70 -> 60 us; T =
// 1500, D = F = 4096, down: two rounds 192 wide where two of 256 took 119 us for the
// forward, now 104.5; T = 1021, D = 2048, F = 5512, gate gradients: 116 tiles 192
// wide, backward 5 us less.)
Cut cut_alone(int64_t M, int64_t N, int64_t K, bool b_mn, int most) {
  const int64_t kiters = div_up(K, kFfnTileK), rows = div_up(M, kFfnTileM);
  Cut best = {256, 1, (int)kiters};
  double least = 1e30;
  for (int w = 256; w >= 128; w -= 64) {
    const double stage = w == 256 ? 1.0 : w == 192 ? (b_mn ? 1.02 : 0.8) : b_mn ? 0.7 : 0.6;
    const double ends = w == 192 && b_mn ? 3.0 : 4.0 * stage;
    const int64_t fewest = most > 1 ? div_up(kiters, kDeepest) : 1;
    for (int64_t s = fewest; s == fewest || (s <= most && kiters >= 8 * s); ++s) {
      const int64_t per = div_up(kiters, s), slices = div_up(kiters, per);
      const double rounds = (double)div_up(rows * div_up(N, w) * slices, kPairs);
      const double cost = rounds * (per * stage + ends) + join_cost(M, N, slices);
      if (cost < least - 1e-9) {
        least = cost;
        best = {w, (int)slices, (int)per};
      }
    }
  }
  return best;
}

// grad_x beside the weight gradients in one launch: wide tiles, the depth sliced
// where one tile of it would outlast an equal share of the launch by more than the
// joining costs (T = 1956, D = 144, F = 8584, 4 slices: backward 173 -> 112 us; T =
// 512, D = 2048, F = 4096, 2 slices: 85 -> 68).
Cut cut_grad_x(int64_t T, int64_t D, int64_t F) {
  const int64_t kx = div_up(2 * F, kFfnTileK), kw = div_up(T, kFfnTileK);
  const int64_t total = div_up(T, 256) * div_up(D, 256) * kx + (div_up(2 * F, 256) * div_up(D, 256) + div_up(D, 256) * div_up(F, 256)) * kw;
  const int64_t share = div_up(total, kPairs);
  const int64_t fewest = div_up(kx, kDeepest);
  int64_t s = div_up(kx, share);
  if (s > 16) s = 16;
  while (s > 1 && kx < 8 * s) --s;
  if (s < fewest) s = fewest;
  const int64_t per = div_up(kx, s), slices = div_up(kx, per);
  const int64_t then = per > share ? per : share;
  if (fewest == 1 && (slices == 1 || kx - then < join_cost(T, D, slices))) return {256, 1, (int)kx};
  return {256, (int)slices, (int)per};
}
// The weight gradients: sums over the tokens.
Cut cut_tokens(int64_t T) {
  const int64_t kiters = div_up(T, kFfnTileK), per = div_up(kiters, div_up(kiters, kDeepest));
  return {256, (int)div_up(kiters, per), (int)per};
}
Cut whole(int64_t K) { return {256, 1, (int)div_up(K, kFfnTileK)}; }
constexpr int kMostSlices = 16;

struct FwdLayout {
  size_t a, part, total;
};
// Sums of the slices of a product with M x N outputs.
size_t part_bytes(const Cut& c, int64_t M, int64_t N) { return c.slices > 1 ? up256((size_t)c.slices * M * N * 4) : 0; }
Cut cut_down(int64_t T, int64_t D, int64_t F) { return T <= kFewTokens ? whole(F) : cut_alone(T, D, F, false, kMostSlices); }
Cut cut_gx(int64_t T, int64_t D, int64_t F) { return T <= kFewTokens ? whole(2 * F) : cut_grad_x(T, D, F); }

FwdLayout fwd_layout(int64_t T, int64_t D, int64_t F) {
  FwdLayout l;
  l.a = 256;
  l.part = l.a + up256((size_t)T * F * 2);
  l.total = l.part + part_bytes(cut_down(T, D, F), T, D);
  return l;
}
struct BwdLayout {
  size_t gg, a, part, part_gu, part_down, total;
};
BwdLayout bwd_layout(int64_t T, int64_t D, int64_t F) {
  BwdLayout l;
  l.gg = 256;
  l.a = l.gg + up256((size_t)T * F * 4);
  l.part = l.a + up256((size_t)T * F * 2);
  l.part_gu = l.part + part_bytes(cut_gx(T, D, F), T, D);
  l.part_down = l.part_gu + part_bytes(cut_tokens(T), 2 * F, D);
  l.total = l.part_down + part_bytes(cut_tokens(T), D, F);
  return l;
}

// pair_of: rows of B come from two planes (gate and up), 128 columns a tile.
GemmShape shape(int64_t M, int64_t N, int64_t K, const Cut& cut, bool pair_of, bool f16, bool a_mn, bool b_mn) {
  GemmShape g;
  g.tile_n = cut.tile_n;
  const int64_t step = pair_of ? 128 : g.tile_n;
  g.tiles_m = (int)div_up(M, kFfnTileM);
  g.tiles_n = (int)div_up(N, step);
  g.slices = cut.slices;
  g.kiters = (int)div_up(K, kFfnTileK);
  g.kslice = cut.kslice;
  // A band of at most 32 MB of A stays in L2 while B passes by (T = 4096, D =
  // 4096, F = 8192 forward: 506 us with 8 tile rows, 490 with these 16).
  const int64_t row_bytes = K * 2 * kFfnTileM;
  g.band = (int)((int64_t(32) << 20) / row_bytes);
  g.band = g.band < 4 ? 4 : g.band > 16 ? 16 : g.band;
  g.by_area = FastDiv((uint32_t)(g.tiles_m * g.tiles_n));
  g.by_band = FastDiv((uint32_t)(g.band * g.tiles_n));
  g.by_rows = FastDiv((uint32_t)g.band);
  g.by_last = FastDiv((uint32_t)(g.tiles_m % g.band ? g.tiles_m % g.band : g.band));
  g.a_mn = a_mn;
  g.b_mn = b_mn;
  g.idesc = (f16 ? (1u << 4) : ((1u << 4) | (1u << 7) | (1u << 10))) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) |
            ((uint32_t)(g.tile_n >> 3) << 17) | ((uint32_t)(kFfnTileM >> 4) << 24);
  return g;
}

FfnCall call(uint32_t* err, uint32_t wait_us, int withhold, int sms) {
  FfnCall c;
  c.err = err;
  c.wait_ns = wait_us ? (uint64_t)wait_us * 1000u : 2000000000ull;
  c.withhold = withhold;
  c.sms = sms;
  return c;
}

mhc_status_t device(int* sms) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return fail(MHC_ERR_RUNTIME, "no CUDA device");
  const DeviceInfo di = device_info(dev);
  if (!di.ok) return fail(MHC_ERR_RUNTIME, "device %d is not an sm_103 GPU", dev);
  *sms = di.sms;
  return MHC_OK;
}

}  // namespace

extern "C" {

mhc_status_t mhc_ffn_workspace_size(int64_t T, int64_t D, int64_t F, size_t* bytes) {
  clear_error();
  if (!bytes) return fail(MHC_ERR_NULLPTR, "bytes must be non-NULL");
  const mhc_status_t st = check_sizes(T, D, F);
  if (st != MHC_OK) return st;
  *bytes = T ? fwd_layout(T, D, F).total : 0;
  return MHC_OK;
}

mhc_status_t mhc_ffn_backward_workspace_size(int64_t T, int64_t D, int64_t F, size_t* bytes) {
  clear_error();
  if (!bytes) return fail(MHC_ERR_NULLPTR, "bytes must be non-NULL");
  const mhc_status_t st = check_sizes(T, D, F);
  if (st != MHC_OK) return st;
  *bytes = T ? bwd_layout(T, D, F).total : 0;
  return MHC_OK;
}

mhc_status_t mhc_ffn_run(const mhc_ffn_args* a, void* stream) {
  clear_error();
  if (!a) return fail(MHC_ERR_NULLPTR, "args must be non-NULL");
  const int64_t T = a->T, D = a->D, F = a->F;
  mhc_status_t st = check_sizes(T, D, F);
  if (st == MHC_OK) st = check_common(a->dtype, a->act, a->wait_limit_us, a->withhold_copy);
  if (st != MHC_OK || T == 0) return st;
  if (!a->x || !a->w_gate_up || !a->w_down || !a->y || !a->workspace)
    return fail(MHC_ERR_NULLPTR, "x, w_gate_up, w_down, y and the workspace are required");
  if ((a->codes == nullptr) != (a->scales == nullptr))
    return fail(MHC_ERR_PARAM_INVALID, "codes and scales go together (both or neither)");
  if (a->gate_up && a->codes) return fail(MHC_ERR_PARAM_INVALID, "give gate_up or codes, not both");
  const void* v16[] = {a->x, a->w_gate_up, a->w_down, a->y, a->gate_up, a->codes};
  for (const void* p : v16)
    if (!aligned(p, 16)) return fail(MHC_ERR_PARAM_INVALID, "tensors must be 16-byte aligned");
  if (!aligned(a->workspace, 256)) return fail(MHC_ERR_PARAM_INVALID, "the workspace must be 256-byte aligned");
  const FwdLayout l = fwd_layout(T, D, F);
  if (a->workspace_bytes < l.total)
    return fail(MHC_ERR_PARAM_INVALID, "workspace too small: %zu bytes given, %zu needed", a->workspace_bytes, l.total);
  const size_t xb = (size_t)T * D * 2, wb = (size_t)F * D * 2, kb = (size_t)T * F * 2, blocks = div_up(F, MHC_CKPT_BLOCK);
  if ((st = check_apart({{"y", a->y, xb},
                         {"gate_up", a->gate_up, 2 * kb},
                         {"codes", a->codes, kb},
                         {"scales", a->scales, (size_t)T * 2 * blocks},
                         {"workspace", a->workspace, l.total}},
                        {{"x", a->x, xb}, {"w_gate_up", a->w_gate_up, 2 * wb}, {"w_down", a->w_down, wb}})) != MHC_OK)
    return st;
  FfnFwdLaunch L;
  int sms = 0;
  if ((st = device(&sms)) != MHC_OK) return st;
  const bool f16 = a->dtype == MHC_DTYPE_FP16;
  uint8_t* ws = static_cast<uint8_t*>(a->workspace);
  L.call = call(reinterpret_cast<uint32_t*>(ws), a->wait_limit_us, a->withhold_copy, sms);
  L.T = (int)T;
  L.D = (int)D;
  L.F = (int)F;
  L.act = a->act;
  L.kept = a->gate_up ? 1 : a->codes ? 2 : 0;
  L.a_buf = ws + l.a;
  L.y = a->y;
  L.gate_up = a->gate_up;
  L.codes = a->codes;
  L.scales = a->scales;
  L.gu = shape(T, F, D, whole(D), true, f16, false, false);
  L.down = shape(T, D, F, cut_down(T, D, F), false, f16, false, false);
  L.part = L.down.slices > 1 ? reinterpret_cast<float*>(ws + l.part) : nullptr;
  const bool few = T <= kFewTokens;
  const uint32_t tok_box = few ? (uint32_t)((T + 15) & ~int64_t(15)) : kFfnBoxK;
  if (!map_2d(&L.x, a->x, f16, D, T, 1, tok_box) || !map_2d(&L.wgu, a->w_gate_up, f16, D, F, 2, kFfnBoxK) ||
      !map_2d(&L.a, L.a_buf, f16, F, T, 1, tok_box) ||
      !map_2d(&L.wd, a->w_down, f16, F, D, 1, few ? kFfnBoxK : (uint32_t)L.down.tile_n / 2))
    return fail(MHC_ERR_RUNTIME, "encoding a tensor map failed");
  const cudaError_t e = launch_ffn_forward(L, f16, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(MHC_ERR_RUNTIME, "feed-forward launch failed: %s", cudaGetErrorString(e));
  return MHC_OK;
}

mhc_status_t mhc_ffn_backward_run(const mhc_ffn_bwd_args* a, void* stream) {
  clear_error();
  if (!a) return fail(MHC_ERR_NULLPTR, "args must be non-NULL");
  const int64_t T = a->T, D = a->D, F = a->F;
  mhc_status_t st = check_sizes(T, D, F);
  if (st == MHC_OK) st = check_common(a->dtype, a->act, a->wait_limit_us, a->withhold_copy);
  if (st != MHC_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (!a->grad_w_gate_up || !a->grad_w_down) return fail(MHC_ERR_NULLPTR, "both weight gradients are required");
  if (T == 0) {
    cudaError_t e = cudaMemsetAsync(a->grad_w_gate_up, 0, (size_t)D * F * 4, s);
    if (e == cudaSuccess) e = cudaMemsetAsync(a->grad_w_down, 0, (size_t)D * F * 2, s);
    if (e != cudaSuccess) return fail(MHC_ERR_RUNTIME, "clearing the weight gradients failed: %s", cudaGetErrorString(e));
    return MHC_OK;
  }
  if (!a->grad_y || !a->x || !a->w_gate_up || !a->w_down || !a->grad_x || !a->workspace)
    return fail(MHC_ERR_NULLPTR, "grad_y, x, w_gate_up, w_down, grad_x and the workspace are required");
  if ((a->codes == nullptr) != (a->scales == nullptr))
    return fail(MHC_ERR_PARAM_INVALID, "codes and scales go together (both or neither)");
  if (!a->gate_up && !a->codes) return fail(MHC_ERR_NULLPTR, "gate_up or codes and scales are required");
  if (a->gate_up && a->codes) return fail(MHC_ERR_PARAM_INVALID, "give gate_up or codes, not both");
  const void* v16[] = {a->grad_y, a->x, a->w_gate_up, a->w_down, a->gate_up, a->codes,
                       a->grad_x, a->grad_w_gate_up, a->grad_w_down};
  for (const void* p : v16)
    if (!aligned(p, 16)) return fail(MHC_ERR_PARAM_INVALID, "tensors must be 16-byte aligned");
  if (!aligned(a->workspace, 256)) return fail(MHC_ERR_PARAM_INVALID, "the workspace must be 256-byte aligned");
  const BwdLayout l = bwd_layout(T, D, F);
  if (a->workspace_bytes < l.total)
    return fail(MHC_ERR_PARAM_INVALID, "workspace too small: %zu bytes given, %zu needed", a->workspace_bytes, l.total);
  const size_t xb = (size_t)T * D * 2, wb = (size_t)F * D * 2, kb = (size_t)T * F * 2, blocks = div_up(F, MHC_CKPT_BLOCK);
  if ((st = check_apart({{"grad_x", a->grad_x, xb},
                         {"grad_w_gate_up", a->grad_w_gate_up, 2 * wb},
                         {"grad_w_down", a->grad_w_down, wb},
                         {"workspace", a->workspace, l.total}},
                        {{"grad_y", a->grad_y, xb},
                         {"x", a->x, xb},
                         {"w_gate_up", a->w_gate_up, 2 * wb},
                         {"w_down", a->w_down, wb},
                         {"gate_up", a->gate_up, 2 * kb},
                         {"codes", a->codes, kb},
                         {"scales", a->scales, (size_t)T * 2 * blocks}})) != MHC_OK)
    return st;
  FfnBwdLaunch L;
  int sms = 0;
  if ((st = device(&sms)) != MHC_OK) return st;
  const bool f16 = a->dtype == MHC_DTYPE_FP16;
  uint8_t* ws = static_cast<uint8_t*>(a->workspace);
  L.call = call(reinterpret_cast<uint32_t*>(ws), a->wait_limit_us, a->withhold_copy, sms);
  L.T = (int)T;
  L.D = (int)D;
  L.F = (int)F;
  L.act = a->act;
  L.kept = a->gate_up ? 1 : 2;
  L.gate_up = a->gate_up;
  L.codes = a->codes;
  L.scales = a->scales;
  L.gg_buf = ws + l.gg;
  L.a_buf = ws + l.a;
  L.grad_x = a->grad_x;
  L.grad_w_gate_up = a->grad_w_gate_up;
  L.grad_w_down = a->grad_w_down;
  const uint32_t tok_box = T <= kFewTokens ? (uint32_t)((T + 15) & ~int64_t(15)) : kFfnBoxK;
  if (!map_2d(&L.gy_k, a->grad_y, f16, D, T, 1, tok_box) || !map_2d(&L.wd_mn, a->w_down, f16, F, D, 1, kFfnBoxMn) ||
      !map_2d(&L.gg_k, L.gg_buf, f16, 2 * F, T, 1, tok_box) || !map_2d(&L.wgu_mn, a->w_gate_up, f16, D, 2 * F, 1, kFfnBoxMn) ||
      !map_2d(&L.gg_mn, L.gg_buf, f16, 2 * F, T, 1, kFfnBoxMn) || !map_2d(&L.x_mn, a->x, f16, D, T, 1, kFfnBoxMn) ||
      !map_2d(&L.gy_mn, a->grad_y, f16, D, T, 1, kFfnBoxMn) || !map_2d(&L.a_mn, L.a_buf, f16, F, T, 1, kFfnBoxMn))
    return fail(MHC_ERR_RUNTIME, "encoding a tensor map failed");
  L.ga = shape(T, F, D, cut_alone(T, F, D, true, 1), false, f16, false, true);
  L.gx = shape(T, D, 2 * F, cut_gx(T, D, F), false, f16, false, true);
  L.gwgu = shape(2 * F, D, T, cut_tokens(T), false, f16, true, true);
  L.gwd = shape(D, F, T, cut_tokens(T), false, f16, true, true);
  L.part = L.gx.slices > 1 ? reinterpret_cast<float*>(ws + l.part) : nullptr;
  L.part_gu = L.gwgu.slices > 1 ? reinterpret_cast<float*>(ws + l.part_gu) : nullptr;
  L.part_down = L.gwd.slices > 1 ? reinterpret_cast<float*>(ws + l.part_down) : nullptr;
  const cudaError_t e = launch_ffn_backward(L, f16, s);
  if (e != cudaSuccess) return fail(MHC_ERR_RUNTIME, "feed-forward backward launch failed: %s", cudaGetErrorString(e));
  return MHC_OK;
}

mhc_status_t mhc_ffn_status(const void* workspace, void* stream) {
  clear_error();
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint32_t word = 0;
  cudaError_t e = cudaSuccess;
  if (workspace) e = cudaMemcpyAsync(&word, workspace, sizeof word, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return fail(MHC_ERR_RUNTIME, "CUDA error: %s", cudaGetErrorString(e));
  if (word) return fail(MHC_ERR_RUNTIME, "device error word 0x%x: a wait gave up", word);
  return MHC_OK;
}

}  // extern "C"
