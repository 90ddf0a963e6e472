// mhc_ffn.cuh -- launch plumbing shared by the feed-forward block's files.
#pragma once

#include "mhc_ckpt.cuh"

namespace mhc {

// n / d for 0 <= n < 2^31 by a multiplication: with 2^sh < d <= 2^(sh + 1) and
// mul = ceil(2^(32 + sh) / d), mul d exceeds 2^(32 + sh) by less than d, which
// times n stays below 2^(32 + sh).  (Tiles are found this way by every role: T =
// 3388, D = 504, F = 15800, forward 172.4 -> 168.8 us.)
struct FastDiv {
  uint32_t mul = 0;
  int sh = -1;                 // -1: d = 1
  FastDiv() = default;
  explicit FastDiv(uint32_t d) {
    if (d < 2) return;
    for (sh = 0; (2ull << sh) < d;) ++sh;
    mul = (uint32_t)(((1ull << (32 + sh)) + d - 1) / d);
  }
  __device__ __forceinline__ int operator()(int n) const { return sh < 0 ? n : (int)(__umulhi((uint32_t)n, mul) >> sh); }
};

// One matrix product D[M, N] = A B^T on 16-bit operands: operand row r, depth
// k.  "K-major" operands store k contiguously, "MN-major" ones r.
struct GemmShape {
  int tile_n;                  // width of a tile: 256, 192 or 128
  int tiles_m, tiles_n;
  int slices;                  // parts of the depth that are tiles of their own
  int kiters, kslice;          // chunks of 64 of the whole depth, and of a slice (the last may have fewer)
  int band;                    // tile rows walked together, column by column
  FastDiv by_area, by_band, by_rows, by_last;   // tiles of a slice, of a band; rows of a band, of the last
  uint32_t idesc;
  int a_mn, b_mn;              // operand stored MN-major
};

__host__ __device__ inline int gemm_tiles(const GemmShape& g) { return g.tiles_m * g.tiles_n * g.slices; }

// What the launches of one call share.
struct FfnCall {
  uint32_t* err;               // device error word; the next word counts tiles (ffn_gemm_kernel)
  uint64_t wait_ns;
  int withhold;                // test hook of the call's last launch
  int sms;
};

// Up to this many tokens the few-token kernels run (mhc_ffn_few.cuh).
constexpr int kFewTokens = 128;

// Forward: kept = 0 none, 1 16-bit, 2 8-bit.  For few tokens the maps of x and
// a have boxes of all tokens.
struct FfnFwdLaunch {
  CUtensorMap x, wgu, a, wd;
  GemmShape gu, down;
  FfnCall call;
  int T, D, F, act, kept;
  void *a_buf, *y, *gate_up, *codes, *scales;
  float* part;                     // sums of the slices of down, where it has more than one
};
cudaError_t launch_ffn_forward(const FfnFwdLaunch& L, bool f16, cudaStream_t s);

struct FfnBwdLaunch {
  CUtensorMap gy_k, wd_mn;         // ga = grad_y Wd
  CUtensorMap gg_k, wgu_mn;        // grad_x = [gg, gu] [Wg; Wu]
  CUtensorMap gg_mn, x_mn;         // grad_w_gate_up = [gg, gu]^T x
  CUtensorMap gy_mn, a_mn;         // grad_w_down = grad_y^T a
  // for few tokens gy_k and gg_k have boxes of all tokens
  GemmShape ga, gx, gwgu, gwd;
  FfnCall call;
  int T, D, F, act, kept;
  const void *gate_up, *codes, *scales;
  void *gg_buf, *a_buf, *grad_x, *grad_w_gate_up, *grad_w_down;
  float *part, *part_gu, *part_down;   // of gx, gwgu and gwd, where they have more than one slice
};
cudaError_t launch_ffn_backward(const FfnBwdLaunch& L, bool f16, cudaStream_t s);

constexpr int kFfnTileM = 256, kFfnTileN = 256, kFfnTileK = 64;
constexpr uint32_t kFfnBoxK = 128, kFfnBoxMn = 64;   // tensor-map box rows of a K-major / MN-major operand
                                                       // (half of a tile's width for a K-major B)

}  // namespace mhc
