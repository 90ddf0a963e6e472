// mhc_experts_gemm.cuh -- the grouped products of the routed experts: jobs, epilogues
// and the launch plumbing shared by the forward and the backward.
//
// Products with an expert's weights (gate and up, down, gate gradients, grad_x) take
// the weights as the 256-row operand and the expert's tokens as the other, up to 256
// at a time: an expert's rows are rounded up to 32, not to a tile of 256, and a few
// tokens stream the weights as fast as they come.  Accumulator lanes are then rows of
// the weights and columns are tokens, so epilogues write transposed.  The weight
// gradients are ordinary tiles whose depth is the expert's rows.
#pragma once

#include "mhc_experts.cuh"
#include "mhc_group_gemm.cuh"

namespace mhc {

// How the weights lie: rows along K (down), rows along K with eight gate rows and
// eight up rows in turn (gate and up), or MN-major (gate gradients, grad_x).
enum { kRowsK = 0, kRowsGateUp = 1, kRowsMn = 2 };

template <int kRows, bool F16>
struct ExpertsJob {
  static constexpr bool kAMn = kRows == kRowsMn, kBMn = false, kDraw = true;
  CUtensorMap a, b[4];           // b: boxes of 16, 32, 64 and 128 tokens
  const int* head;
  const int4* table;
  int tiles_m, kiters;
  FastDiv by_m;

  struct Raw {
    int4 lo, hi;
  };
  __device__ __forceinline__ void prefetch() const {
    tma_prefetch_desc(&a);
#pragma unroll
    for (int i = 0; i < 4; ++i) tma_prefetch_desc(&b[i]);
  }
  __device__ __forceinline__ int tiles() const { return head[2] * tiles_m; }
  __device__ __forceinline__ Raw fetch(int t) const {
    const int i = by_m(t);
    return {table[2 * i], table[2 * i + 1]};
  }
  // Tile t: the tiles of a band share a tile of the weights one after the other.
  __device__ __forceinline__ GTile make(int t, const Raw& w) const {
    GTile g;
    const int r = t - w.lo.y * tiles_m, j = r % w.lo.z, off = j * w.hi.y + 32 * min(j, w.hi.z);
    g.e = w.lo.x;
    g.tm = r / w.lo.z;
    g.tn = 0;
    g.row0 = w.lo.w + off;
    g.rows = min(w.hi.y + (j < w.hi.z ? 32 : 0), w.hi.x - off);
    g.width = (g.rows + 31) & ~31;
    g.kiters = kiters;
    g.kind = 0;
    return g;
  }
  static __device__ __forceinline__ int box(const GTile& g) {
    const int half = g.width >> 1;
    return half <= 16 ? 0 : half <= 32 ? 1 : half <= 64 ? 2 : 3;
  }
  __device__ __forceinline__ int bytes(const GTile& g) const { return kGemmOpBytes + (16 << box(g)) * kFfnTileK * 2; }
  __device__ __forceinline__ int steps(const GTile&, int) const { return kFfnTileK / 16; }
  __device__ __forceinline__ uint32_t idesc(const GTile& g) const { return grp_idesc(F16, kAMn, false, g.width); }
  __device__ __forceinline__ void load(const GTile& g, int k, uint32_t sa, uint32_t sb, uint32_t bar, int rank) const {
    const int k0 = k * kFfnTileK;
    if constexpr (kRows == kRowsGateUp) {
      tma_load_5d_pair(sa, &a, bar, k0, 0, 0, g.tm * 16 + rank * 8, g.e);
    } else if constexpr (kRows == kRowsK) {
      tma_load_3d_pair(sa, &a, bar, k0, g.tm * kFfnTileM + rank * kGemmHalf, g.e);
    } else {
      const int m0 = g.tm * kFfnTileM + rank * kGemmHalf;
      tma_load_3d_pair(sa, &a, bar, m0, k0, g.e);
      tma_load_3d_pair(sa + 8192, &a, bar, m0 + 64, k0, g.e);
    }
    tma_load_2d_pair(sb, &b[box(g)], bar, k0, g.row0 + rank * (g.width >> 1));
  }
};

// grad_w_gate_up = [gg, gu]^T x (kind 0) and grad_w_down = grad_y^T (w a) (kind 1), the
// sums over an expert's rows.  These lie between rows of zeros at multiples of 16, so
// the last step of a depth takes nothing of the next expert's.
template <bool F16>
struct WeightGradJob {
  static constexpr bool kAMn = true, kBMn = true, kDraw = true;
  CUtensorMap a[2], b[2];
  const int *counts, *starts;
  int E, tiles_n[2], area[2], width[2];
  FastDiv by_expert, by_n[2];

  struct Raw {
    int count, start;
  };
  __device__ __forceinline__ void prefetch() const {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      tma_prefetch_desc(&a[i]);
      tma_prefetch_desc(&b[i]);
    }
  }
  __device__ __forceinline__ int tiles() const { return E * (area[0] + area[1]); }
  __device__ __forceinline__ Raw fetch(int t) const {
    const int e = by_expert(t);
    return {counts[e], starts[e]};
  }
  __device__ __forceinline__ GTile make(int t, const Raw& w) const {
    GTile g;
    g.e = by_expert(t);
    int r = t - g.e * (area[0] + area[1]);
    g.kind = r >= area[0] ? 1 : 0;
    r -= g.kind ? area[0] : 0;
    g.tm = g.kind ? by_n[1](r) : by_n[0](r);
    g.tn = r - g.tm * tiles_n[g.kind];
    g.row0 = w.start;
    g.rows = w.count;
    g.width = width[g.kind];
    g.kiters = (w.count + kFfnTileK - 1) / kFfnTileK;
    return g;
  }
  __device__ __forceinline__ int bytes(const GTile& g) const { return kGemmOpBytes + (g.width > 128 ? 16384 : 8192); }
  __device__ __forceinline__ int steps(const GTile& g, int k) const {
    return min(kFfnTileK / 16, (g.rows - k * kFfnTileK + kPlanPad - 1) / kPlanPad);
  }
  __device__ __forceinline__ uint32_t idesc(const GTile& g) const { return grp_idesc(F16, true, true, g.width); }
  __device__ __forceinline__ void load(const GTile& g, int k, uint32_t sa, uint32_t sb, uint32_t bar, int rank) const {
    const int k0 = g.row0 + k * kFfnTileK, m0 = g.tm * kFfnTileM + rank * kGemmHalf, n0 = g.tn * g.width + rank * (g.width >> 1);
    const CUtensorMap *ta = g.kind ? &a[1] : &a[0], *tb = g.kind ? &b[1] : &b[0];
    tma_load_2d_pair(sa, ta, bar, m0, k0);
    tma_load_2d_pair(sa + 8192, ta, bar, m0 + 64, k0);
    tma_load_2d_pair(sb, tb, bar, n0, k0);
    if (g.width > 128) tma_load_2d_pair(sb + 8192, tb, bar, n0 + 64, k0);
  }
};

// ------------------------------------------------------------- epilogues

// The accumulator's column `row` and lane m as 24 bits at [row, m] of two planes.
struct EpiRows {
  using Pre = NoPre;
  uint16_t* hi;
  uint8_t* lo;
  int M;
  __device__ __forceinline__ void pre(const GTile&, Pre&, int, int, int, int) const {}
  __device__ __forceinline__ void tile(const GTile& g, Pre&, int, int, uint32_t taddr, int rank, int q, int grp, uint8_t* buf,
                                       int lane, int) const {
    const int m0 = g.tm * kFfnTileM + rank * kGemmHalf + q * 32;
    if (m0 >= M) return;
#pragma unroll 1
    for (int c = grp * 32; c < g.rows; c += 64) {
      float v[32];
      acc_ld32(taddr + c, v);
      const size_t at = (size_t)(g.row0 + c) * M + m0;
      store_transposed24(v, buf, reinterpret_cast<uint8_t*>(hi + at), lo + at, (size_t)M, g.rows - c, M - m0, lane);
    }
  }
};

// Lanes of a warp: eight gate rows, the same eight up rows, and once more.  Lanes
// eight apart exchange half their columns, so that each has gate and up of sixteen.
template <bool F16, bool kKept>
struct EpiExpertGateUp {
  using Pre = NoPre;
  uint16_t *a, *gate_up;
  int F, act;
  __device__ __forceinline__ void pre(const GTile&, Pre&, int, int, int, int) const {}
  __device__ __forceinline__ void tile(const GTile& g, Pre&, int, int, uint32_t taddr, int rank, int q, int grp, uint8_t* buf,
                                       int lane, int) const {
    const int f0 = g.tm * 128 + rank * 64 + q * 16;
    if (f0 >= F) return;
    const bool up = (lane & 8) != 0;
    const int fi = ((lane >> 4) << 3) + (lane & 7);
    uint16_t* st = reinterpret_cast<uint16_t*>(buf);
#pragma unroll 1
    for (int c = grp * 32; c < g.rows; c += 64) {
      const int rows = g.rows - c;
      const size_t row0 = (size_t)(g.row0 + c);
      float v[32];
      acc_ld32(taddr + c, v);
      if constexpr (kKept) {                     // rows of 64 bytes: 16 gate sums, 16 up sums
#pragma unroll
        for (int j = 0; j < 32; j += 2) {
          const uint32_t w = pack2<F16>(v[j], v[j + 1]);
          st[j * 32 + (up ? 16 : 0) + fi] = (uint16_t)w;
          st[(j + 1) * 32 + (up ? 16 : 0) + fi] = (uint16_t)(w >> 16);
        }
        __syncwarp();
        const int piece = lane & 3, p = piece >> 1, h = (piece & 1) * 8;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = i * 8 + (lane >> 2);
          const uint4 w = *reinterpret_cast<const uint4*>(buf + r * 64 + piece * 16);
          if (r < rows && f0 + h < F) *reinterpret_cast<uint4*>(gate_up + ((row0 + r) * 2 + p) * F + f0 + h) = w;
        }
        __syncwarp();
      }
      float o[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const float got = __shfl_xor_sync(0xFFFFFFFFu, up ? v[j] : v[16 + j], 8);
        const float z = up ? got : v[j], u = up ? v[16 + j] : got;
        o[j] = z * sigmoid_fast(act_arg(z, act)) * u;
      }
      // rows of 32 bytes; the second sixteen 32 bytes further, so that the two
      // halves' writes fall into different banks
#pragma unroll
      for (int j = 0; j < 16; j += 2) {
        const uint32_t w = pack2<F16>(o[j], o[j + 1]);
        st[(j + (up ? 17 : 0)) * 16 + fi] = (uint16_t)w;
        st[(j + 1 + (up ? 17 : 0)) * 16 + fi] = (uint16_t)(w >> 16);
      }
      __syncwarp();
      const int h = (lane & 1) * 8;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = i * 16 + (lane >> 1);
        const uint4 w = *reinterpret_cast<const uint4*>(buf + (r + i) * 32 + h * 2);
        if (r < rows && f0 + h < F) *reinterpret_cast<uint4*>(a + (row0 + r) * F + f0 + h) = w;
      }
      __syncwarp();
    }
  }
};

// acc = ga before the weight: gg, gu, w a, and this warp's 32 terms of a row's
// sum_f a ga.  Sixteen tokens at a time, whose kept sums and weights are loaded one step
// ahead (the first before the tile's sums are there).
template <bool F16>
struct EpiExpertDgate {
  struct Pre {
    uint4 k[4];                  // piece i * 32 + lane: token / 8, gate or up / 4, eight columns
    float w;
  };
  const uint16_t* gate_up;
  const float* w_row;            // weight of each row
  uint16_t *gg, *wa;
  float* part;                   // [ceil(F / 32)][cap_rows]
  int F, act;
  long long cap_rows;
  __device__ __forceinline__ void load(Pre& p, const GTile& g, int f0, int c, int lane) const {
    const int rows = g.rows - c, h = (lane & 3) * 8, plane = (lane >> 2) & 1;
    const size_t row0 = (size_t)(g.row0 + c);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = i * 4 + (lane >> 3);
      p.k[i] = make_uint4(0, 0, 0, 0);
      if (r < rows && f0 + h < F) p.k[i] = *reinterpret_cast<const uint4*>(gate_up + ((row0 + r) * 2 + plane) * F + f0 + h);
    }
    p.w = lane < rows && lane < 16 ? w_row[row0 + lane] : 0.0f;
  }
  __device__ __forceinline__ void pre(const GTile& g, Pre& p, int rank, int q, int grp, int lane) const {
    load(p, g, g.tm * kFfnTileM + rank * kGemmHalf + q * 32, grp * 16, lane);
  }
  __device__ __forceinline__ void tile(const GTile& g, Pre& p, int, int, uint32_t taddr, int rank, int q, int grp, uint8_t* buf,
                                       int lane, int) const {
    const int f0 = g.tm * kFfnTileM + rank * kGemmHalf + q * 32;
    if (f0 >= F) return;
    const bool in = f0 + lane < F;
    uint16_t* st = reinterpret_cast<uint16_t*>(buf);
#pragma unroll 1
    for (int c = grp * 16; c < g.rows; c += 32) {
      const int rows = g.rows - c;
      const size_t row0 = (size_t)(g.row0 + c);
#pragma unroll
      for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4*>(buf + (i * 32 + lane) * 16) = p.k[i];
      const float wl = p.w;
      if (c + 32 < g.rows) load(p, g, f0, c + 32, lane);
      __syncwarp();
      uint16_t kz[16], ku[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        kz[j] = st[j * 64 + lane];
        ku[j] = st[j * 64 + 32 + lane];
      }
      __syncwarp();
      float ga[16];
      tmem_ld16(taddr + c, ga);
      float dot[16];
#pragma unroll
      for (int j = 0; j < 16; j += 2) {
        float og[2], ou[2], oa[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float w = __shfl_sync(0xFFFFFFFFu, wl, j + i);
          const float z = unpack2<F16>(kz[j + i]).x, u = unpack2<F16>(ku[j + i]).x;
          float a;
          gate_grads(z, u, ga[j + i] * w, act, og[i], ou[i], a);
          dot[j + i] = in ? a * ga[j + i] : 0.0f;
          oa[i] = a * w;
        }
        const uint32_t pg = pack2<F16>(og[0], og[1]), pu = pack2<F16>(ou[0], ou[1]), pa = pack2<F16>(oa[0], oa[1]);
        st[j * 32 + lane] = (uint16_t)pg;
        st[(j + 1) * 32 + lane] = (uint16_t)(pg >> 16);
        st[512 + j * 32 + lane] = (uint16_t)pu;
        st[512 + (j + 1) * 32 + lane] = (uint16_t)(pu >> 16);
        st[1024 + j * 32 + lane] = (uint16_t)pa;
        st[1024 + (j + 1) * 32 + lane] = (uint16_t)(pa >> 16);
      }
      __syncwarp();
      const int h = (lane & 3) * 8;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = i * 8 + (lane >> 2);
        const uint4 vg = *reinterpret_cast<const uint4*>(buf + r * 64 + h * 2);
        const uint4 vu = *reinterpret_cast<const uint4*>(buf + 1024 + r * 64 + h * 2);
        const uint4 va = *reinterpret_cast<const uint4*>(buf + 2048 + r * 64 + h * 2);
        if (r < rows && f0 + h < F) {
          *reinterpret_cast<uint4*>(gg + (row0 + r) * 2 * F + f0 + h) = vg;
          *reinterpret_cast<uint4*>(gg + ((row0 + r) * 2 + 1) * F + f0 + h) = vu;
          *reinterpret_cast<uint4*>(wa + (row0 + r) * F + f0 + h) = va;
        }
      }
      // sums over the lanes: lanes halve the columns they carry, column j ends in
      // lanes 2 j and 2 j + 1
#pragma unroll
      for (int n = 8; n > 0; n >>= 1) {
        const bool hi = (lane & (2 * n)) != 0;
#pragma unroll
        for (int j = 0; j < n; ++j) {
          const float send = hi ? dot[j] : dot[n + j], keep = hi ? dot[n + j] : dot[j];
          dot[j] = keep + __shfl_xor_sync(0xFFFFFFFFu, send, 2 * n);
        }
      }
      dot[0] += __shfl_xor_sync(0xFFFFFFFFu, dot[0], 1);
      if (!(lane & 1) && (lane >> 1) < rows) part[(long long)(f0 >> 5) * cap_rows + row0 + (lane >> 1)] = dot[0];
      __syncwarp();
    }
  }
};

// out[e][m, n] of either weight gradient; an expert without rows gets zeros.  A sum
// in several parts is joined in fp32 in a room of the warp's own.
template <bool F16>
struct EpiWeightGrad {
  using Pre = NoPre;
  uint16_t* out[2];
  int M[2], N[2];
  float* room;                   // [CTA][warp][128 columns][32 lanes], where a sum may have parts
  __device__ __forceinline__ void pre(const GTile&, Pre&, int, int, int, int) const {}
  __device__ __forceinline__ void tile(const GTile& g, Pre&, int p, int parts, uint32_t taddr, int rank, int q, int grp,
                                       uint8_t* buf, int lane, int pair) const {
    const int Mk = g.kind ? M[1] : M[0], Nk = g.kind ? N[1] : N[0];
    const int m0 = g.tm * kFfnTileM + rank * kGemmHalf + q * 32, n0 = g.tn * g.width, half = g.width >> 1;
    uint16_t* o = (g.kind ? out[1] : out[0]) + (size_t)g.e * Mk * Nk;
    if (m0 >= Mk) return;
    float* mine = room + ((size_t)(pair * 2 + rank) * 8 + grp * 4 + q) * 128 * 32 + lane;
    const int beg = grp * half, end = beg + half;
#pragma unroll 1
    for (int c = beg; c < end && n0 + c < Nk; c += 64) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (h && c + 32 >= end) break;
        float v[32];
        if (parts == 0) {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = 0.0f;
        } else {
          acc_ld32(taddr + c + 32 * h, v);
        }
        if (parts > 1) {
          float* at = mine + (size_t)(c - beg + 32 * h) * 32;
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            if (p > 0) v[i] += at[i * 32];
            if (p + 1 < parts) at[i * 32] = v[i];
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4*>(buf + sw128(lane, h * 4 + i)) = pack8v<F16>(v + 8 * i);
      }
      if (parts <= 1 || p + 1 == parts)
        stage_flush(buf, reinterpret_cast<uint8_t*>(o + (size_t)m0 * Nk + n0 + c), (size_t)Nk * 2, Mk - m0,
                    min(min(64, end - c), Nk - n0 - c) * 2, lane);
      else
        __syncwarp();
    }
  }
};

// --------------------------------------------------------------- launches

struct ExpertsCall {
  uint32_t* header;              // error word, then a counter of drawn tiles for each launch
  uint64_t wait_ns;
  int withhold, sms;
};

struct ExpertsFwdLaunch {
  CUtensorMap wgu, wd, x[4], a[4];
  ExpertsCall call;
  PlanView plan;
  PlanLayout lay;
  long long T;
  int E, k, D, F, act;
  const void* x_in;
  const float* weights;
  void *xs, *a_buf, *y, *gate_up;              // xs: rows of x, then the outputs' upper planes
  uint8_t* lo;                                 // their lower planes
};
cudaError_t launch_experts_forward(const ExpertsFwdLaunch& L, bool f16, cudaStream_t s);

struct ExpertsBwdLaunch {
  CUtensorMap wd_mn, wgu_mn, gy[4], gg[4], gg_mn, xs_mn, gy_mn, wa_mn;
  ExpertsCall call;
  PlanView plan;
  PlanLayout lay;
  long long T;
  int E, k, D, F, act;
  const void *grad_y, *x_in, *gate_up;
  const float* weights;
  void *xs, *gys, *gg_buf, *wa_buf, *grad_x, *grad_w_gate_up, *grad_w_down;   // xs, gys: then grad_x's rows
  float *w_row, *part, *grad_weights, *room;
};
cudaError_t launch_experts_backward(const ExpertsBwdLaunch& L, bool f16, cudaStream_t s);

inline GrpCall grp_call(const ExpertsCall& c, int counter, bool last, int b_rows) {
  GrpCall g;
  g.err = c.header;
  g.counter = c.header + counter;
  g.wait_ns = c.wait_ns;
  g.withhold = last ? c.withhold : 0;
  grp_ring(&g, b_rows);
  return g;
}
// Rows of the token boxes of the plan's widest tile, per CTA.
inline int token_rows(int width) { return width <= 32 ? 16 : width <= 64 ? 32 : width <= 128 ? 64 : 128; }

template <int kRows, bool F16>
ExpertsJob<kRows, F16> experts_job(const CUtensorMap& a, const CUtensorMap (&b)[4], const PlanView& p, int m, int per_tile, int depth) {
  ExpertsJob<kRows, F16> j;
  j.a = a;
  for (int i = 0; i < 4; ++i) j.b[i] = b[i];
  j.head = p.head;
  j.table = p.table;
  j.tiles_m = (m + per_tile - 1) / per_tile;
  j.kiters = (depth + kFfnTileK - 1) / kFfnTileK;
  j.by_m = FastDiv((uint32_t)j.tiles_m);
  return j;
}

// Launches of the row kernels.
template <class K, class... A>
cudaError_t launch_rows(K* k, long long warps, int sms, bool dependent, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  const long long blocks = (warps + 7) / 8, most = 8ll * sms;
  cfg.gridDim = dim3((unsigned)(blocks < 1 ? 1 : blocks < most ? blocks : most));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = dependent ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, k, args...);
}

// out[t] = sum_j w_tj rows[place_tj] of 24-bit rows, in the order of j; w = 1 without
// weights.  A warp takes 256 columns of a token, eight a lane, eight experts in flight.
template <bool F16>
__device__ __forceinline__ void combine_item(long long item, int segs, int k, int D, const int* places, const float* weights,
                                             const uint16_t* hi, const uint8_t* lo, uint16_t* out, int lane) {
  const long long t = item / segs;
  const int c0 = (int)(item - t * segs) * 256 + lane * 8;
  float s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) s[i] = 0.0f;
  const int at = lane < k ? places[t * k + lane] : -1;
  const float wt = lane < k && weights ? weights[t * k + lane] : 1.0f;
#pragma unroll 1
  for (int j0 = 0; j0 < k; j0 += 8) {
    uint4 v[8];
    uint2 l[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int p = __shfl_sync(0xFFFFFFFFu, at, (j0 + j) & 31);
      v[j] = make_uint4(0, 0, 0, 0);
      l[j] = make_uint2(0, 0);
      if (j0 + j < k && p >= 0 && c0 < D) {
        v[j] = __ldcs(reinterpret_cast<const uint4*>(hi + (size_t)p * D + c0));
        l[j] = __ldcs(reinterpret_cast<const uint2*>(lo + (size_t)p * D + c0));
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int p = __shfl_sync(0xFFFFFFFFu, at, (j0 + j) & 31);
      float w = __shfl_sync(0xFFFFFFFFu, wt, (j0 + j) & 31);
      if (j0 + j >= k || p < 0) w = 0.0f;
      const uint32_t u[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t b = i < 2 ? l[j].x >> (16 * (i & 1)) : l[j].y >> (16 * (i & 1));   // two low bytes
        s[2 * i] = fmaf(w, __uint_as_float((u[i] << 16) | ((b & 0xFFu) << 8)), s[2 * i]);
        s[2 * i + 1] = fmaf(w, __uint_as_float((u[i] & 0xFFFF0000u) | (b & 0xFF00u)), s[2 * i + 1]);
      }
    }
  }
  if (c0 < D) *reinterpret_cast<uint4*>(out + (size_t)t * D + c0) = pack8v<F16>(s);
}

// Row r of the plan's order from row slot / k of a tensor, zeros where it is padding: a
// warp takes 1024 columns, four pieces a lane.
__device__ __forceinline__ void gather_item(int slot, int k, int r, int seg, int D, const uint16_t* from, uint16_t* to, int lane) {
  const int c0 = seg * 1024 + lane * 8;
  uint4 v[4];
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    v[h] = make_uint4(0, 0, 0, 0);
    if (slot >= 0 && c0 + 256 * h < D) v[h] = *reinterpret_cast<const uint4*>(from + (size_t)(slot / k) * D + c0 + 256 * h);
  }
#pragma unroll
  for (int h = 0; h < 4; ++h)
    if (c0 + 256 * h < D) *reinterpret_cast<uint4*>(to + (size_t)r * D + c0 + 256 * h) = v[h];
}

}  // namespace mhc
