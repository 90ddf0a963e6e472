// mhc_experts_gemm.cuh -- the grouped products of the routed experts: jobs, epilogues
// and the launch plumbing shared by the forward and the backward.
//
// Products with an expert's weights (gate and up, down, gate gradients, grad_x) take
// the weights as the 256-row operand and the expert's tokens as the other, up to 256
// at a time: an expert's rows are rounded up to 32, not to a tile of 256, and a few
// tokens stream the weights as fast as they come.  Accumulator lanes are then rows of
// the weights and columns are tokens, so epilogues write transposed.  The weight
// gradients are ordinary tiles whose depth is the expert's rows.
//
// Bound by: the weights' stream for few tokens (one token, 8 experts of 4096 x 2048: 6.2 and
// 5.7 TB/s); the tensor cores and their power for many (pipe active at 4096 tokens, 4 of 16
// experts: 86% in gate and up and in grad_x, 80% in down, 83% in the weight gradients, 70% in
// the gate gradients, whose epilogue moves five 16-bit values for each of its sums).
#pragma once

#include "mhc_experts.cuh"
#include "mhc_group_gemm.cuh"

namespace mhc {

// How the weights lie: rows along K (down), rows along K with eight gate rows and
// eight up rows in turn (gate and up), or MN-major (gate gradients, grad_x).
enum { kRowsK = 0, kRowsGateUp = 1, kRowsMn = 2 };

template <int kRows, bool F16>
struct ExpertsJob {
  // A call's first launch is ordered behind the plan, so the launches behind it may read
  // that before they wait.
  static constexpr bool kAMn = kRows == kRowsMn, kBMn = false, kDraw = true, kEarly = true;
  CUtensorMap a, b[4];           // b: boxes of 16, 32, 64 and 128 tokens
  const int* head;
  const int4* table;
  int E, width, cap_rows, cap_tiles;
  int tiles_m, kiters;
  int blocks;                    // kRowsMn: a has blocks of 64 columns as a dimension of its own (columns a multiple of 64)
  FastDiv by_m;

  struct Raw {
    int4 lo, hi;
  };
  __device__ __forceinline__ void prefetch() const {
    tma_prefetch_desc(&a);
#pragma unroll
    for (int i = 0; i < 4; ++i) tma_prefetch_desc(&b[i]);
  }
  __device__ __forceinline__ int tiles() const { return min(max(head[2], 0), cap_tiles) * tiles_m; }
  __device__ __forceinline__ Raw fetch(int t) const {
    const int i = by_m(t);
    return {table[2 * i], table[2 * i + 1]};
  }
  // Tile t: the tiles of a band share a tile of the weights one after the other.
  __device__ __forceinline__ GTile make(int t, const Raw& w) const {
    GTile g;
    const int r = t - w.lo.y * tiles_m, n = max(w.lo.z, 1), j = r % n, off = j * w.hi.y + 32 * min(j, w.hi.z);
    g.e = min(max(w.lo.x, 0), E - 1);
    g.tm = min(max(r / n, 0), tiles_m - 1);
    g.tn = 0;
    g.row0 = min(max(w.lo.w + off, 0), cap_rows);
    g.rows = min(min(w.hi.y + (j < w.hi.z ? 32 : 0), w.hi.x - off), min(width, cap_rows - g.row0));
    g.rows = max(g.rows, 0);
    g.width = (g.rows + 31) & ~31;
    g.kiters = g.rows ? kiters : 0;
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
  __device__ __forceinline__ void load_a(const GTile& g, int k, uint32_t sa, uint32_t bar, int rank) const {
    const int k0 = k * kFfnTileK;
    if constexpr (kRows == kRowsGateUp) {
      tma_load_5d_pair(sa, &a, bar, k0, 0, 0, g.tm * 16 + rank * 8, g.e);
    } else if constexpr (kRows == kRowsK) {
      tma_load_3d_pair(sa, &a, bar, k0, g.tm * kFfnTileM + rank * kGemmHalf, g.e);
    } else {
      const int m0 = g.tm * kFfnTileM + rank * kGemmHalf;
      if (blocks) {
        tma_load_4d_pair(sa, &a, bar, 0, k0, m0 >> 6, g.e);
      } else {
        tma_load_3d_pair(sa, &a, bar, m0, k0, g.e);
        tma_load_3d_pair(sa + 8192, &a, bar, m0 + 64, k0, g.e);
      }
    }
  }
  __device__ __forceinline__ void load_b(const GTile& g, int k, uint32_t sb, uint32_t bar, int rank) const {
    tma_load_2d_pair(sb, &b[box(g)], bar, k * kFfnTileK, g.row0 + rank * (g.width >> 1));
  }
};

// grad_w_gate_up = [gg, gu]^T x (kind 0) and grad_w_down = grad_y^T (w a) (kind 1), the
// sums over an expert's rows.  These lie between rows of zeros at multiples of 16, so
// the last step of a depth takes nothing of the next expert's.
template <bool F16>
struct WeightGradJob {
  static constexpr bool kAMn = true, kBMn = true, kDraw = true, kEarly = false;
  // a, b: blocks of 64 columns are a dimension of their own, so that one copy brings two
  // (four copies a stage by one thread took twice as long as the products); narrow: b's for
  // tiles of at most 128 columns
  CUtensorMap a[2], b[2], narrow[2];
  const int *counts, *starts;
  int E, cap_rows, tiles_n[2], area[2], width[2];
  FastDiv by_expert, by_n[2];

  struct Raw {
    int count, start;
  };
  __device__ __forceinline__ void prefetch() const {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      tma_prefetch_desc(&a[i]);
      tma_prefetch_desc(width[i] > 128 ? &b[i] : &narrow[i]);
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
    g.row0 = min(max(w.start, 0), cap_rows);
    g.rows = min(max(w.count, 0), cap_rows - g.row0);
    g.width = width[g.kind];
    g.kiters = (g.rows + kFfnTileK - 1) / kFfnTileK;
    return g;
  }
  __device__ __forceinline__ int bytes(const GTile& g) const { return kGemmOpBytes + (g.width > 128 ? 16384 : 8192); }
  __device__ __forceinline__ int steps(const GTile& g, int k) const {
    return min(kFfnTileK / 16, (g.rows - k * kFfnTileK + kPlanPad - 1) / kPlanPad);
  }
  __device__ __forceinline__ uint32_t idesc(const GTile& g) const { return grp_idesc(F16, true, true, g.width); }
  __device__ __forceinline__ void load_a(const GTile& g, int k, uint32_t sa, uint32_t bar, int rank) const {
    const int k0 = g.row0 + k * kFfnTileK, m0 = g.tm * kFfnTileM + rank * kGemmHalf;
    tma_load_3d_pair(sa, g.kind ? &a[1] : &a[0], bar, 0, k0, m0 >> 6);
  }
  __device__ __forceinline__ void load_b(const GTile& g, int k, uint32_t sb, uint32_t bar, int rank) const {
    const int k0 = g.row0 + k * kFfnTileK, n0 = g.tn * g.width + rank * (g.width >> 1);
    if (g.width > 128) tma_load_3d_pair(sb, g.kind ? &b[1] : &b[0], bar, 0, k0, n0 >> 6);
    else tma_load_2d_pair(sb, g.kind ? &narrow[1] : &narrow[0], bar, n0, k0);
  }
};

// ------------------------------------------------------------- epilogues

// An fp32 sum with half a step of its upper 24 bits added, which then are the nearest (16
// significant bits, 2^-16 of the sum off at most).  Not to infinities and NaN, nor to what
// would become infinite.
__device__ __forceinline__ uint32_t upper24(float v) {
  return __float_as_uint(v) + (fabsf(v) < 0x1.ffffp127f ? 0x80u : 0u);
}

// The accumulator's column `row` and lane m as the upper 24 bits of the sum at [row, m] of
// two planes: 16 bits, and 8 whose order inside sixteen columns is 0 8 1 9 .. 7 15.  What a
// token's sum is off by is then 2^-16 of a term at most, with either sign; rows rounded to 16
// bits were half of y's error (1.7 times what its own rounding leaves, so 1.4), in fp32 they
// cost a third more traffic.
struct EpiRows {
  using Pre = NoPre;
  uint16_t* hi;
  uint8_t* lo;
  int M, lo_pitch;
  __device__ __forceinline__ void pre(const GTile&, Pre&, int, int, int, int) const {}
  __device__ __forceinline__ void tile(const GTile& g, Pre&, int, int, uint32_t taddr, int rank, int q, int grp, uint8_t* buf,
                                       int lane, int) const {
    const int m0 = g.tm * kFfnTileM + rank * kGemmHalf + q * 32;
    if (m0 >= M) return;
    const uint32_t sh = smem_u32(buf) + (lane & 7) * kPitch64 + (lane >> 3) * 16;
    const uint32_t sl = smem_u32(buf) + 32 * kPitch64 + (((lane >> 4) << 3) + (lane & 7)) * kPitch32 + ((lane >> 3) & 1) * 16;
#pragma unroll 1
    for (int c = grp * 32; c < g.rows; c += 64) {
      float v[4][4][2];
      frag_ld<4>(taddr + c, v);
      uint32_t low[4][2];
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        uint32_t u[4][2], w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          u[i][0] = upper24(v[i][b][0]);
          u[i][1] = upper24(v[i][b][1]);
          w[i] = __byte_perm(u[i][0], u[i][1], 0x7632);
        }
        frag_st_t(sh + b * 8 * kPitch64, w[0], w[1], w[2], w[3]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t x = __byte_perm(u[2 * i][0], u[2 * i + 1][0], 0x0051);
          const uint32_t y = __byte_perm(u[2 * i][1], u[2 * i + 1][1], 0x0051);
          low[b][i] = __byte_perm(x, y, 0x5410);
        }
      }
      frag_st_t(sl, low[0][0], low[0][1], low[1][0], low[1][1]);
      frag_st_t(sl + 16 * kPitch32, low[2][0], low[2][1], low[3][0], low[3][1]);
      __syncwarp();
      const size_t row0 = (size_t)(g.row0 + c);
      flush64<32>(buf, reinterpret_cast<uint8_t*>(hi + row0 * M + m0), (size_t)M * 2, g.rows - c, (M - m0 + 7) >> 3, lane);
      flush32(buf + 32 * kPitch64, lo + row0 * lo_pitch + m0, lo_pitch, g.rows - c, (M - m0 + 15) >> 4, lane);
      __syncwarp();
    }
  }
};

// Rows of a warp: eight of the gate, the same eight of up, and once more, so that a lane
// has both sums of its elements.
template <bool F16, bool kKept, int kAct>
struct EpiExpertGateUp {
  using Pre = NoPre;
  uint16_t *a, *gate_up;
  int F;
  __device__ __forceinline__ void pre(const GTile&, Pre&, int, int, int, int) const {}
  __device__ __forceinline__ void tile(const GTile& g, Pre&, int, int, uint32_t taddr, int rank, int q, int grp, uint8_t* buf,
                                       int lane, int) const {
    const int f0 = g.tm * 128 + rank * 64 + q * 16;
    if (f0 >= F) return;
    const int pieces = (F - f0) >> 3;
    // kept: rows of 16 gate and 16 up sums; a: rows of 16
    const uint32_t sk = smem_u32(buf) + (lane & 7) * kPitch64 + (lane >> 3) * 16;
    const uint32_t sa = smem_u32(buf) + 32 * kPitch64 + (((lane >> 4) << 3) + (lane & 7)) * kPitch32 + ((lane >> 3) & 1) * 16;
#pragma unroll 1
    for (int c = grp * 32; c < g.rows; c += 64) {
      const int rows = g.rows - c;
      const size_t row0 = (size_t)(g.row0 + c);
      float v[4][4][2];
      frag_ld<4>(taddr + c, v);
      if constexpr (kKept) {
#pragma unroll
        for (int b = 0; b < 4; ++b)
          frag_st_t(sk + b * 8 * kPitch64, pack2<F16>(v[0][b][0], v[0][b][1]), pack2<F16>(v[2][b][0], v[2][b][1]),
                    pack2<F16>(v[1][b][0], v[1][b][1]), pack2<F16>(v[3][b][0], v[3][b][1]));
      }
      uint32_t o[4][2];
#pragma unroll
      for (int b = 0; b < 4; ++b)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float x[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float z = v[2 * h][b][e];
            x[e] = z * sigmoid_fast(act_arg(z, kAct)) * v[2 * h + 1][b][e];
          }
          o[b][h] = pack2<F16>(x[0], x[1]);
        }
      frag_st_t(sa, o[0][0], o[0][1], o[1][0], o[1][1]);
      frag_st_t(sa + 16 * kPitch32, o[2][0], o[2][1], o[3][0], o[3][1]);
      __syncwarp();
      if constexpr (kKept) {                     // pieces 0 and 1 gate, 2 and 3 up
        const int p = (lane >> 1) & 1, h = lane & 1;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = i * 8 + (lane >> 2);
          const uint4 w = *reinterpret_cast<const uint4*>(buf + r * kPitch64 + (lane & 3) * 16);
          if (r < rows && h < pieces) *reinterpret_cast<uint4*>(gate_up + ((row0 + r) * 2 + p) * F + f0 + 8 * h) = w;
        }
      }
      flush32(buf + 32 * kPitch64, reinterpret_cast<uint8_t*>(a + row0 * F + f0), (size_t)F * 2, rows, pieces, lane);
      __syncwarp();
    }
  }
};

// acc = ga before the weight: gg, gu, w a, and this warp's 32 terms of a row's
// sum_f a ga.  Sixteen tokens at a time, whose kept sums and weights are loaded one step
// ahead (the first before the tile's sums are there).
template <bool F16, int kAct>
struct EpiExpertDgate {
  struct Pre {
    uint4 k[4];                  // piece i * 32 + lane: token / 8, gate or up / 4, eight columns
    float2 w[2];                 // of the lane's tokens 8 b + 2 (lane % 4)
  };
  const uint16_t* gate_up;
  const float* w_row;            // weight of each row
  uint16_t *gg, *wa;
  float* part;                   // [ceil(F / 32)][cap_rows]
  int F;
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
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int r = 8 * b + 2 * (lane & 3);
      p.w[b].x = r < rows ? w_row[row0 + r] : 0.0f;
      p.w[b].y = r + 1 < rows ? w_row[row0 + r + 1] : 0.0f;
    }
  }
  __device__ __forceinline__ void pre(const GTile& g, Pre& p, int rank, int q, int grp, int lane) const {
    load(p, g, g.tm * kFfnTileM + rank * kGemmHalf + q * 32, grp * 16, lane);
  }
  __device__ __forceinline__ void tile(const GTile& g, Pre& p, int, int, uint32_t taddr, int rank, int q, int grp, uint8_t* buf,
                                       int lane, int) const {
    const int f0 = g.tm * kFfnTileM + rank * kGemmHalf + q * 32;
    if (f0 >= F) return;
    const uint32_t s0 = smem_u32(buf), frag = (lane & 7) * kPitch64 + (lane >> 3) * 16;
    const uint32_t sk = s0 + (lane & 7) * kPitch128 + (lane >> 3) * 16;
    const int pieces = (F - f0) >> 3;
#pragma unroll 1
    for (int c = grp * 16; c < g.rows; c += 32) {
      const int rows = g.rows - c;
      const size_t row0 = (size_t)(g.row0 + c);
      // rows of a token's gate and up sums
#pragma unroll
      for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4*>(buf + (i * 4 + (lane >> 3)) * kPitch128 + (lane & 7) * 16) = p.k[i];
      const float2 wt[2] = {p.w[0], p.w[1]};
      if (c + 32 < g.rows) load(p, g, f0, c + 32, lane);
      __syncwarp();
      uint32_t kz[2][4], ku[2][4];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        frag_lds_t(sk + b * 8 * kPitch128, kz[b]);
        frag_lds_t(sk + b * 8 * kPitch128 + 64, ku[b]);
      }
      float ga[4][2][2];
      frag_ld<2>(taddr + c, ga);
      __syncwarp();
      float dot[2][2] = {{0.0f, 0.0f}, {0.0f, 0.0f}};
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        uint32_t og[4], ou[4], oa[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 z = unpack2<F16>(kz[b][i]), u = unpack2<F16>(ku[b][i]);
          float g0, u0, a0, g1, u1, a1;
          gate_grads(z.x, u.x, ga[i][b][0] * wt[b].x, kAct, g0, u0, a0);
          gate_grads(z.y, u.y, ga[i][b][1] * wt[b].y, kAct, g1, u1, a1);
          const bool in = f0 + 8 * i < F;        // columns beyond F hold what the sums of nothing times a NaN are
          dot[b][0] = in ? fmaf(a0, ga[i][b][0], dot[b][0]) : dot[b][0];
          dot[b][1] = in ? fmaf(a1, ga[i][b][1], dot[b][1]) : dot[b][1];
          og[i] = pack2<F16>(g0, g1);
          ou[i] = pack2<F16>(u0, u1);
          oa[i] = pack2<F16>(a0 * wt[b].x, a1 * wt[b].y);
        }
        const uint32_t at = s0 + frag + b * 8 * kPitch64;
        frag_st_t(at, og[0], og[1], og[2], og[3]);
        frag_st_t(at + 16 * kPitch64, ou[0], ou[1], ou[2], ou[3]);
        frag_st_t(at + 32 * kPitch64, oa[0], oa[1], oa[2], oa[3]);
      }
      __syncwarp();
      flush64<16>(buf, reinterpret_cast<uint8_t*>(gg + row0 * 2 * F + f0), (size_t)F * 4, rows, pieces, lane);
      flush64<16>(buf + 16 * kPitch64, reinterpret_cast<uint8_t*>(gg + (row0 * 2 + 1) * F + f0), (size_t)F * 4, rows, pieces, lane);
      flush64<16>(buf + 32 * kPitch64, reinterpret_cast<uint8_t*>(wa + row0 * F + f0), (size_t)F * 2, rows, pieces, lane);
#pragma unroll
      for (int o = 4; o < 32; o <<= 1)
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int e = 0; e < 2; ++e) dot[b][e] += __shfl_xor_sync(0xFFFFFFFFu, dot[b][e], o);
      if (lane < 8) {                            // lane 4 b + n has tokens 8 b + 2 n and the next
        const int r = 8 * (lane >> 2) + 2 * (lane & 3);
        float* to = part + (long long)(f0 >> 5) * cap_rows + row0 + r;
        const float x = lane < 4 ? dot[0][0] : dot[1][0], y = lane < 4 ? dot[0][1] : dot[1][1];
        if (r < rows) to[0] = x;
        if (r + 1 < rows) to[1] = y;
      }
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
  uint8_t* lo;                                 // their lower planes, rows of rows_low_pitch
};
cudaError_t launch_experts_forward(const ExpertsFwdLaunch& L, bool f16, cudaStream_t s);

struct ExpertsBwdLaunch {
  CUtensorMap wd_mn, wgu_mn, gy[4], gg[4];
  CUtensorMap gg_mn, xs_mn, gy_mn, wa_mn, xs_narrow, wa_narrow;
  int wd_blocks, wgu_blocks;                   // ExpertsJob::blocks
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

inline int rows_low_pitch(int D) { return (D + 15) & ~15; }

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
  j.blocks = 0;
  j.head = p.head;
  j.E = p.E;
  j.width = p.width;
  j.cap_rows = p.cap_rows;
  j.cap_tiles = p.cap_tiles;
  j.table = p.table;
  j.tiles_m = (m + per_tile - 1) / per_tile;
  j.kiters = (depth + kFfnTileK - 1) / kFfnTileK;
  j.by_m = FastDiv((uint32_t)j.tiles_m);
  return j;
}

// Launches of the row kernels: blocks of eight warps.
template <class K, class... A>
cudaError_t launch_rows(K* k, long long warps, bool dependent, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)((warps + 7) / 8));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = dependent ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, k, args...);
}

// out[t] = sum_j w_tj rows[place_tj] of 24-bit rows, in the order of j; w = 1 without
// weights.  A warp takes 256 columns of a token, eight a lane, eight experts in flight.
// Bound by HBM: 68 us for 8 rows each of 4096 tokens of 4096 columns (436 MB: 6.4 TB/s; 77
// with as many blocks as fit at once, each taking more in turn).
template <bool F16>
__device__ __forceinline__ void combine_item(long long item, int segs, int k, int D, const int* places, const float* weights,
                                             int cap_rows, const uint16_t* hi, const uint8_t* lo, int lo_pitch, uint16_t* out,
                                             int lane) {
  const long long t = item / segs;
  const int c0 = (int)(item - t * segs) * 256 + lane * 8;
  float s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) s[i] = 0.0f;
  int at = lane < k ? places[t * k + lane] : -1;
  if (at >= cap_rows) at = -1;
  const float wt = lane < k && weights ? weights[t * k + lane] : 1.0f;
  // a lane's eight low bytes are every second of sixteen, from the first or the second on
  const uint32_t pick0 = (c0 & 8) ? 0x1050u : 0x1040u, pick1 = (c0 & 8) ? 0x3270u : 0x3260u;
#pragma unroll 1
  for (int j0 = 0; j0 < k; j0 += 4) {
    uint4 v[4], l[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int p = __shfl_sync(0xFFFFFFFFu, at, (j0 + j) & 31);
      v[j] = l[j] = make_uint4(0, 0, 0, 0);
      if (j0 + j < k && p >= 0 && c0 < D) {
        v[j] = *reinterpret_cast<const uint4*>(hi + (size_t)p * D + c0);
        l[j] = *reinterpret_cast<const uint4*>(lo + (size_t)p * lo_pitch + (c0 & ~15));
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int p = __shfl_sync(0xFFFFFFFFu, at, (j0 + j) & 31);
      float w = __shfl_sync(0xFFFFFFFFu, wt, (j0 + j) & 31);
      if (j0 + j >= k || p < 0) w = 0.0f;
      const uint32_t u[4] = {v[j].x, v[j].y, v[j].z, v[j].w}, b[4] = {l[j].x, l[j].y, l[j].z, l[j].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // {0, low byte, upper half}: byte 0 is whatever comes after the 24 bits
        s[2 * i] = fmaf(w, __uint_as_float(__byte_perm(u[i], b[i], pick0) & 0xFFFFFF00u), s[2 * i]);
        s[2 * i + 1] = fmaf(w, __uint_as_float(__byte_perm(u[i], b[i], pick1) & 0xFFFFFF00u), s[2 * i + 1]);
      }
    }
  }
  if (c0 < D) *reinterpret_cast<uint4*>(out + (size_t)t * D + c0) = pack8v<F16>(s);
}

// Copies of a token's row to the rows of its slots: a warp takes 512 columns, two pieces a
// lane, reads them once and writes them k times.  (A warp for each written row read x k
// times, beyond the L2 where the writes had replaced it: 66 us for 8 copies of 4096 rows of
// 4096 columns and 74 for 4 of 8192; so it is 49 and 54, 6.1 and 6.2 TB/s, with a block for
// every eight warps; with as many blocks as fit at once, each taking more in turn, 56 and 63.)
constexpr int kGatherCols = 512;
__device__ __forceinline__ void gather_item(int k, int at, int c0, int D, const uint16_t* from, uint16_t* to) {
  uint4 v[2];
#pragma unroll
  for (int h = 0; h < 2; ++h)
    if (c0 + 256 * h < D) v[h] = *reinterpret_cast<const uint4*>(from + c0 + 256 * h);
#pragma unroll 4
  for (int j = 0; j < k; ++j) {
    const int p = __shfl_sync(0xFFFFFFFFu, at, j);
    if (p < 0) continue;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (c0 + 256 * h < D) *reinterpret_cast<uint4*>(to + (size_t)p * D + c0 + 256 * h) = v[h];
  }
}
__device__ __forceinline__ void zero_item(int row, int c0, int D, uint16_t* to) {
#pragma unroll
  for (int h = 0; h < 2; ++h)
    if (c0 + 256 * h < D) *reinterpret_cast<uint4*>(to + (size_t)row * D + c0 + 256 * h) = make_uint4(0, 0, 0, 0);
}

// Rows of padding behind expert e's: [first, last).
__device__ __forceinline__ void padding_rows(const PlanView& p, int e, int* first, int* last) {
  const long long f = (long long)p.starts[e] + p.counts[e], l = p.starts[e + 1];
  *first = (int)max(0ll, min(f, (long long)p.cap_rows));
  *last = (int)max((long long)*first, min(min(l, f + kPlanPad - 1), (long long)p.cap_rows));
}

}  // namespace mhc
