// mhc_orth.cu -- orthogonalised updates (include/mhc_orth.h): norm, scaled fp16 copy,
// and the Newton-Schulz products on the tensor cores.
//
// Kept in fp16 by powers of two: X as S X, S near sqrt(max(rows, cols)), so that an
// orthogonal X has entries of size one; A as 2^12 A (its diagonal is near one, its other
// entries as small as 2^-18); b A + c A A as a power that leaves it below 2^15 for
// singular values up to 1.4.  Every product's epilogue applies its factors in fp32.
// A and A A are symmetric: tiles on and below the diagonal are formed, the others
// written from them.  Few deep tiles are cut along the depth.  Bound by the tensor cores and their power: five steps of a 4096 x 8192
// matrix take 1.71 ms (1.27 at the rate of a burst), of 32 of 2816 x 1024 1.52 (0.84).
#include <math.h>

#include "mhc_group_gemm.cuh"
#include "mhc_host.cuh"
#include "../../include/mhc_ffn.h"
#include "../../include/mhc_orth.h"

namespace mhc {
namespace {

constexpr int kNormBlock = 16384;                // elements that one block of the norm sums at least
constexpr int kNormBlocks = 1216;                // blocks in all, at least one a matrix: eight an SM (608: 41 us for 32 of 2816 x 1024, not 37)

__device__ __forceinline__ float pow2f(int e) { return __int_as_float((e + 127) << 23); }   // e in [-126, 127]

template <int kType>
__device__ __forceinline__ void load8(const void* p, long long at, long long end, bool whole, float (&v)[8]) {
  if (whole) {
    if constexpr (kType == MHC_DTYPE_FP32) {
      const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
      const float4 b = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + at + 4);
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
      const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at);
      const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 t = unpack2<kType == MHC_DTYPE_FP16>(w[i]);
        v[2 * i] = t.x;
        v[2 * i + 1] = t.y;
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = 0.0f;
    if (at + i < end) {
      if constexpr (kType == MHC_DTYPE_FP32) v[i] = static_cast<const float*>(p)[at + i];
      else if constexpr (kType == MHC_DTYPE_BF16) v[i] = __bfloat162float(static_cast<const __nv_bfloat16*>(p)[at + i]);
      else v[i] = __half2float(static_cast<const __half*>(p)[at + i]);
    }
  }
}

// The exponent of a positive fp64 number (no subnormal), and a power of two.
__device__ __forceinline__ int exponent(double v) { return ((__double2hiint(v) >> 20) & 0x7FF) - 1023; }
__device__ __forceinline__ double pow2d(int e) { return __hiloint2double((e + 1023) << 20, 0); }

// Sums of squares of one block's part of a matrix.  A thread's 128 bytes (64 values, or 32 of
// fp32) share a power of two that brings the largest near one, so no square over- or
// underflows; a thread's sum (compensated) and a warp's are an fp32 number and such a power,
// a block's is fp64.
// (184 MB: 80 us with an fp64 addition for every eight values, 43 with one a thread and step
// and for the sum over the block, 37 now: 5.0 TB/s.)
template <int kType>
__global__ void __launch_bounds__(256) orth_norm_kernel(uint32_t* header, const void* x, long long count, bool whole, double* part) {
  constexpr int kV = kType == MHC_DTYPE_FP32 ? 4 : 8;          // groups of eight values
  constexpr long long kUnit = 256 * 8;                         // a group of each thread
  __shared__ float room[8];
  __shared__ int room_e[8];
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x < 8) header[threadIdx.x] = 0u;
  pdl_trigger();
  const long long base = (long long)blockIdx.y * count, end = base + count, units = (count + kUnit - 1) / kUnit;
  const long long last = min(units * (blockIdx.x + 1) / gridDim.x * kUnit, count);
  float acc = 0.0f, low = 0.0f;                  // (acc - low) 4^at, at the largest exponent so far
  int at = -126;
  for (long long i0 = units * blockIdx.x / gridDim.x * kUnit + threadIdx.x * 8; i0 < last; i0 += kV * kUnit) {
    float v[kV][8];
#pragma unroll
    for (int b = 0; b < kV; ++b) {
      const long long i = i0 + b * kUnit;
      if (i < last) {
        load8<kType>(x, base + i, end, whole, v[b]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[b][j] = 0.0f;
      }
    }
    float top = 0.0f;
    if (kType != MHC_DTYPE_FP16) {               // whose squares fp32 holds as they are
#pragma unroll
      for (int b = 0; b < kV; ++b)
#pragma unroll
        for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(v[b][j]));
    }
    const int e = kType == MHC_DTYPE_FP16 ? 0 : min(max((int)(__float_as_uint(top) >> 23) - 127, -126), 126);   // of a subnormal -126
    const float f = pow2f(-e);                   // leaves the largest below 4
    float s[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) s[j] = 0.0f;
#pragma unroll
    for (int b = 0; b < kV; ++b)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float q = kType == MHC_DTYPE_FP16 ? v[b][j] : v[b][j] * f;
        s[j] = fmaf(q, q, s[j]);
      }
    const float sum = ((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]));   // not finite: nor were all values
    const int most = max(at, e);
    const float old = pow2f(max(2 * (at - most), -126)), y = fmaf(sum, pow2f(max(2 * (e - most), -126)), -low * old);
    acc *= old;
    const float t = acc + y;                     // compensated: a block may add thousands
    low = (t - acc) - y;
    acc = sum < INFINITY ? t : NAN;
    at = most;
  }
  const int most = __reduce_max_sync(0xFFFFFFFFu, at);
  acc *= pow2f(max(2 * (at - most), -126));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xFFFFFFFFu, acc, o);
  if ((threadIdx.x & 31) == 0) {
    room[threadIdx.x >> 5] = acc;
    room_e[threadIdx.x >> 5] = most;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    double sum = 0.0;
#pragma unroll
    for (int w = 0; w < 8; ++w) sum = fma((double)room[w], pow2d(2 * room_e[w]), sum);
    part[(size_t)blockIdx.y * gridDim.x + blockIdx.x] = sum;
  }
}

// S x / (norm + eps) in fp16, rows of `pitch`: 184 MB of bf16 to as many take 62 us (6.0
// TB/s; 75 with the factor from fp64 roots and quotients in every thread).
template <int kType>
__global__ void __launch_bounds__(256) orth_scale_kernel(const void* x, int rows, int cols, int pitch, bool whole,
                                                         const double* part, int parts, float eps, double S, uint16_t* out) {
  __shared__ double room[8];
  __shared__ float factor[2];
  pdl_trigger();
  pdl_wait();
  if ((int)(threadIdx.x & ~31u) < parts) {
    double s = 0.0;
    for (int i = threadIdx.x; i < parts; i += 256) s += part[(size_t)blockIdx.y * parts + i];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    if ((threadIdx.x & 31) == 0) room[threadIdx.x >> 5] = s;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    double s = room[0];
    for (int w = 1; w < 8 && w * 32 < parts; ++w) s += room[w];
    // root and quotient in fp32 of what is left beside powers of two
    int e = exponent(s) >> 1;
    const double norm = s == 0.0 ? 0.0 : (double)sqrtf((float)(s * pow2d(-2 * e))) * pow2d(e), d = norm + (double)eps;
    e = exponent(d);
    const float q = (float)S / (float)(d * pow2d(-e));
    // S / d as f0 f1, both within fp32
    e = min(max(-e, -200), 200);
    factor[0] = d == 0.0 ? 0.0f : pow2f(e >> 1);
    factor[1] = d == 0.0 ? 0.0f : d != d ? NAN : q * pow2f(e - (e >> 1));
  }
  __syncthreads();
  const float f0 = factor[0], f1 = factor[1];
  const int groups = pitch / 8;
  const long long base = (long long)blockIdx.y * rows, items = (long long)rows * groups;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < items; i += (long long)gridDim.x * 256) {
    const int r = (int)(i / groups), c = (int)(i - (long long)r * groups) * 8;
    float v[8];
    const long long at = (base + r) * cols + c;
    load8<kType>(x, at, at - c + cols, whole, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = v[j] * f0 * f1;
    *reinterpret_cast<uint4*>(out + (size_t)(base + r) * pitch + c) = pack8v<true>(v);
  }
}

// Products of a batch of matrices.  kSym: A = B, tiles on and below the diagonal.
template <bool kA, bool kB, bool kSym>
struct OrthJob {
  static constexpr bool kAMn = kA, kBMn = kB, kDraw = false, kEarly = false;
  CUtensorMap a, b;              // MN-major: blocks of 64 columns are a dimension of their own
                                 // (b's of tiles narrower than 256 not)
  CUtensorMap b_half;            // b's of the tiles from `whole` on
  int whole;                     // tiles before these are whole; each later one is half a tile
  GemmShape g;                   // tiles of one matrix
  int count, per, width, kiters;
  int split;                     // log2(256 / width)
  int parts, part_kiters;        // of the depth, tiles of their own: `row0` is a tile's first chunk, `rows` its part
  FastDiv by_matrix, by_parts;

  struct Raw {};
  __device__ __forceinline__ void prefetch() const {
    tma_prefetch_desc(&a);
    tma_prefetch_desc(&b);
  }
  __device__ __forceinline__ int tiles() const { return count; }
  __device__ __forceinline__ Raw fetch(int) const { return {}; }
  __device__ __forceinline__ GTile make(int t, const Raw&) const {
    GTile o;
    int half = 0;
    const bool halved = t >= whole;
    if (halved) {                // the last round's few tiles in halves, for twice as many pairs
      half = (t - whole) & 1;
      t = whole + ((t - whole) >> 1);
    }
    o.e = by_matrix(t);
    const int r = t - o.e * per;
    if constexpr (kSym) {        // row tm begins at tm (tm + 1) / 2 squares of 256
      const int sq = r >> split;
      int tm = (int)((sqrtf(8.0f * (float)sq + 1.0f) - 1.0f) * 0.5f);
      while ((tm + 1) * (tm + 2) / 2 <= sq) ++tm;
      while (tm * (tm + 1) / 2 > sq) --tm;
      o.tm = tm;
      o.tn = r - ((tm * (tm + 1) / 2) << split);
      o.kind = o.tn < (tm << split);             // below the diagonal: its mirror is written too
    } else {
      tile_coords(g, r, o.tm, o.tn);
      o.kind = 0;
    }
    o.row0 = o.rows = 0;
    o.width = halved ? width >> 1 : width;
    if (halved) o.tn = 2 * o.tn + half;
    o.kiters = kiters;
    if (parts > 1) {
      const int e = by_parts(o.e);
      o.rows = o.e - e * parts;
      o.e = e;
      o.row0 = o.rows * part_kiters;
      o.kiters = min(part_kiters, kiters - o.row0);
    }
    return o;
  }
  __device__ __forceinline__ int bytes(const GTile& o) const {
    const int half = o.width >> 1;
    return kGemmOpBytes + (kB ? (half + 63) & ~63 : half) * kFfnTileK * 2;
  }
  __device__ __forceinline__ int steps(const GTile&, int) const { return kFfnTileK / 16; }
  __device__ __forceinline__ uint32_t idesc(const GTile& o) const { return grp_idesc(true, kA, kB, o.width); }
  __device__ __forceinline__ void load_a(const GTile& o, int k, uint32_t sa, uint32_t bar, int rank) const {
    const int k0 = (o.row0 + k) * kFfnTileK, m0 = o.tm * kFfnTileM + rank * kGemmHalf;
    if constexpr (kA) {
      tma_load_4d_pair(sa, &a, bar, 0, k0, m0 >> 6, o.e);
    } else {
      tma_load_3d_pair(sa, &a, bar, k0, m0, o.e);
    }
  }
  __device__ __forceinline__ void load_b(const GTile& o, int k, uint32_t sb, uint32_t bar, int rank) const {
    const int k0 = (o.row0 + k) * kFfnTileK, n0 = o.tn * o.width + rank * (o.width >> 1);
    const CUtensorMap* t = o.width == width ? &b : &b_half;
    if constexpr (kB) {
      if (o.width > 128) tma_load_4d_pair(sb, t, bar, 0, k0, n0 >> 6, o.e);
      else tma_load_3d_pair(sb, t, bar, n0, k0, o.e);
    } else {
      tma_load_3d_pair(sb, t, bar, k0, n0, o.e);
    }
  }
};

// out = alpha c + beta acc.  fp16 matrices of `pitch` columns (columns behind the last
// are never read), or with kLast the result itself.  kSym writes the tile's mirror too.
// What the fp16 of A's diagonal leaves goes into that of b A + c A A (to first order, by its
// own square's diagonal), and what that leaves into the factor of X's rows or, kCols,
// columns.  Of a matrix of few rows these are all that counts: A is then nearly a multiple
// of 1, each row's roundings are one of A's and one of b A + c A A, and the iteration grows
// them up to tenfold (results without: 1.2 to 3.4 times their own bf16 rounding off, now
// 1.05 to 1.2).
template <bool kHasC, bool kSym, int kLast, bool kCols>  // kLast: 0 fp16 between products, 1 bf16 result, 2 fp16 result
struct EpiOrth {
  const float* left;             // by the diagonal of c (kSym) or of the other operand
  float* leaves;                 // what this one's leaves (kSym); rows of side_pitch
  int side_pitch;
  const uint16_t* c;
  uint16_t* out;
  int M, N, pitch;               // of c and of out but the result's, whose pitch is N
  float alpha, beta;
  bool whole;                    // the result's rows are 16-byte aligned
  // c of two steps of 32 columns, the first two loaded before the tile's sums are there:
  // rows i * 8 + lane / 4, eight columns; and what the diagonal leaves, of these rows
  struct Pre {
    uint4 w[2][4];
    float rows[4];
  };
  __device__ __forceinline__ void load(Pre& p, int h, const GTile& g, int m0, int c0, int lane) const {
    const int col = c0 + (lane & 3) * 8;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = m0 + i * 8 + (lane >> 2);
      p.w[h][i] = make_uint4(0, 0, 0, 0);
      if (row < M && c0 < N && col < pitch) p.w[h][i] = *reinterpret_cast<const uint4*>(c + ((size_t)g.e * M + row) * pitch + col);
    }
  }
  __device__ __forceinline__ void pre(const GTile& g, Pre& p, int rank, int q, int grp, int lane) const {
    if constexpr (kHasC) {
      const int m0 = g.tm * kFfnTileM + rank * kGemmHalf + q * 32, half = g.width >> 1, c0 = g.tn * g.width + grp * half;
      load(p, 0, g, m0, c0, lane);
      load(p, 1, g, m0, half > 32 ? c0 + 32 : N, lane);
      if constexpr (!kCols) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = m0 + i * 8 + (lane >> 2);
          p.rows[i] = row < M ? left[(size_t)g.e * side_pitch + row] : 0.0f;
        }
      }
    }
  }
  __device__ __forceinline__ void step(const GTile& g, Pre& ahead, int h, int col, int end, int m0, uint32_t taddr, uint8_t* buf,
                                       int lane) const {
    constexpr bool kF16 = kLast != 1;
    const int c0 = g.tn * g.width + col;
    const size_t plane = (size_t)g.e * M;
    const uint32_t frag = smem_u32(buf) + (lane & 7) * kPitch64 + (lane >> 3) * 16;
    float2 f[4];                                 // factors of c, the columns'
    if constexpr (kCols) {
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int n = c0 + b * 8 + (lane & 3) * 2;
        f[b] = make_float2(0.0f, 0.0f);
        if (n < N) f[b] = *reinterpret_cast<const float2*>(left + (size_t)g.e * side_pitch + n);
        f[b] = make_float2(fmaf(beta, f[b].x, alpha), fmaf(beta, f[b].y, alpha));
      }
    }
    if constexpr (kHasC) {
#pragma unroll
      for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4*>(buf + (i * 8 + (lane >> 2)) * kPitch64 + (lane & 3) * 16) = ahead.w[h][i];
      load(ahead, h, g, m0, col + 64 < end ? c0 + 64 : N, lane);
      __syncwarp();
    }
    float v[4][4][2];
    frag_ld<4>(taddr + col, v);
    uint32_t w[4][4];
    // elements of the diagonal: of lanes whose row of eight is one of their two columns
    float at[4], was[4];
    const bool second = (lane >> 2) & 1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t k[4] = {0, 0, 0, 0};
      if constexpr (kHasC) frag_lds(frag + i * 8 * kPitch64, k);
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const float2 t = unpack2<true>(k[b]);
        float x = beta * v[i][b][0], y = beta * v[i][b][1];
        if constexpr (kHasC) {
          const float row = kSym ? alpha : fmaf(beta, ahead.rows[i], alpha);
          x = fmaf(beta, v[i][b][0], (kCols ? f[b].x : row) * t.x);
          y = fmaf(beta, v[i][b][1], (kCols ? f[b].y : row) * t.y);
        }
        w[i][b] = pack2<kF16>(x, y);
        if (kSym && i == b) at[i] = second ? y : x;
        if (kSym && kHasC && i == b) was[i] = second ? t.y : t.x;
      }
    }
    if constexpr (kSym) {
      if (c0 == m0 && lane >> 3 == (lane & 3)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = m0 + i * 8 + (lane >> 2);
          if constexpr (kHasC) at[i] = fmaf(ahead.rows[i], fmaf(2.0f * beta, was[i], alpha), at[i]);
          const uint32_t r = pack2<true>(at[i], at[i]);
          w[i][i] = second ? __byte_perm(w[i][i], r, 0x5410) : __byte_perm(w[i][i], r, 0x3254);
          if (row < M) leaves[(size_t)g.e * side_pitch + row] = at[i] - unpack2<true>(r).x;
        }
      }
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) frag_st(frag + i * 8 * kPitch64, w[i][0], w[i][1], w[i][2], w[i][3]);
    __syncwarp();
    if (kLast == 0) {
      flush64<32>(buf, reinterpret_cast<uint8_t*>(out + (plane + m0) * pitch + c0), (size_t)pitch * 2, M - m0, (pitch - c0) >> 3, lane);
    } else if (whole) {
      flush64<32>(buf, reinterpret_cast<uint8_t*>(out + (plane + m0) * N + c0), (size_t)N * 2, M - m0, (N - c0) >> 3, lane);
    } else {
      const int rows = min(32, M - m0);
      if (c0 + lane < N)
        for (int r = 0; r < rows; ++r)
          out[(plane + m0 + r) * N + c0 + lane] = *reinterpret_cast<const uint16_t*>(buf + r * kPitch64 + lane * 2);
    }
    if constexpr (kSym) {
      if (g.kind) {
        __syncwarp();
#pragma unroll
        for (int b = 0; b < 4; ++b) frag_st_t(frag + b * 8 * kPitch64, w[0][b], w[1][b], w[2][b], w[3][b]);
        __syncwarp();
        flush64<32>(buf, reinterpret_cast<uint8_t*>(out + (plane + c0) * pitch + m0), (size_t)pitch * 2, N - c0, (pitch - m0) >> 3, lane);
      }
    }
    __syncwarp();
  }
  __device__ __forceinline__ void tile(const GTile& g, Pre& ahead, int, int, uint32_t taddr, int rank, int q, int grp, uint8_t* buf,
                                       int lane, int) const {
    const int m0 = g.tm * kFfnTileM + rank * kGemmHalf + q * 32, n0 = g.tn * g.width, half = g.width >> 1;
    if (m0 >= M) return;
    const int beg = grp * half, end = beg + half;
#pragma unroll 1
    for (int col = beg; col < end && n0 + col < N; col += 64) {
      step(g, ahead, 0, col, end, m0, taddr, buf, lane);
      if (col + 32 < end && n0 + col + 32 < N) step(g, ahead, 1, col + 32, end, m0, taddr, buf, lane);
    }
  }
};

// A part's sums as they are, for the kernel below to join.
struct EpiParts {
  float* room;                   // [matrix][part][M][pitch]
  int M, pitch, parts;
  using Pre = NoPre;
  __device__ __forceinline__ void pre(const GTile&, NoPre&, int, int, int, int) const {}
  __device__ __forceinline__ void tile(const GTile& g, NoPre&, int, int, uint32_t taddr, int rank, int q, int grp, uint8_t*, int lane,
                                       int) const {
    const int m0 = g.tm * kFfnTileM + rank * kGemmHalf + q * 32, n0 = g.tn * g.width, half = g.width >> 1;
    if (m0 >= M) return;
    float* to = room + ((size_t)g.e * parts + g.rows) * M * pitch;
#pragma unroll 1
    for (int col = grp * half; col < (grp + 1) * half && n0 + col < pitch; col += 32) {
      float v[4][4][2];
      frag_ld<4>(taddr + col, v);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = m0 + i * 8 + (lane >> 2);
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const int n = n0 + col + b * 8 + (lane & 3) * 2;
          if (row < M && n < pitch) *reinterpret_cast<float2*>(to + (size_t)row * pitch + n) = make_float2(v[i][b][0], v[i][b][1]);
        }
      }
    }
  }
};

// A = beta times the sum of the parts in their order, and what its diagonal leaves.  Squares
// of 256 on and below the diagonal are there; a block takes 32 x 32 and writes its mirror.
__global__ void __launch_bounds__(256) orth_join_kernel(const float* room, int parts, int side, int pitch, int blocks, float beta,
                                                        uint16_t* out, float* leaves) {
  __shared__ uint16_t tile[32][33];
  pdl_trigger();
  const int bi = blockIdx.x / blocks, i0 = bi * 32, j0 = ((int)blockIdx.x - bi * blocks) * 32;
  const bool mirror = i0 >> 8 != j0 >> 8;
  if (i0 >> 8 < j0 >> 8) return;
  pdl_wait();
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5, j = j0 + tx;
  const size_t plane = (size_t)side * pitch;
  const float* from = room + (size_t)blockIdx.y * parts * plane;
  uint16_t* to = out + (size_t)blockIdx.y * plane;
  float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
  for (int p = 0; p < parts; ++p)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int i = i0 + ty + 8 * q;
      if (i < side && j < side) s[q] += from[p * plane + (size_t)i * pitch + j];
    }
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int i = i0 + ty + 8 * q;
    const float v = s[q] * beta;
    const __half h = __float2half_rn(v);
    const uint16_t w = __half_as_ushort(h);
    tile[ty + 8 * q][tx] = w;
    if (i < side && j < side) {
      to[(size_t)i * pitch + j] = w;
      if (i == j) leaves[(size_t)blockIdx.y * pitch + i] = v - __half2float(h);
    }
  }
  if (mirror) {
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int r = ty + 8 * q;
      if (j0 + r < side && i0 + tx < side) to[(size_t)(j0 + r) * pitch + i0 + tx] = tile[tx][r];
    }
  }
}

// --------------------------------------------------------------------- host

// How a product's tiles are cut.  In times of a stage of a tile of 256 (0.28 us): a stage of
// 128 columns takes 0.6 and of 64 0.5 of it; an epilogue, 9 for 256 columns, runs beside the
// next tile's stages and after the last one's.  (515 x 259: three tiles of 256 or ten of 64.)
// A product X X^T whose few tiles are deep is cut along its depth too, into parts that leave
// few pairs idle and take eight chunks or more; another launch joins them (12).  Five steps
// of 128 x 16384: 368 -> 157 us, 1024 x 8192 317 -> 252, 1024 x 4096 222 -> 205.
struct Cut {
  int width, parts, part_kiters;
};
int64_t tiles_of(int64_t M, int64_t N, int w, bool sym) {
  const int64_t tm = (M + 255) / 256;
  return !sym ? tm * ((N + w - 1) / w) : tm == 1 ? (N + w - 1) / w : tm * (tm + 1) / 2 * (256 / w);
}
Cut cut(int64_t batch, int64_t M, int64_t N, int64_t K, bool sym, bool gram, int pairs) {
  const int64_t kiters = (K + kFfnTileK - 1) / kFfnTileK;
  Cut best = {256, 1, (int)kiters};
  double least = 1e30;
  for (int w = 256; w >= 64; w /= 2) {
    if (w > 64 && N <= w / 2) continue;
    const double stage = w == 256 ? 1.0 : w == 128 ? 0.6 : 0.5, epi = 9.0 * w / 256;
    const int64_t tiles = batch * tiles_of(M, N, w, sym);
    int64_t most = gram ? pairs / tiles : 1;
    if (most > kiters / 8) most = kiters / 8;
    for (int64_t parts = 1; parts <= (most > 1 ? most : 1); parts += most > 1 ? most - 1 : 1) {
      const int64_t each = (kiters + parts - 1) / parts;
      const double rounds = (double)((tiles * parts + pairs - 1) / pairs), main = each * stage;
      const double cost = rounds * (main > epi ? main : epi) + epi + (parts > 1 ? 12.0 : 0.0);
      if (cost < least) {
        least = cost;
        best = {w, (int)((kiters + each - 1) / each), (int)each};
      }
    }
  }
  return best;
}
constexpr int kPairs = 76;       // that products are cut for, whatever the device: a workspace's size goes by it

size_t up256(size_t v) { return (v + 255) & ~size_t(255); }

struct OrthLayout {
  int64_t parts, pitch, side, spitch;
  Cut gram;                      // X X^T
  size_t norm, left[2], x[2], p, q, room, total;
};
OrthLayout orth_layout(int64_t batch, int64_t rows, int64_t cols) {
  OrthLayout l;
  const int64_t count = rows * cols;
  l.parts = (count + kNormBlock - 1) / kNormBlock;
  const int64_t most = batch > kNormBlocks / 2 ? 1 : kNormBlocks / (batch > 0 ? batch : 1);
  if (l.parts > most) l.parts = most;
  l.pitch = (cols + 7) & ~int64_t(7);
  l.side = rows < cols ? rows : cols;
  l.spitch = (l.side + 7) & ~int64_t(7);
  const size_t xb = up256((size_t)batch * rows * l.pitch * 2), pb = up256((size_t)batch * l.side * l.spitch * 2);
  l.norm = 256;
  const size_t db = up256((size_t)batch * l.spitch * 4);
  l.left[0] = l.norm + up256((size_t)batch * l.parts * 8);
  l.left[1] = l.left[0] + db;
  l.x[0] = l.left[1] + db;
  l.x[1] = l.x[0] + xb;
  l.p = l.x[1] + xb;
  l.q = l.p + pb;
  l.gram = cut(batch, l.side, l.side, rows < cols ? cols : rows, true, true, kPairs);
  l.room = l.q + pb + 256;                      // orth_map_blocks reads a little past a buffer
  l.total = l.room + (l.gram.parts > 1 ? up256((size_t)batch * l.gram.parts * l.side * l.spitch * 4) : 0);
  return l;
}

bool orth_map(CUtensorMap* m, const void* base, int64_t cols, int64_t rows, int64_t pitch, int64_t batch, uint32_t box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t d[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)batch};
  cuuint64_t st[2] = {(cuuint64_t)pitch * 2, (cuuint64_t)(pitch * rows) * 2};
  cuuint32_t b[3] = {64, box_rows, 1}, es[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(base), d, st, b, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// MN-major: boxes of two blocks of 64 columns; the last block may run into a row's padding
// and the next row, whose results are not kept.
bool orth_map_blocks(CUtensorMap* m, const void* base, int64_t cols, int64_t rows, int64_t pitch, int64_t batch) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t d[4] = {64, (cuuint64_t)rows, (cuuint64_t)(cols + 63) / 64, (cuuint64_t)batch};
  cuuint64_t st[3] = {(cuuint64_t)pitch * 2, 128, (cuuint64_t)(pitch * rows) * 2};
  cuuint32_t b[4] = {64, kFfnBoxMn, 2, 1}, es[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, const_cast<void*>(base), d, st, b, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Matrix {
  void* p;
  int64_t rows, cols, pitch;
};

// One product: out = alpha c + beta (op A)(op B)^T.
struct Product {
  int64_t batch, M, N, K;
  GrpCall call;
  int sms;
  const float* left;             // EpiOrth
  float* leaves;
  int64_t side_pitch;
  const uint16_t* c;
  uint16_t* out;
  int64_t pitch;
  double alpha, beta;
  bool whole;
};
// A job over matrices a and b of a product cut as `c` says.
template <bool kA, bool kB, bool kSym>
bool orth_job(OrthJob<kA, kB, kSym>* job, const Product& p, const Matrix& a, const Matrix& b, const Cut& c) {
  job->width = c.width;
  job->split = c.width == 256 ? 0 : c.width == 128 ? 1 : 2;
  job->parts = c.parts;
  job->part_kiters = c.part_kiters;
  if (!(kA ? orth_map_blocks(&job->a, a.p, a.cols, a.rows, a.pitch, p.batch)
           : orth_map(&job->a, a.p, a.cols, a.rows, a.pitch, p.batch, (uint32_t)kGemmHalf)) ||
      !(kB && c.width > 128 ? orth_map_blocks(&job->b, b.p, b.cols, b.rows, b.pitch, p.batch)
                            : orth_map(&job->b, b.p, b.cols, b.rows, b.pitch, p.batch, kB ? kFfnBoxMn : (uint32_t)c.width / 2)))
    return false;
  GemmShape& g = job->g;
  g = GemmShape();
  g.tiles_m = (int)((p.M + kFfnTileM - 1) / kFfnTileM);
  g.tiles_n = (int)((p.N + c.width - 1) / c.width);
  g.band = 8;
  g.by_band = FastDiv((uint32_t)(g.band * g.tiles_n));
  g.by_rows = FastDiv((uint32_t)g.band);
  g.by_last = FastDiv((uint32_t)(g.tiles_m % g.band ? g.tiles_m % g.band : g.band));
  job->per = (int)tiles_of(p.M, p.N, c.width, kSym);
  job->count = (int)(job->per * p.batch * c.parts);
  job->by_matrix = FastDiv((uint32_t)job->per);
  job->by_parts = FastDiv((uint32_t)c.parts);
  job->kiters = (int)((p.K + kFfnTileK - 1) / kFfnTileK);
  job->whole = job->count;
  job->b_half = job->b;
  return true;
}

template <bool kA, bool kB, bool kHasC, bool kSym, int kLast>
cudaError_t product(const Product& p, const Matrix& a, const Matrix& b, bool* mapped, cudaStream_t s) {
  OrthJob<kA, kB, kSym> job;
  *mapped = orth_job(&job, p, a, b, cut(p.batch, p.M, p.N, p.K, kSym, false, p.sms / 2));
  if (!*mapped) return cudaErrorInvalidValue;
  // Where the last round has tiles for at most half the pairs, these are halved: 320 tiles of
  // 32 matrices of 1024, 5 rounds, now 4.6.
  const int pairs = p.sms / 2, over = job.count % pairs;
  if (job.width == 256 && job.count > pairs && over > 0 && 2 * over <= pairs) {
    job.whole = job.count - over;
    job.count += over;
    if (!orth_map(&job.b_half, b.p, b.cols, b.rows, b.pitch, p.batch, kB ? kFfnBoxMn : 64u)) {
      *mapped = false;
      return cudaErrorInvalidValue;
    }
  }
  const EpiOrth<kHasC, kSym, kLast, !kSym && !kB> e = {p.left, p.leaves, (int)p.side_pitch, p.c, p.out, (int)p.M, (int)p.N, (int)p.pitch, (float)p.alpha, (float)p.beta, p.whole};
  return launch_group(job, p.call, e, job.count, p.sms, true, s);
}

// A = beta X X^T (kMn: X^T X) in parts of the depth.
template <bool kMn>
cudaError_t gram(const Product& p, const Matrix& x, const Cut& c, float* room, bool* mapped, cudaStream_t s) {
  OrthJob<kMn, kMn, true> job;
  *mapped = orth_job(&job, p, x, x, c);
  if (!*mapped) return cudaErrorInvalidValue;
  const EpiParts epi = {room, (int)p.M, (int)p.pitch, c.parts};
  const cudaError_t e = launch_group(job, p.call, epi, job.count, p.sms, true, s);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  const unsigned blocks = (unsigned)((p.M + 31) / 32);
  cfg.gridDim = dim3(blocks * blocks, (unsigned)p.batch);
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, orth_join_kernel, static_cast<const float*>(room), c.parts, (int)p.M, (int)p.pitch, (int)blocks,
                            (float)p.beta, p.out, p.leaves);
}

template <int kType>
cudaError_t start(const mhc_orth_args& a, const OrthLayout& l, uint8_t* ws, double S, int sms, cudaStream_t s) {
  const long long count = a.rows * a.cols;
  const bool flat = count % 8 == 0 && aligned(a.x, 16), rows = a.cols % 8 == 0 && aligned(a.x, 16);
  double* part = reinterpret_cast<double*>(ws + l.norm);
  orth_norm_kernel<kType><<<dim3((unsigned)l.parts, (unsigned)a.batch), 256, 0, s>>>(reinterpret_cast<uint32_t*>(ws), a.x, count, flat, part);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  const long long items = a.rows * (l.pitch / 8), blocks = (items + 1023) / 1024;
  const long long most = (8ll * sms + a.batch - 1) / a.batch;
  cfg.gridDim = dim3((unsigned)(blocks < most ? blocks : most), (unsigned)a.batch);
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, orth_scale_kernel<kType>, a.x, (int)a.rows, (int)a.cols, (int)l.pitch, rows,
                            static_cast<const double*>(part), (int)l.parts, a.eps, S, reinterpret_cast<uint16_t*>(ws + l.x[0]));
}

}  // namespace
}  // namespace mhc

using namespace mhc;

extern "C" {

mhc_status_t mhc_orth_workspace_size(int64_t batch, int64_t rows, int64_t cols, size_t* bytes) {
  clear_error();
  if (!bytes) return fail(MHC_ERR_NULLPTR, "bytes must be non-NULL");
  if (batch < 0 || batch > 65535) return fail(MHC_ERR_PARAM_INVALID, "batch must be in [0, 65535] (got %lld)", (long long)batch);
  if (rows < 1 || rows > 32768 || cols < 1 || cols > 32768)
    return fail(MHC_ERR_PARAM_INVALID, "rows and cols must be in [1, 32768] (got %lld, %lld)", (long long)rows, (long long)cols);
  *bytes = batch ? orth_layout(batch, rows, cols).total : 0;
  return MHC_OK;
}

mhc_status_t mhc_orth_run(const mhc_orth_args* a, void* stream) {
  clear_error();
  if (!a) return fail(MHC_ERR_NULLPTR, "args must be non-NULL");
  size_t need = 0;
  mhc_status_t st = mhc_orth_workspace_size(a->batch, a->rows, a->cols, &need);
  if (st != MHC_OK) return st;
  if (a->dtype != MHC_DTYPE_BF16 && a->dtype != MHC_DTYPE_FP16 && a->dtype != MHC_DTYPE_FP32)
    return fail(MHC_ERR_PARAM_INVALID, "dtype must be MHC_DTYPE_BF16, _FP16 or _FP32 (got %d)", (int)a->dtype);
  if (a->out_dtype != MHC_DTYPE_BF16 && a->out_dtype != MHC_DTYPE_FP16)
    return fail(MHC_ERR_PARAM_INVALID, "out_dtype must be MHC_DTYPE_BF16 or MHC_DTYPE_FP16 (got %d)", (int)a->out_dtype);
  if (a->steps < 1 || a->steps > 32) return fail(MHC_ERR_PARAM_INVALID, "steps must be in [1, 32] (got %d)", (int)a->steps);
  if (!(a->eps >= 0.0f) || !isfinite(a->eps)) return fail(MHC_ERR_PARAM_INVALID, "eps must be finite and not negative");
  if (a->wait_limit_us > 10000000u) return fail(MHC_ERR_PARAM_INVALID, "wait_limit_us must be at most 10 s");
  if (a->withhold_copy != 0 && a->withhold_copy != 1) return fail(MHC_ERR_PARAM_INVALID, "withhold_copy must be 0 or 1");
  if (!a->coefficients) return fail(MHC_ERR_NULLPTR, "coefficients are required");
  for (int i = 0; i < 3 * a->steps; ++i)
    if (!isfinite(a->coefficients[i]) || fabsf(a->coefficients[i]) > 1000.0f)
      return fail(MHC_ERR_PARAM_INVALID, "coefficients must be finite and at most 1000 in size");
  if (a->batch == 0) return MHC_OK;
  if (!a->x || !a->out || !a->workspace) return fail(MHC_ERR_NULLPTR, "x, out and the workspace are required");
  const size_t esize = a->dtype == MHC_DTYPE_FP32 ? 4 : 2, count = (size_t)a->batch * a->rows * a->cols;
  if (!aligned(a->x, esize) || !aligned(a->out, 2) || !aligned(a->workspace, 256))
    return fail(MHC_ERR_PARAM_INVALID, "x and out must be aligned to their elements, the workspace to 256 bytes");
  if (a->workspace_bytes < need)
    return fail(MHC_ERR_PARAM_INVALID, "workspace too small: %zu bytes given, %zu needed", a->workspace_bytes, need);
  const OrthLayout l = orth_layout(a->batch, a->rows, a->cols);
  const int64_t tiles = ((a->rows + 255) / 256) * ((a->cols + 63) / 64) * a->batch;
  if (tiles > (int64_t(1) << 30)) return fail(MHC_ERR_PARAM_INVALID, "too many tiles");
  if ((st = check_apart({{"out", a->out, count * 2}, {"workspace", a->workspace, l.total}}, {{"x", a->x, count * esize}})) != MHC_OK)
    return st;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return fail(MHC_ERR_RUNTIME, "no CUDA device");
  const DeviceInfo di = device_info(dev);
  if (!di.ok) return fail(MHC_ERR_RUNTIME, "device %d is not an sm_103 GPU", dev);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(a->workspace);
  const int64_t m = a->rows, n = a->cols, side = l.side;
  const bool tall = m > n;
  const double S = ldexp(1.0, (int)lround(0.5 * log2((double)(m > n ? m : n)))), SA = 4096.0;
  cudaError_t e = a->dtype == MHC_DTYPE_FP32   ? start<MHC_DTYPE_FP32>(*a, l, ws, S, di.sms, s)
                  : a->dtype == MHC_DTYPE_BF16 ? start<MHC_DTYPE_BF16>(*a, l, ws, S, di.sms, s)
                                               : start<MHC_DTYPE_FP16>(*a, l, ws, S, di.sms, s);
  if (e != cudaSuccess) return fail(MHC_ERR_RUNTIME, "orthogonalisation launch failed: %s", cudaGetErrorString(e));
  Product p = {};
  p.batch = a->batch;
  p.call.err = reinterpret_cast<uint32_t*>(ws);
  p.call.counter = nullptr;
  p.call.wait_ns = a->wait_limit_us ? (uint64_t)a->wait_limit_us * 1000u : 2000000000ull;
  grp_ring(&p.call, 128);
  p.sms = di.sms;
  p.side_pitch = l.spitch;
  float *left_a = reinterpret_cast<float*>(ws + l.left[0]), *left_b = reinterpret_cast<float*>(ws + l.left[1]);
  Matrix A = {ws + l.p, side, side, l.spitch}, B = {ws + l.q, side, side, l.spitch};
  for (int i = 0; i < a->steps; ++i) {
    const double ca = a->coefficients[3 * i], cb = a->coefficients[3 * i + 1], cc = a->coefficients[3 * i + 2];
    const double bound = fmax(2.0 * fabs(cb) + 4.0 * fabs(cc), 1.0);
    const double SB = ldexp(1.0, (int)floor(log2(32768.0 / bound)));
    const bool last = i + 1 == a->steps;
    Matrix X = {ws + l.x[i & 1], m, n, l.pitch};
    bool mapped = true;
    p.call.withhold = 0;
    p.M = p.N = side;
    p.K = tall ? m : n;
    p.left = nullptr;
    p.leaves = left_a;
    p.c = nullptr;
    p.out = static_cast<uint16_t*>(A.p);
    p.pitch = l.spitch;
    p.alpha = 0.0;
    p.beta = SA / (S * S);
    if (l.gram.parts > 1) {
      float* room = reinterpret_cast<float*>(ws + l.room);
      e = tall ? gram<true>(p, X, l.gram, room, &mapped, s) : gram<false>(p, X, l.gram, room, &mapped, s);
    } else {
      e = tall ? product<true, true, false, true, 0>(p, X, X, &mapped, s) : product<false, false, false, true, 0>(p, X, X, &mapped, s);
    }
    if (e == cudaSuccess) {
      p.K = side;
      p.left = left_a;
      p.leaves = left_b;
      p.c = static_cast<const uint16_t*>(A.p);
      p.out = static_cast<uint16_t*>(B.p);
      p.alpha = cb * SB / SA;
      p.beta = cc * SB / (SA * SA);
      e = product<false, false, true, true, 0>(p, A, A, &mapped, s);
    }
    if (e == cudaSuccess) {
      p.call.withhold = last ? a->withhold_copy : 0;
      p.M = m;
      p.N = n;
      p.left = left_b;
      p.leaves = nullptr;
      p.c = static_cast<const uint16_t*>(X.p);
      p.out = last ? static_cast<uint16_t*>(a->out) : reinterpret_cast<uint16_t*>(ws + l.x[(i + 1) & 1]);
      p.pitch = l.pitch;
      p.alpha = last ? ca / S : ca;
      p.beta = last ? 1.0 / (SB * S) : 1.0 / SB;
      p.whole = n % 8 == 0 && aligned(a->out, 16);
      const int kind = !last ? 0 : a->out_dtype == MHC_DTYPE_BF16 ? 1 : 2;
      if (tall)
        e = kind == 0   ? product<false, false, true, false, 0>(p, X, B, &mapped, s)
            : kind == 1 ? product<false, false, true, false, 1>(p, X, B, &mapped, s)
                        : product<false, false, true, false, 2>(p, X, B, &mapped, s);
      else
        e = kind == 0   ? product<false, true, true, false, 0>(p, B, X, &mapped, s)
            : kind == 1 ? product<false, true, true, false, 1>(p, B, X, &mapped, s)
                        : product<false, true, true, false, 2>(p, B, X, &mapped, s);
    }
    if (!mapped) return fail(MHC_ERR_RUNTIME, "encoding a tensor map failed");
    if (e != cudaSuccess) return fail(MHC_ERR_RUNTIME, "orthogonalisation launch failed: %s", cudaGetErrorString(e));
  }
  return MHC_OK;
}

mhc_status_t mhc_orth_status(const void* workspace, void* stream) { return mhc_ffn_status(workspace, stream); }

}  // extern "C"
