// mhc_ckpt.cu -- 8-bit activation checkpoints on sm_103a: pack, restore, and
// the post-mapping that packs its own output (include/mhc_ckpt.h).
//
// All three are streaming kernels bounded by HBM: pack reads 2 and writes 1 +
// 1/128 bytes an element, restore the reverse, the post-mapping adds 1 + 1/128
// bytes an output element to what it moves anyway.  A block of 128 columns is
// 16 lanes of eight elements, so its maximum takes four shuffles on packed
// 16-bit pairs and each lane turns its own 16 bytes into 8.
#include <atomic>

#include "mhc_ckpt.cuh"
#include "mhc_host.cuh"
#include "../../include/mhc_ckpt.h"

namespace mhc {
namespace {

constexpr int kCkptThreads = 256;
constexpr int kUnroll = 4;     // consecutive blocks of one half-warp, all loads in flight

// kFlat: D is a multiple of 128, so block b starts at element 128 b.
template <bool F16, bool kFlat>
__global__ void __launch_bounds__(kCkptThreads)
    ckpt_pack_kernel(long long total, int nblk, int D, const uint16_t* __restrict__ x, uint8_t* __restrict__ codes,
                     uint8_t* __restrict__ scales) {
  const int l = threadIdx.x & 15;
  const uint32_t mask = 0xFFFFu << (threadIdx.x & 16);
  const long long b0 = (((long long)blockIdx.x * kCkptThreads + threadIdx.x) >> 4) * kUnroll;
  if (b0 >= total) return;                         // whole half-warps leave
  const uint64_t once = policy_evict_first();
  long long off[kUnroll];
  bool in[kUnroll];
  uint4 v[kUnroll];
  {
    long long row = 0;
    int cb = 0;
    if (!kFlat) {
      row = total <= 0xFFFFFFFFll ? (long long)((uint32_t)b0 / (uint32_t)nblk) : b0 / nblk;
      cb = (int)(b0 - row * nblk);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (kFlat) {
        off[u] = (b0 + u) * kCkptBlock + l * 8;
        in[u] = b0 + u < total;
      } else {
        const int col = cb * kCkptBlock + l * 8;
        off[u] = row * D + col;
        in[u] = b0 + u < total && col < D;
        if (++cb == nblk) { cb = 0; ++row; }
      }
      v[u] = in[u] ? ld_global_v4_hint(x + off[u], once) : make_uint4(0, 0, 0, 0);
    }
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    uint2 c;
    const int e = ckpt_block16<F16>(v[u], mask, c);
    if (in[u]) __stcs(reinterpret_cast<uint2*>(codes + off[u]), c);
    if (l == 0 && b0 + u < total) scales[b0 + u] = (uint8_t)(e + 127);
  }
}

template <bool F16, bool kFlat>
__global__ void __launch_bounds__(kCkptThreads)
    ckpt_restore_kernel(long long vecs, int vrow, int nblk, const uint8_t* __restrict__ codes,
                        const uint8_t* __restrict__ scales, uint16_t* __restrict__ x) {
  using X = XType<F16>;
  const uint64_t once = policy_evict_first();
  const long long v0 = (long long)blockIdx.x * (kCkptThreads * kUnroll) + threadIdx.x;
  uint2 c[kUnroll];
  uint32_t sb[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const long long v = v0 + u * kCkptThreads;
    c[u] = make_uint2(0, 0);
    sb[u] = 127;
    if (v < vecs) {
      long long sidx = v >> 4;
      if (!kFlat) {
        const long long row = vecs <= 0xFFFFFFFFll ? (long long)((uint32_t)v / (uint32_t)vrow) : v / vrow;
        sidx = row * nblk + ((v - row * vrow) >> 4);
      }
      c[u] = __ldcs(reinterpret_cast<const uint2*>(codes) + v);
      sb[u] = __ldg(scales + sidx);
    }
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const long long v = v0 + u * kCkptThreads;
    if (v >= vecs) break;
    const float s = ckpt_scale(sb[u]);
    const uint32_t w[2] = {c[u].x, c[u].y};
    uint32_t o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = e4m3x2_f2(w[e >> 1] >> (16 * (e & 1)));
      const typename X::T2 p = X::from_f2(f.x * s, f.y * s);     // exact
      o[e] = *reinterpret_cast<const uint32_t*>(&p);
    }
    st_global_v4_hint(x + v * 8, make_uint4(o[0], o[1], o[2], o[3]), once);
  }
}

// The post-mapping (out[j] = post[j] x + sum_i comb[i][j] residual[i], fp32 sums
// in that order, RN-even) and the checkpoint of its rounded output: the 16 lanes
// that hold a block of 128 columns join their maxima and encode from registers.
//
// A warp takes an equal run of pieces (one token, 256 kV columns); a lane has kV
// vectors of eight columns of each tensor, copied to its own places in shared
// memory one piece ahead, so that the copies of a piece run under the work on
// the one before (with loads into registers instead, at the 16 warps per SM that
// they leave, T = 4096, n = 4, D = 4096 took 83 us where it takes 61.6 now, 89% of
// measured HBM; n = 8, T = 16384, D = 2048: 250 us, 83%).
//
// Two columns share a packed fp32 instruction (the same rounding as two plain
// ones); the coefficients lie in shared memory, each twice.
template <int NS>
struct PcStage {
  static constexpr int kV = NS <= 4 ? 2 : 1;
  uint4 x[kV][32], r[kV][NS][32];
};
template <int NS>
struct PcWarp {
  PcStage<NS> stages[2];
  float2 coef[(NS + 1) * NS];            // post[j], then comb[i][j], as (c, c)
};

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
// Two bf16 as packed fp32.
__device__ __forceinline__ uint64_t widen2(uint32_t w) {
  return (uint64_t)(w << 16) | ((uint64_t)(w & 0xFFFF0000u) << 32);
}
__device__ __forceinline__ uint32_t narrow2(uint64_t v) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float((uint32_t)v), __uint_as_float((uint32_t)(v >> 32)));
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <int NS>
__global__ void __launch_bounds__(kCkptThreads, 2)
    post_ckpt_kernel(int T, int D, const __nv_bfloat16* __restrict__ x, const __nv_bfloat16* __restrict__ res,
                     const float* __restrict__ post, const float* __restrict__ comb, __nv_bfloat16* __restrict__ out,
                     uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  using Stage = PcStage<NS>;
  constexpr int kV = Stage::kV, kCoef = NS + NS * NS;
  extern __shared__ __align__(16) uint8_t pc_smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long gw = (long long)blockIdx.x * (kCkptThreads / 32) + warp, nw = (long long)gridDim.x * (kCkptThreads / 32);
  const int nv = D >> 3, nblk = (D + kCkptBlock - 1) / kCkptBlock, segs = (nv + 32 * kV - 1) / (32 * kV);
  const long long pieces = (long long)T * segs;
  const long long first = pieces * gw / nw, last = pieces * (gw + 1) / nw;
  if (first >= last) return;
  const uint64_t once = policy_evict_first();
  const uint32_t mask = 0xFFFFu << (lane & 16);
  PcWarp<NS>& mine = reinterpret_cast<PcWarp<NS>*>(pc_smem)[warp];
  auto fetch = [&](long long t, int seg, Stage& st) {
#pragma unroll
    for (int q = 0; q < kV; ++q) {
      const int v = (seg * kV + q) * 32 + lane;
      const bool in = v < nv;
      copy16(&st.x[q][lane], x + (in ? t * D + v * 8 : 0), in, once);
#pragma unroll
      for (int i = 0; i < NS; ++i) copy16(&st.r[q][i][lane], res + (in ? (t * NS + i) * D + v * 8 : 0), in, once);
    }
  };
  long long t = first / segs;
  int seg = (int)(first - t * segs);
  fetch(t, seg, mine.stages[0]);
  copies_commit();
  long long have = -1;                             // token whose coefficients are loaded
  int buf = 0;
  for (long long u = first; u < last; ++u, buf ^= 1) {
    long long tn = t;
    int sn = seg + 1;
    if (sn == segs) { sn = 0; ++tn; }
    if (u + 1 < last) fetch(tn, sn, mine.stages[buf ^ 1]);
    copies_commit();
    if (have != t) {
      have = t;
      __syncwarp();
#pragma unroll
      for (int k = lane; k < kCoef; k += 32) {
        const float c = k < NS ? __ldg(post + t * NS + k) : __ldg(comb + t * (NS * NS) + k - NS);
        mine.coef[k] = make_float2(c, c);
      }
      __syncwarp();
    }
    copies_wait<1>();
    const Stage& st = mine.stages[buf];
#pragma unroll
    for (int q = 0; q < kV; ++q) {
      const int v = (seg * kV + q) * 32 + lane;
      if ((v & ~15) >= nv) continue;               // this half-warp's block lies beyond the row
      const uint64_t* coef = reinterpret_cast<const uint64_t*>(mine.coef);
      uint64_t xf[4], rf[NS][4];
      {
        const uint4 w = st.x[q][lane];
        xf[0] = widen2(w.x);
        xf[1] = widen2(w.y);
        xf[2] = widen2(w.z);
        xf[3] = widen2(w.w);
      }
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        const uint4 w = st.r[q][i][lane];
        rf[i][0] = widen2(w.x);
        rf[i][1] = widen2(w.y);
        rf[i][2] = widen2(w.z);
        rf[i][3] = widen2(w.w);
      }
      auto stream = [&](int j) {
        const uint64_t c0 = coef[j];
        uint64_t acc[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] = mul2(c0, xf[e]);
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          const uint64_t c = coef[NS + i * NS + j];
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[e] = fma2(c, rf[i][e], acc[e]);
        }
        // beyond the row: nothing for the maximum (a NaN coefficient times 0)
        return v < nv ? make_uint4(narrow2(acc[0]), narrow2(acc[1]), narrow2(acc[2]), narrow2(acc[3])) : make_uint4(0, 0, 0, 0);
      };
      auto store = [&](int j, const uint4& o, const uint2& c8, int ex) {
        const size_t row = (size_t)t * NS + j;
        if (v < nv) {
          st_global_v4_hint(out + row * D + (size_t)v * 8, o, once);
          __stcs(reinterpret_cast<uint2*>(codes + row * D + (size_t)v * 8), c8);
        }
        if ((lane & 15) == 0) scales[row * nblk + (v >> 4)] = (uint8_t)(ex + 127);
      };
#pragma unroll
      for (int j = 0; j + 1 < NS; j += 2) {
        const uint4 o0 = stream(j), o1 = stream(j + 1);
        int ex[2];
        uint2 c8[2];
        ckpt_block16x2<false>(o0, o1, mask, ex, c8);
        store(j, o0, c8[0], ex[0]);
        store(j + 1, o1, c8[1], ex[1]);
      }
      if constexpr (NS % 2 == 1) {
        const uint4 o = stream(NS - 1);
        uint2 c8;
        const int ex = ckpt_block16<false>(o, mask, c8);
        store(NS - 1, o, c8, ex);
      }
    }
    t = tn;
    seg = sn;
  }
}

template <int NS>
cudaError_t launch_post_ckpt(int64_t T, int64_t D, const void* x, const void* res, const float* post,
                             const float* comb, void* out, void* codes, void* scales, cudaStream_t s) {
  // CTAs that the device holds at once, looked up once per device
  static std::atomic<int> known[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  int resident = known[dev].load(std::memory_order_relaxed);
  constexpr size_t smem = (kCkptThreads / 32) * sizeof(PcWarp<NS>);
  if (resident == 0) {
    int per_sm = 0;
    if ((e = cudaFuncSetAttribute(post_ckpt_kernel<NS>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) !=
        cudaSuccess)
      return e;
    if ((e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, post_ckpt_kernel<NS>, kCkptThreads, smem)) !=
        cudaSuccess)
      return e;
    resident = (per_sm > 0 ? per_sm : 1) * (device_info(dev).sms > 0 ? device_info(dev).sms : 1);
    known[dev].store(resident, std::memory_order_relaxed);
  }
  // Runs of kRun pieces keep the rows in flight near one another in memory and
  // the last round short (T = 32768, n = 4, D = 7168: 895 us with one run per
  // resident warp, 771 with runs of 8, 758 with 4); where they would leave SMs
  // idle, equal shares of all.
  constexpr int kRun = 4;
  const long long cols = 256 * PcStage<NS>::kV, warps = kCkptThreads / 32;
  const long long pieces = T * ((D + cols - 1) / cols);
  long long grid = (pieces + kRun * warps - 1) / (kRun * warps);
  if (grid < resident) grid = resident;
  if (grid * warps > pieces) grid = (pieces + warps - 1) / warps;
  post_ckpt_kernel<NS><<<(int)grid, kCkptThreads, smem, s>>>(
      (int)T, (int)D, static_cast<const __nv_bfloat16*>(x), static_cast<const __nv_bfloat16*>(res), post, comb,
      static_cast<__nv_bfloat16*>(out), static_cast<uint8_t*>(codes), static_cast<uint8_t*>(scales));
  return cudaGetLastError();
}

// pack: x is read and codes and scales are written, else the reverse.
mhc_status_t check_matrix(int64_t rows, int64_t D, int32_t dtype, const void* x, const void* codes, const void* scales,
                          bool pack) {
  if (dtype != MHC_DTYPE_BF16 && dtype != MHC_DTYPE_FP16)
    return fail(MHC_ERR_PARAM_INVALID, "dtype must be MHC_DTYPE_BF16 or MHC_DTYPE_FP16 (got %d)", (int)dtype);
  if (D < 8 || D > (int64_t(1) << 20) || (D % 8) != 0)
    return fail(MHC_ERR_PARAM_INVALID, "D must be a multiple of 8 in [8, 2^20] (got %lld)", (long long)D);
  if (rows < 0 || rows > (int64_t(1) << 38) / D)
    return fail(MHC_ERR_PARAM_INVALID, "rows must be >= 0 and rows * D at most 2^38 (got %lld)", (long long)rows);
  if (rows == 0) return MHC_OK;
  if (!x || !codes || !scales) return fail(MHC_ERR_NULLPTR, "x, codes and scales are required");
  if (!aligned(x, 16)) return fail(MHC_ERR_PARAM_INVALID, "x must be 16-byte aligned");
  if (!aligned(codes, 8)) return fail(MHC_ERR_PARAM_INVALID, "codes must be 8-byte aligned");
  const size_t values = (size_t)rows * D, blocks = (size_t)rows * ((D + kCkptBlock - 1) / kCkptBlock);
  const Span c = {"codes", codes, values}, s = {"scales", scales, blocks}, v = {"x", x, 2 * values};
  return pack ? check_apart({c, s}, {v}) : check_apart({v}, {c, s});
}

}  // namespace
}  // namespace mhc

using namespace mhc;

extern "C" {

mhc_status_t mhc_ckpt8_pack_run(int64_t rows, int64_t D, int32_t dtype, const void* x, void* codes, void* scales,
                                void* stream) {
  clear_error();
  const mhc_status_t st = check_matrix(rows, D, dtype, x, codes, scales, true);
  if (st != MHC_OK || rows == 0) return st;
  const int nblk = (int)((D + kCkptBlock - 1) / kCkptBlock);
  const long long total = rows * nblk;
  const long long per = (kCkptThreads / 16) * kUnroll;
  const unsigned grid = (unsigned)((total + per - 1) / per);     // rows * D <= 2^38: below 2^31
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const uint16_t* xp = static_cast<const uint16_t*>(x);
  uint8_t *cp = static_cast<uint8_t*>(codes), *sp = static_cast<uint8_t*>(scales);
  const bool flat = D % kCkptBlock == 0, f16 = dtype == MHC_DTYPE_FP16;
  auto* k = f16 ? (flat ? ckpt_pack_kernel<true, true> : ckpt_pack_kernel<true, false>)
                : (flat ? ckpt_pack_kernel<false, true> : ckpt_pack_kernel<false, false>);
  k<<<grid, kCkptThreads, 0, s>>>(total, nblk, (int)D, xp, cp, sp);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(MHC_ERR_RUNTIME, "checkpoint pack launch failed: %s", cudaGetErrorString(e));
  return MHC_OK;
}

mhc_status_t mhc_ckpt8_restore_run(int64_t rows, int64_t D, int32_t dtype, const void* codes, const void* scales,
                                   void* x, void* stream) {
  clear_error();
  const mhc_status_t st = check_matrix(rows, D, dtype, x, codes, scales, false);
  if (st != MHC_OK || rows == 0) return st;
  const int nblk = (int)((D + kCkptBlock - 1) / kCkptBlock), vrow = (int)(D / 8);
  const long long vecs = rows * vrow;
  const long long per = kCkptThreads * kUnroll;
  const unsigned grid = (unsigned)((vecs + per - 1) / per);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const uint8_t *cp = static_cast<const uint8_t*>(codes), *sp = static_cast<const uint8_t*>(scales);
  uint16_t* xp = static_cast<uint16_t*>(x);
  const bool flat = D % kCkptBlock == 0, f16 = dtype == MHC_DTYPE_FP16;
  auto* k = f16 ? (flat ? ckpt_restore_kernel<true, true> : ckpt_restore_kernel<true, false>)
                : (flat ? ckpt_restore_kernel<false, true> : ckpt_restore_kernel<false, false>);
  k<<<grid, kCkptThreads, 0, s>>>(vecs, vrow, nblk, cp, sp, xp);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(MHC_ERR_RUNTIME, "checkpoint restore launch failed: %s", cudaGetErrorString(e));
  return MHC_OK;
}

mhc_status_t mhc_post_ckpt_run(int64_t T, int64_t n, int64_t D, const void* x, const void* residual, const float* post,
                               const float* comb, void* out, void* codes, void* scales, void* stream) {
  clear_error();
  if (T < 0 || T > (int64_t(1) << 30)) return fail(MHC_ERR_PARAM_INVALID, "T must be in [0, 2^30]");
  if (n < 1 || n > 8) return fail(MHC_ERR_PARAM_INVALID, "n must be in [1, 8] (got %lld)", (long long)n);
  if (D < 8 || D > (int64_t(1) << 20) || (D % 8) != 0)
    return fail(MHC_ERR_PARAM_INVALID, "D must be a multiple of 8 in [8, 2^20] (got %lld)", (long long)D);
  if (T == 0) return MHC_OK;
  if (!x || !residual || !post || !comb || !out || !codes || !scales)
    return fail(MHC_ERR_NULLPTR, "x, residual, post, comb, out, codes and scales are required");
  if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(out, 16))
    return fail(MHC_ERR_PARAM_INVALID, "x, residual and out must be 16-byte aligned");
  if (!aligned(codes, 8)) return fail(MHC_ERR_PARAM_INVALID, "codes must be 8-byte aligned");
  if (!aligned(post, 4) || !aligned(comb, 4)) return fail(MHC_ERR_PARAM_INVALID, "post and comb must be 4-byte aligned");
  const size_t xb = (size_t)T * D * 2, pb = (size_t)T * n * 4, values = (size_t)T * n * D;
  const mhc_status_t st =
      check_apart({{"out", out, 2 * values},
                   {"codes", codes, values},
                   {"scales", scales, (size_t)T * n * ((D + kCkptBlock - 1) / kCkptBlock)}},
                  {{"x", x, xb}, {"residual", residual, 2 * values}, {"post", post, pb}, {"comb", comb, pb * n}});
  if (st != MHC_OK) return st;
  using Fn = cudaError_t (*)(int64_t, int64_t, const void*, const void*, const float*, const float*, void*, void*,
                             void*, cudaStream_t);
  static const Fn table[8] = {launch_post_ckpt<1>, launch_post_ckpt<2>, launch_post_ckpt<3>, launch_post_ckpt<4>,
                              launch_post_ckpt<5>, launch_post_ckpt<6>, launch_post_ckpt<7>, launch_post_ckpt<8>};
  const cudaError_t e = table[n - 1](T, D, x, residual, post, comb, out, codes, scales, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(MHC_ERR_RUNTIME, "post-mapping launch failed: %s", cudaGetErrorString(e));
  return MHC_OK;
}

}  // extern "C"
