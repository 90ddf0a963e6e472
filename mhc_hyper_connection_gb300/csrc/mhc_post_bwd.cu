// mhc_post_bwd.cu -- the backward of the mHC post-mapping on sm_103a
// (include/mhc_post_backward.h): per token, with g the gradient of out,
//     grad_x = sum_j post[j] g[j]          grad_residual[i] = sum_j comb[i][j] g[j]
//     grad_post[j] = <g[j], x>             grad_comb[i][j]  = <residual[i], g[j]>
//
// One pass over g, x and the residual streams.  Bounded by HBM: (2n + 1) 2
// bytes read (n - n/128 fewer from a checkpoint) and (n + 1) 2 written per
// column, against 2 (n + n^2) products.  Those run on the tensor cores: on the
// CUDA cores they took longer than the memory (n = 8, T = 16384, D = 2048 from a
// checkpoint: 430 us, 51% of measured HBM; now 240 us, 91%; n = 4, T = 32768, D =
// 7168: 1092 us, now 1040, 93%).
#include <atomic>

#include "mhc_ckpt.cuh"
#include "mhc_host.cuh"
#include "../../include/mhc_post_backward.h"

namespace mhc {
namespace {

constexpr int kPbThreads = 256;
constexpr int kPbWarps = kPbThreads / 32;

struct PostBwdParams {
  int codes16;                         // rows of codes are 16-byte aligned
  int T, D, wpt;                       // wpt: warps that share a token (a power of two up to kPbWarps)
  const __nv_bfloat16 *g, *x, *res;
  const uint8_t *codes, *scales;
  const float *post, *comb;
  __nv_bfloat16 *gx, *gres;
  float *gpost, *gcomb;
};

__device__ __forceinline__ void unpack8(uint4 v, float (&f)[8]) {
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&v);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 p = __bfloat1622float2(h[e]);
    f[2 * e] = p.x;
    f[2 * e + 1] = p.y;
  }
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  uint4 o;
  __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&o);
#pragma unroll
  for (int e = 0; e < 4; ++e) h[e] = __floats2bfloat162_rn(f[2 * e], f[2 * e + 1]);
  return o;
}

// Rows of a warp's 8 x 32 pieces: the streams of one token (n >= 5), of two at
// four rows each (n = 3, 4), of four at two (n = 2) or of eight (n = 1).  Lane 4 r + q holds row r, eight columns from 8 q, of g
// and of the residual; that is at once both operands' register layout of a
// 16 x 8 x 16 tensor-core product over the columns (their order inside a sum
// does not matter), whose result is the dot products of all row pairs: no
// joining over lanes.  The residual rows are the upper eight rows of A, the
// tokens' x the lower ones.
//
// The outputs are products over the rows: [comb; post] (16 x 8) times g (8 x
// columns).  movmatrix turns a register of g into the B operand, and the result
// comes out in the layout that g came in: eight consecutive columns a lane.
// comb and post enter as three bf16 terms (24 bits, as fp32 has), so a product
// is as exact as in fp32.  Such a split turns an infinity in g into NaN, and the
// tokens of a warp share the product over rows, so a piece with a result that
// is not finite is formed again in plain fp32 (direct_piece).
//
// A code is scaled before it enters a product (1.1 us of 240 at n = 8, T = 16384,
// D = 2048, 1.4 of 70 at n = 4, T = D = 4096): codes run up to 448, and their products with gradients above 2^113 would
// overflow in sums whose scaled values do not.
//
// Sums: the tensor core adds at most 64 columns, then fp32 registers (a long
// chain inside it would round toward zero at every step).
__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_1688(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t b0) {
  asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5}, {%6}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(b0));
}
__device__ __forceinline__ uint32_t movmatrix(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// Two bf16 values times two powers of two.
__device__ __forceinline__ uint32_t scaled2(uint32_t v, uint32_t s) {
  const __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&v), *reinterpret_cast<const __nv_bfloat162*>(&s));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// c = t[0] + t[1] + t[2] in bf16 terms
__device__ __forceinline__ void split3(float c, float (&t)[3]) {
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    t[i] = __bfloat162float(__float2bfloat16_rn(c));
    c = fabsf(t[i]) < __int_as_float(0x7F800000) ? c - t[i] : 0.0f;
  }
}

// Row r, columns 8 q .. of [comb; post] g in fp32: g's rows come from the lanes
// that hold them.  `coef` points at the first of this row's n coefficients,
// `src` is the first row of its token.
template <int NS>
__device__ __noinline__ uint4 direct_piece(uint4 g, const float* coef, int src, int lane) {
  float o[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) o[e] = 0.0f;
  for (int j = 0; j < NS; ++j) {
    const int from = (src + j) * 4 + (lane & 3);
    uint4 w;
    w.x = __shfl_sync(0xFFFFFFFFu, g.x, from);
    w.y = __shfl_sync(0xFFFFFFFFu, g.y, from);
    w.z = __shfl_sync(0xFFFFFFFFu, g.z, from);
    w.w = __shfl_sync(0xFFFFFFFFu, g.w, from);
    float f[8];
    unpack8(w, f);
    const float c = coef ? __ldg(coef + j) : 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = j == 0 ? c * f[e] : fmaf(c, f[e], o[e]);
  }
  return pack8(o);
}

// A warp's 128 columns in shared memory: each lane's own pieces of g, of the
// residual and, in the lanes with an x row, of x; codes as rows of 128 bytes, 160
// apart (free of bank conflicts), copied 16 bytes at a time where their rows are
// so aligned (n = 8, T = 16384, D = 2048: 10 us less than 8 at a time).  The next
// 128 columns are copied while these are worked on.
template <int NS, bool kCkpt>
struct PbStage {
  static constexpr int kTok = NS == 1 ? 8 : NS == 2 ? 4 : NS <= 4 ? 2 : 1;   // tokens of a warp
  uint4 g[4][32];
  uint4 x[4][4 * kTok];
  uint4 r[kCkpt ? 80 : 128];
};

template <int NS, bool kCkpt>
__global__ void __launch_bounds__(kPbThreads, 2) post_bwd_kernel(const PostBwdParams p) {
  using Stage = PbStage<NS, kCkpt>;
  constexpr int kTok = Stage::kTok, kStride = 8 / kTok;              // rows between the tokens
  extern __shared__ __align__(16) uint8_t pb_smem[];
  __shared__ float part[kPbWarps][16 * 8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = lane >> 2, q = lane & 3;
  const int wpt = p.wpt, sub = warp & (wpt - 1);
  const long long t0 = ((long long)blockIdx.x * (kPbWarps / wpt) + warp / wpt) * kTok;
  const int D = p.D, nblk = (D + kCkptBlock - 1) / kCkptBlock;
  const int tau = r / kStride, s = r % kStride;
  const bool row_ok = s < NS && t0 + tau < p.T, x_ok = r < kTok && t0 + r < p.T;
  const size_t row = (size_t)(t0 + tau) * NS + s;                    // of g, the residual and its gradient
  float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};                           // rows r and 8 + r, columns 2 q, 2 q + 1

  if (t0 < p.T) {                                                    // uniform over the warp
    const uint64_t once = policy_evict_first();
    // A operand of the outputs: row r comb, row 8 + r post, over g's rows 2 q, 2 q + 1
    uint32_t ac[3], ap[3];
    {
      float tc[2][3], tp[2][3];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int k = 2 * q + e, tk = k / kStride, j = k % kStride;
        const bool ok = j < NS && t0 + tk < p.T;
        split3(ok && row_ok && tk == tau ? __ldg(p.comb + row * NS + j) : 0.0f, tc[e]);
        split3(ok && x_ok && tk == r ? __ldg(p.post + (size_t)(t0 + tk) * NS + j) : 0.0f, tp[e]);
      }
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        ac[i] = bf16x2(tc[0][i], tc[1][i]);
        ap[i] = bf16x2(tp[0][i], tp[1][i]);
      }
    }
    const __nv_bfloat16* gp = p.g + row * D + q * 8;
    const __nv_bfloat16* xp = p.x + (size_t)(t0 + r) * D + q * 8;
    __nv_bfloat16* gres = p.gres + row * D + q * 8;
    __nv_bfloat16* gx = p.gx + (size_t)(t0 + r) * D + q * 8;
    Stage* stages = reinterpret_cast<Stage*>(pb_smem) + 2 * warp;
    auto fetch = [&](int blk, Stage& st) {
      const int c0 = blk * 128, left = D - c0 - q * 8;               // this lane's columns from c0: u * 32 < left
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const bool in = u * 32 < left && row_ok;
        copy16(&st.g[u][lane], in ? gp + c0 + u * 32 : p.g, in, once);
        if constexpr (kCkpt) {
          uint8_t* cr = reinterpret_cast<uint8_t*>(st.r) + r * 160;
          if (!p.codes16) {
            copy8(cr + u * 32 + q * 8, in ? p.codes + row * D + q * 8 + c0 + u * 32 : p.codes, in, once);
          } else if (u < 2) {
            const int b = u * 64 + q * 16;
            const bool cin = row_ok && c0 + b < D;
            copy16(cr + b, cin ? p.codes + row * D + c0 + b : p.codes, cin, once);
          }
        } else copy16(&st.r[u * 32 + lane], in ? p.res + row * D + q * 8 + c0 + u * 32 : p.res, in, once);
        if (r < kTok) {
          const bool xin = u * 32 < left && x_ok;
          copy16(&st.x[u][lane], xin ? xp + c0 + u * 32 : p.x, xin, once);
        }
      }
    };
    if (sub < nblk) fetch(sub, stages[0]);
    copies_commit();
    int buf = 0;
    for (int blk = sub; blk < nblk; blk += wpt, buf ^= 1) {          // blocks of 128 columns
      const int c0 = blk * 128, left = D - c0 - q * 8;
      const Stage& st = stages[buf];
      if (kCkpt) __syncwarp();                                       // codes are read by other lanes than copied them
      if (blk + wpt < nblk) fetch(blk + wpt, stages[buf ^ 1]);
      copies_commit();
      copies_wait<1>();
      if (kCkpt) __syncwarp();
      uint32_t scale = 0x3F803F80u;                                  // the block's 2^e in bf16, twice
      if (kCkpt && row_ok) scale = (uint32_t)__ldg(p.scales + row * nblk + blk) * 0x00800080u;
      float dot[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const uint4 gv = st.g[u][lane];
        const uint4 xv = r < kTok ? st.x[u][lane] : make_uint4(0, 0, 0, 0);
        const uint32_t gw[4] = {gv.x, gv.y, gv.z, gv.w}, xw[4] = {xv.x, xv.y, xv.z, xv.w};
        uint32_t rw[4];
        if constexpr (kCkpt) {
          const uint2 cv = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint8_t*>(st.r) + r * 160 + u * 32 + q * 8);
#pragma unroll
          for (int e = 0; e < 4; ++e) {                              // a code's value, scaled or not, is exact in bf16
            const float2 f = e4m3x2_f2((e < 2 ? cv.x : cv.y) >> (16 * (e & 1)));
            rw[e] = scaled2(bf16x2(f.x, f.y), scale);
          }
        } else {
          const uint4 rv = st.r[u * 32 + lane];
          rw[0] = rv.x;
          rw[1] = rv.y;
          rw[2] = rv.z;
          rw[3] = rv.w;
        }
        if ((u & 1) == 0) dot[0] = dot[1] = dot[2] = dot[3] = 0.0f;
        mma_16816(dot, rw[0], xw[0], rw[1], xw[1], gw[0], gw[1]);
        mma_16816(dot, rw[2], xw[2], rw[3], xw[3], gw[2], gw[3]);
        if (u & 1) {
          acc[0] += dot[0];
          acc[1] += dot[1];
          acc[2] += dot[2];
          acc[3] += dot[3];
        }
        uint32_t o[4], ox[4];
        float size = 0.0f;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const uint32_t b = movmatrix(gw[t]);
          float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
          mma_1688(c, ac[2], ap[2], b);                              // smallest terms first
          mma_16816(c, ac[0], ap[0], ac[1], ap[1], b, b);
          o[t] = bf16x2(c[0], c[1]);
          ox[t] = bf16x2(c[2], c[3]);
          size += fabsf(c[0]) + fabsf(c[1]);
          size += fabsf(c[2]) + fabsf(c[3]);
        }
        uint4 ov = make_uint4(o[0], o[1], o[2], o[3]), oxv = make_uint4(ox[0], ox[1], ox[2], ox[3]);
        if (__any_sync(0xFFFFFFFFu, !(size < __int_as_float(0x7F800000)))) {
          ov = direct_piece<NS>(gv, row_ok ? p.comb + row * NS : nullptr, tau * kStride, lane);
          oxv = direct_piece<NS>(gv, x_ok ? p.post + (size_t)(t0 + r) * NS : nullptr, x_ok ? r * kStride : 0, lane);
        }
        const bool in = u * 32 < left;
        if (in && row_ok) st_global_v4_hint(gres + c0 + u * 32, ov, once);
        if (in && x_ok) st_global_v4_hint(gx + c0 + u * 32, oxv, once);
      }
    }
  }
  if (wpt > 1) {                        // join the token's warps, in warp order
    float* mine = part[warp];
    mine[r * 8 + 2 * q] = acc[0];
    mine[r * 8 + 2 * q + 1] = acc[1];
    mine[(8 + r) * 8 + 2 * q] = acc[2];
    mine[(8 + r) * 8 + 2 * q + 1] = acc[3];
    __syncthreads();
    if (sub != 0) return;
    for (int w = 1; w < wpt; ++w) {
      const float* o = part[warp + w];
      acc[0] += o[r * 8 + 2 * q];
      acc[1] += o[r * 8 + 2 * q + 1];
      acc[2] += o[(8 + r) * 8 + 2 * q];
      acc[3] += o[(8 + r) * 8 + 2 * q + 1];
    }
  }
  if (t0 >= p.T) return;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int k = 2 * q + e, tk = k / kStride, j = k % kStride;
    if (j < NS && row_ok && tk == tau) p.gcomb[row * NS + j] = acc[e];
    if (j < NS && x_ok && tk == r) p.gpost[(size_t)(t0 + r) * NS + j] = acc[2 + e];
  }
}

template <int NS, bool kCkpt>
cudaError_t launch_kept(const PostBwdParams& p, unsigned grid, cudaStream_t s) {
  constexpr size_t smem = 2 * kPbWarps * sizeof(PbStage<NS, kCkpt>);
  static std::atomic<bool> ready[64];                      // per device: the shared-memory limit is set
  auto* k = post_bwd_kernel<NS, kCkpt>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!ready[dev].load(std::memory_order_relaxed)) {
    if ((e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) != cudaSuccess) return e;
    ready[dev].store(true, std::memory_order_relaxed);
  }
  k<<<grid, kPbThreads, smem, s>>>(p);
  return cudaGetLastError();
}

template <int NS>
cudaError_t launch_ns(const PostBwdParams& p, unsigned grid, cudaStream_t s) {
  return p.codes ? launch_kept<NS, true>(p, grid, s) : launch_kept<NS, false>(p, grid, s);
}

}  // namespace
}  // namespace mhc

using namespace mhc;

extern "C" mhc_status_t mhc_post_backward_run(const mhc_post_bwd_args* a, void* stream) {
  clear_error();
  if (!a) return fail(MHC_ERR_NULLPTR, "args must be non-NULL");
  const int64_t T = a->T, n = a->n, D = a->D;
  if (T < 0 || T > (int64_t(1) << 30)) return fail(MHC_ERR_PARAM_INVALID, "T must be in [0, 2^30]");
  if (n < 1 || n > 8) return fail(MHC_ERR_PARAM_INVALID, "n must be in [1, 8] (got %lld)", (long long)n);
  if (D < 8 || D > (int64_t(1) << 20) || (D % 8) != 0)
    return fail(MHC_ERR_PARAM_INVALID, "D must be a multiple of 8 in [8, 2^20] (got %lld)", (long long)D);
  if (T == 0) return MHC_OK;
  if (!a->grad_out || !a->x || !a->post || !a->comb || !a->grad_x || !a->grad_residual || !a->grad_post || !a->grad_comb)
    return fail(MHC_ERR_NULLPTR, "grad_out, x, post, comb and the four gradients are required");
  if ((a->codes == nullptr) != (a->scales == nullptr))
    return fail(MHC_ERR_PARAM_INVALID, "codes and scales go together (both or neither)");
  if (!a->residual && !a->codes) return fail(MHC_ERR_NULLPTR, "residual or its checkpoint is required");
  if (a->residual && a->codes) return fail(MHC_ERR_PARAM_INVALID, "give residual or its checkpoint, not both");
  const void* v16[] = {a->grad_out, a->x, a->residual, a->grad_x, a->grad_residual};
  for (const void* q : v16)
    if (q && !aligned(q, 16)) return fail(MHC_ERR_PARAM_INVALID, "bf16 tensors must be 16-byte aligned");
  if (!aligned(a->codes, 8)) return fail(MHC_ERR_PARAM_INVALID, "codes must be 8-byte aligned");
  const void* v4[] = {a->post, a->comb, a->grad_post, a->grad_comb};
  for (const void* q : v4)
    if (!aligned(q, 4)) return fail(MHC_ERR_PARAM_INVALID, "fp32 tensors must be 4-byte aligned");
  const size_t xb = (size_t)T * D * 2, pb = (size_t)T * n * 4, values = (size_t)T * n * D;
  const mhc_status_t st = check_apart({{"grad_x", a->grad_x, xb},
                                       {"grad_residual", a->grad_residual, 2 * values},
                                       {"grad_post", a->grad_post, pb},
                                       {"grad_comb", a->grad_comb, pb * n}},
                                      {{"grad_out", a->grad_out, 2 * values},
                                       {"x", a->x, xb},
                                       {"residual", a->residual, 2 * values},
                                       {"codes", a->codes, values},
                                       {"scales", a->scales, (size_t)T * n * ((D + kCkptBlock - 1) / kCkptBlock)},
                                       {"post", a->post, pb},
                                       {"comb", a->comb, pb * n}});
  if (st != MHC_OK) return st;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return fail(MHC_ERR_RUNTIME, "no CUDA device");
  const DeviceInfo di = device_info(dev);
  if (!di.ok) return fail(MHC_ERR_RUNTIME, "device %d is not an sm_103 GPU", dev);
  PostBwdParams p;
  p.T = (int)T;
  p.D = (int)D;
  p.g = static_cast<const __nv_bfloat16*>(a->grad_out);
  p.x = static_cast<const __nv_bfloat16*>(a->x);
  p.res = static_cast<const __nv_bfloat16*>(a->residual);
  p.codes = static_cast<const uint8_t*>(a->codes);
  p.codes16 = D % 16 == 0 && aligned(a->codes, 16);
  p.scales = static_cast<const uint8_t*>(a->scales);
  p.post = a->post;
  p.comb = a->comb;
  p.gx = static_cast<__nv_bfloat16*>(a->grad_x);
  p.gres = static_cast<__nv_bfloat16*>(a->grad_residual);
  p.gpost = a->grad_post;
  p.gcomb = a->grad_comb;
  // Few tokens: several warps share those of one, while each still has 256
  // columns, until there are 64 warps per SM (T = 4096, n = 4, D = 4096: 84.9 us
  // with 16, 80.7 with 64: the last round of CTAs is shorter).
  const int64_t tok = n == 1 ? 8 : n == 2 ? 4 : n <= 4 ? 2 : 1, units = (T + tok - 1) / tok;
  p.wpt = 1;
  while (p.wpt < kPbWarps && units * p.wpt < (int64_t)di.sms * 64 && p.wpt * 256 < D) p.wpt *= 2;
  const int64_t per = kPbWarps / p.wpt;
  const unsigned grid = (unsigned)((units + per - 1) / per);
  using Fn = cudaError_t (*)(const PostBwdParams&, unsigned, cudaStream_t);
  static const Fn table[8] = {launch_ns<1>, launch_ns<2>, launch_ns<3>, launch_ns<4>,
                              launch_ns<5>, launch_ns<6>, launch_ns<7>, launch_ns<8>};
  const cudaError_t e = table[n - 1](p, grid, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(MHC_ERR_RUNTIME, "post-mapping backward launch failed: %s", cudaGetErrorString(e));
  return MHC_OK;
}
