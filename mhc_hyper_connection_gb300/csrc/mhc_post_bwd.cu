// mhc_post_bwd.cu -- the backward of the mHC post-mapping on sm_103a
// (include/mhc_post_backward.h): per token, with g the gradient of out,
//     grad_x = sum_j post[j] g[j]          grad_residual[i] = sum_j comb[i][j] g[j]
//     grad_post[j] = <g[j], x>             grad_comb[i][j]  = <residual[i], g[j]>
//
// One pass over g, x and the residual streams: a lane holds eight columns of
// all of them, forms the n + 1 output vectors at once and adds its products to
// n + n^2 running fp32 dot products, which are joined over the lanes once per
// token.  Bounded by HBM: (2n + 1) 2 bytes read (n + 1/128 n fewer from a
// checkpoint) and (n + 1) 2 written per column, against 2 (n + n^2) products.
#include "mhc_ckpt.cuh"
#include "mhc_host.cuh"
#include "../../include/mhc_post_backward.h"

namespace mhc {
namespace {

constexpr int kPbThreads = 256;
constexpr int kPbWarps = kPbThreads / 32;

struct PostBwdParams {
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

// Sums v[0 .. N) over the warp's lanes; lane l gets the sum of v[l].  Halving
// exchange: at each of five steps a lane sends the half of its values that
// the partner keeps, N + 11 shuffles for N = 20 instead of 5 N.
template <int N>
__device__ __forceinline__ float warp_sums(const float* v, int lane) {
  float a[32];
#pragma unroll
  for (int k = 0; k < 32; ++k) a[k] = k < N ? v[k] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const bool up = (lane & o) != 0;
#pragma unroll
    for (int k = 0; k < o; ++k) {
      if (k < N) {
        const float send = up ? a[k] : a[k + o], keep = up ? a[k + o] : a[k];
        a[k] = keep + __shfl_xor_sync(0xFFFFFFFFu, send, o);
      }
    }
  }
  return a[0];
}

template <int NS, bool kCkpt>
__global__ void __launch_bounds__(kPbThreads) post_bwd_kernel(const PostBwdParams p) {
  constexpr int V = NS + NS * NS;
  __shared__ float part[kPbWarps][V];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int wpt = p.wpt, sub = warp & (wpt - 1);
  const long long t = (long long)blockIdx.x * (kPbWarps / wpt) + warp / wpt;
  const bool live = t < p.T;
  const int D = p.D, nv = D >> 3;
  if (live) {
    const uint64_t once = policy_evict_first();
    float pc[NS], cm[NS * NS], acc[V];
#pragma unroll
    for (int j = 0; j < NS; ++j) pc[j] = __ldg(p.post + t * NS + j);
#pragma unroll
    for (int e = 0; e < NS * NS; ++e) cm[e] = __ldg(p.comb + t * (NS * NS) + e);
#pragma unroll
    for (int k = 0; k < V; ++k) acc[k] = 0.0f;
    const __nv_bfloat16* xt = p.x + t * D;
    const __nv_bfloat16* gt = p.g + t * NS * D;
    const int nblk = (D + kCkptBlock - 1) / kCkptBlock;
    for (int v = sub * 32 + lane; v < nv; v += wpt * 32) {
      const size_t col = (size_t)v * 8;
      uint4 graw[NS], rraw[kCkpt ? 1 : NS];
      uint2 craw[kCkpt ? NS : 1];
      uint32_t sb[kCkpt ? NS : 1];
      const uint4 xraw = ld_global_v4_hint(xt + col, once);
#pragma unroll
      for (int j = 0; j < NS; ++j) graw[j] = ld_global_v4_hint(gt + (size_t)j * D + col, once);
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        const size_t row = (size_t)t * NS + i;
        if constexpr (kCkpt) {
          craw[i] = __ldcs(reinterpret_cast<const uint2*>(p.codes + row * D + col));
          sb[i] = __ldg(p.scales + row * nblk + (v >> 4));
        } else {
          rraw[i] = ld_global_v4_hint(p.res + row * D + col, once);
        }
      }
      float gf[NS][8], f[8], o[8];
#pragma unroll
      for (int j = 0; j < NS; ++j) unpack8(graw[j], gf[j]);
      unpack8(xraw, f);
#pragma unroll
      for (int j = 0; j < NS; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[j] = fmaf(f[e], gf[j][e], acc[j]);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        o[e] = pc[0] * gf[0][e];
#pragma unroll
        for (int j = 1; j < NS; ++j) o[e] = fmaf(pc[j], gf[j][e], o[e]);
      }
      st_global_v4_hint(p.gx + t * D + col, pack8(o), once);
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        if constexpr (kCkpt) {
          const float s = ckpt_scale(sb[i]);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 q = e4m3x2_f2((e < 2 ? craw[i].x : craw[i].y) >> (16 * (e & 1)));
            f[2 * e] = q.x * s;
            f[2 * e + 1] = q.y * s;
          }
        } else {
          unpack8(rraw[i], f);
        }
#pragma unroll
        for (int j = 0; j < NS; ++j)
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[NS + i * NS + j] = fmaf(f[e], gf[j][e], acc[NS + i * NS + j]);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          o[e] = cm[i * NS] * gf[0][e];
#pragma unroll
          for (int j = 1; j < NS; ++j) o[e] = fmaf(cm[i * NS + j], gf[j][e], o[e]);
        }
        st_global_v4_hint(p.gres + ((size_t)t * NS + i) * D + col, pack8(o), once);
      }
    }
    // join the lanes: value k of the token ends in lane k & 31
#pragma unroll
    for (int c = 0; c < V; c += 32) {
      constexpr int kLast = V % 32 == 0 ? 32 : V % 32;
      float s;
      if (c + 32 <= V) s = warp_sums<32>(acc + c, lane);
      else s = warp_sums<kLast>(acc + c, lane);
      const int k = c + lane;
      if (k < V) {
        if (wpt == 1) {
          if (k < NS) p.gpost[t * NS + k] = s;
          else p.gcomb[t * (NS * NS) + k - NS] = s;
        } else {
          part[warp][k] = s;
        }
      }
    }
  }
  if (wpt > 1) {                        // join the token's warps, in warp order
    __syncthreads();
    if (live && sub == 0) {
      for (int k = lane; k < V; k += 32) {
        float s = 0.0f;
        for (int w = 0; w < wpt; ++w) s += part[warp + w][k];
        if (k < NS) p.gpost[t * NS + k] = s;
        else p.gcomb[t * (NS * NS) + k - NS] = s;
      }
    }
  }
}

template <int NS>
cudaError_t launch_ns(const PostBwdParams& p, unsigned grid, cudaStream_t s) {
  if (p.codes) post_bwd_kernel<NS, true><<<grid, kPbThreads, 0, s>>>(p);
  else post_bwd_kernel<NS, false><<<grid, kPbThreads, 0, s>>>(p);
  return cudaGetLastError();
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
  p.scales = static_cast<const uint8_t*>(a->scales);
  p.post = a->post;
  p.comb = a->comb;
  p.gx = static_cast<__nv_bfloat16*>(a->grad_x);
  p.gres = static_cast<__nv_bfloat16*>(a->grad_residual);
  p.gpost = a->grad_post;
  p.gcomb = a->grad_comb;
  // Few tokens: several warps share one, while each still has a vector per
  // lane, until there are 16 warps per SM.
  p.wpt = 1;
  while (p.wpt < kPbWarps && T * p.wpt < (int64_t)di.sms * 16 && p.wpt * 256 < D) p.wpt *= 2;
  const int64_t per = kPbWarps / p.wpt;
  const unsigned grid = (unsigned)((T + per - 1) / per);
  using Fn = cudaError_t (*)(const PostBwdParams&, unsigned, cudaStream_t);
  static const Fn table[8] = {launch_ns<1>, launch_ns<2>, launch_ns<3>, launch_ns<4>,
                              launch_ns<5>, launch_ns<6>, launch_ns<7>, launch_ns<8>};
  const cudaError_t e = table[n - 1](p, grid, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(MHC_ERR_RUNTIME, "post-mapping backward launch failed: %s", cudaGetErrorString(e));
  return MHC_OK;
}
