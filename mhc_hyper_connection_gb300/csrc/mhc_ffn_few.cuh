// mhc_ffn_few.cuh -- the feed-forward block's products for few tokens (serving,
// and the backward of small batches).
//
// With up to 128 tokens the weights are read once and used little: the bound is
// HBM.  So the weights are the 128-row side of the tensor-core product and the
// tokens its N side (a multiple of 16), each CTA streams its own rows of the
// weights through a ring of stages, and where the rows alone do not fill the
// device, a cluster of 2 to 8 CTAs shares them, each taking a part of the
// depth.  Their fp32 sums are exchanged over distributed shared memory: each
// CTA gets all parts of its share of the tokens, adds them in rank order (no
// atomics: the same bits every time) and finishes those tokens.
//
// A product's CTAs start as SMs fall free in the one before it (programmatic
// dependent launch) and load the weights' first chunks before they wait for the
// tokens.
//
// One token, D = 7168, F = 8192: 66 us a call for 352 MB of weights, 79% of the
// measured copy rate; the two products' loops stream at 6.9 and 5.3 TB/s, the
// rest is their starts and joins, about 4 us each.  24 tokens at D = 4096, F =
// 8192: 45.5 us (66%).  As ordinary tiles of 256 tokens these took 114 and 80.
// (Calls back to back on changing inputs; where a comment below compares two
// forms, on the same input the same calls take a microsecond or two less.)
#pragma once

#include <mutex>

#include "mhc_ffn_gemm.cuh"

namespace mhc {

constexpr int kFewThreads = 192;                 // producer, MMA issuer, four epilogue warps
// Ring and room of the gate and up product, one CTA per SM (24 tokens, D = 4096, F
// = 8192: 43.9 us, with 160 KB 45.0), and of the others, of which two fit an SM
// (backward of 24 tokens, D = 1024, F = 4096: 32.2 us, with 76 KB 34.2).
constexpr int kFewRingTwo = 214 * 1024;
constexpr int kFewRingOne = 108 * 1024;
constexpr size_t kFewHalfSm = 112 * 1024;        // shared memory of which two CTAs fit an SM
constexpr int kFewMinStages = 3;
constexpr int kFewMaxStages = 12;
constexpr int kFewRows = 128;                    // weight rows of one accumulator
constexpr int kFewMostSplit = 8;                 // CTAs of a cluster
constexpr int kFewMostSmem = 224 * 1024;         // shared memory of a CTA

struct FewTail {
  uint64_t full[kFewMaxStages], empty[kFewMaxStages];
  uint64_t acc_full;
  uint32_t tmem_base;
  uint32_t abort;
};

struct FewShape {
  int T;                       // tokens
  int nt;                      // tokens rounded up to 16
  int tiles, kiters, split;    // 128-row tiles, depth chunks, CTAs that share a tile
  int stages, ring;            // stages and bytes of the ring
  int own_room;                // the exchanged sums lie behind the ring, not in it
  int a_mn;                    // weights stored MN-major
  uint32_t idesc;
  uint32_t* err;
  uint64_t wait_ns;
  int withhold;
  int first;                   // first product of a call: clears the error word, waits for nothing
};

__host__ __device__ constexpr int few_stage_bytes(bool two, int nt) { return (two ? 2 : 1) * 16384 + nt * 128; }
// Tokens that each of `split` CTAs finishes: an equal share, in fours.
__host__ __device__ constexpr int few_share(int nt, int split) { return ((nt + split - 1) / split + 3) & ~3; }
__host__ __device__ constexpr int few_room_bytes(bool two, int nt, int split) {
  return (two ? 2 : 1) * split * few_share(nt, split) * 512;
}
// From 65 tokens on the sums lie in the ring.
constexpr bool few_rooms_fit() {
  for (int nt = 16; nt <= kFewTokens; nt += 16)
    for (int split = 1; split <= kFewMostSplit; ++split)
      for (int two = 0; two < 2; ++two)
        if ((split == 1 || nt > 64) && few_room_bytes(two, nt, split) > (two ? kFewRingTwo : kFewRingOne)) return false;
  return true;
}
static_assert(few_rooms_fit(), "the ring holds the sums");

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}
// The two halves of a cluster barrier.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// Place of a row's 16 bytes: eight rows four apart lie in eight different
// sixteen-byte columns of the banks, and so do eight rows in sequence.
__device__ __forceinline__ int swz_row(int r) { return r ^ ((r >> 3) & 3); }

// ------------------------------------------------------------- epilogues
// One warp per token; a lane has four consecutive weight rows r of its sums.

template <bool F16>
__device__ __forceinline__ uint2 pack4(float4 v) {
  return make_uint2(pack2<F16>(v.x, v.y), pack2<F16>(v.z, v.w));
}

template <bool F16>
struct FewStore {
  static constexpr bool kTwo = false;
  uint16_t* out;
  int N;
  __device__ __forceinline__ void token(int n, int tile, const float4& v, const float4&, int lane) const {
    const int r = tile * kFewRows + 4 * lane;
    if (r < N) *reinterpret_cast<uint2*>(out + (size_t)n * N + r) = pack4<F16>(v);
  }
};

template <bool F16, int kKept>
struct FewGateUp {
  static constexpr bool kTwo = true;
  uint16_t *a, *gate_up;
  uint8_t *codes, *scales;
  int F, act;
  __device__ __forceinline__ void token(int n, int tile, const float4& g, const float4& u, int lane) const {
    const int f = tile * kFewRows + 4 * lane;
    const bool in = f < F;
    float4 p;
    p.x = g.x * sigmoid_fast(act_arg(g.x, act)) * u.x;
    p.y = g.y * sigmoid_fast(act_arg(g.y, act)) * u.y;
    p.z = g.z * sigmoid_fast(act_arg(g.z, act)) * u.z;
    p.w = g.w * sigmoid_fast(act_arg(g.w, act)) * u.w;
    if (in) *reinterpret_cast<uint2*>(a + (size_t)n * F + f) = pack4<F16>(p);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float4 v = h ? u : g;
      const size_t row = (size_t)n * 2 + h;
      if constexpr (kKept == 1) {
        if (in) *reinterpret_cast<uint2*>(gate_up + row * F + f) = pack4<F16>(v);
      }
      if constexpr (kKept == 2) {
        const float inf = __int_as_float(0x7F800000), nan = __int_as_float(0x7FFFFFFF);
        const float e[4] = {v.x, v.y, v.z, v.w};
        float amax = 0.0f;                       // columns beyond F hold zeros (or NaN)
#pragma unroll
        for (int i = 0; i < 4; ++i) amax = fabsf(e[i]) < inf ? fmaxf(amax, fabsf(e[i])) : amax;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
        const int ex = ckpt_exponent<F16>(amax);
        const float inv = pow2_f32(-ex);
        float w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = fabsf(e[i]) < inf ? e[i] * inv : nan;
        if (in) *reinterpret_cast<uint32_t*>(codes + row * F + f) = e4m3x4(w[0], w[1], w[2], w[3]);
        if (lane == 0) scales[row * ((F + kCkptBlock - 1) / kCkptBlock) + tile] = (uint8_t)(ex + 127);
      }
    }
  }
};

template <bool F16, int kKept>
struct FewDgate {
  static constexpr bool kTwo = false;
  const uint16_t* gate_up;
  const uint8_t *codes, *scales;
  uint16_t *gg, *a;
  int F, act;
  __device__ __forceinline__ void token(int n, int tile, const float4& v, const float4&, int lane) const {
    const int f = tile * kFewRows + 4 * lane;
    if (f >= F) return;
    const float ga[4] = {v.x, v.y, v.z, v.w};
    float k[2][4];
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const size_t row = (size_t)n * 2 + p;
      if constexpr (kKept == 1) {
        const uint2 w = *reinterpret_cast<const uint2*>(gate_up + row * F + f);
        const float2 lo = unpack2<F16>(w.x), hi = unpack2<F16>(w.y);
        k[p][0] = lo.x;
        k[p][1] = lo.y;
        k[p][2] = hi.x;
        k[p][3] = hi.y;
      } else {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(codes + row * F + f);
        const float s = ckpt_scale(scales[row * ((F + kCkptBlock - 1) / kCkptBlock) + tile]);
        const float2 lo = e4m3x2_f2(w), hi = e4m3x2_f2(w >> 16);
        k[p][0] = lo.x * s;
        k[p][1] = lo.y * s;
        k[p][2] = hi.x * s;
        k[p][3] = hi.y * s;
      }
    }
    float og[4], ou[4], oa[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) gate_grads(k[0][e], k[1][e], ga[e], act, og[e], ou[e], oa[e]);
    *reinterpret_cast<uint2*>(gg + ((size_t)n * 2) * F + f) = pack4<F16>(make_float4(og[0], og[1], og[2], og[3]));
    *reinterpret_cast<uint2*>(gg + ((size_t)n * 2 + 1) * F + f) = pack4<F16>(make_float4(ou[0], ou[1], ou[2], ou[3]));
    *reinterpret_cast<uint2*>(a + (size_t)n * F + f) = pack4<F16>(make_float4(oa[0], oa[1], oa[2], oa[3]));
  }
};

// ------------------------------------------------------------------ kernel

template <class Epi>
__global__ void __launch_bounds__(kFewThreads, 1)
    ffn_few_kernel(const __grid_constant__ CUtensorMap tw, const __grid_constant__ CUtensorMap tx, const FewShape g,
                   const Epi epi) {
  constexpr bool kTwo = Epi::kTwo;
  constexpr uint32_t kTmemCols = 256;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  FewTail* tail = reinterpret_cast<FewTail*>(smem + g.ring + (g.own_room ? few_room_bytes(kTwo, g.nt, g.split) : 0));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = g.split > 1 ? (int)cluster_rank() : 0;
  const int tile = blockIdx.x / g.split;
  const int k0 = (int)((long long)g.kiters * rank / g.split), k1 = (int)((long long)g.kiters * (rank + 1) / g.split);
  const int stage_bytes = few_stage_bytes(kTwo, g.nt), stages = g.stages;
  Ctl ctl{&tail->abort, g.err, g.wait_ns};

  if (threadIdx.x == 0) {
    if (g.first && blockIdx.x == 0) g.err[0] = g.err[1] = 0u;   // as in ffn_gemm_kernel
    for (int s = 0; s < stages; ++s) {
      mbar_init(&tail->full[s], 1);
      mbar_init(&tail->empty[s], 1);
    }
    mbar_init(&tail->acc_full, 1);
    tail->abort = 0u;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    tma_prefetch_desc(&tw);
    tma_prefetch_desc(&tx);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tail->tmem_base)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = tail->tmem_base;
  pdl_trigger();
  if (g.split > 1) cluster_arrive();             // waited for before the first remote store

  // The timed waits of these warps begin when the product before is complete: a
  // limit then bounds this product's own waits.
  if (warp != 0) pdl_wait();

  if (warp == 0) {
    // ===================================================== TMA producer
    if (lane == 0) {
      int s = 0, iss = 0;
      uint32_t ph = 0;
      const int r0 = tile * kFewRows;
      // the weights of a chunk into its stage, which then expects the tokens too
      auto weights = [&](int k, int st) {
        uint8_t* sw = smem + st * stage_bytes;
        const int kk = k * kFfnTileK;
        mbar_expect_tx(&tail->full[st], (uint32_t)stage_bytes);
        if (g.a_mn) {
          tma_load_3d(sw, &tw, &tail->full[st], r0, kk, 0);
          tma_load_3d(sw + 8192, &tw, &tail->full[st], r0 + 64, kk, 0);
        } else {
          tma_load_3d(sw, &tw, &tail->full[st], kk, r0, 0);
          if (kTwo) tma_load_3d(sw + 16384, &tw, &tail->full[st], kk, r0, 1);
        }
      };
      auto tokens = [&](int k, int st) {
        tma_load_3d(smem + st * stage_bytes + (kTwo ? 2 : 1) * 16384, &tx, &tail->full[st], k * kFfnTileK, 0, 0);
      };
      // test hook: the first CTA leaves out its last chunk
      const int kend = g.withhold && blockIdx.x == 0 ? k1 - 1 : k1;
      const int early = min(stages, kend - k0);
      if (!g.first) {
        for (int k = 0; k < early; ++k) weights(k0 + k, k);
        pdl_wait();                              // the tokens are the previous product's
      }
      for (int k = k0; k < kend; ++k) {
        if (!wait_stage(&tail->empty[s], ph ^ 1u, ctl)) break;
        if (g.first || k - k0 >= early) weights(k, s);
        tokens(k, s);
        ++iss;
        if (++s == stages) { s = 0; ph ^= 1u; }
      }
      for (int q = 0; q < (iss < stages ? iss : stages); ++q) {   // let issued copies land
        if (--s < 0) { s = stages - 1; ph ^= 1u; }
        mbar_drain(&tail->full[s], ph);
      }
    }
  } else if (warp == 1) {
    // ===================================================== MMA issuer
    if (lane == 0) {
      const uint64_t w0 = g.a_mn ? sw128_desc_mn(0, 8192) : sw128_desc(0), x0 = sw128_desc(0);
      const uint32_t wstep = (g.a_mn ? 2048u : 32u) >> 4;
      int s = 0;
      uint32_t ph = 0;
      for (int k = k0; k < k1; ++k) {
        if (!wait_stage(&tail->full[s], ph, ctl)) break;
        tc_fence_after();
        const uint32_t sw = desc_addr(smem + s * stage_bytes), sx = sw + (((kTwo ? 2 : 1) * 16384) >> 4);
#pragma unroll
        for (int ks = 0; ks < kFfnTileK / 16; ++ks) {
          const uint32_t acc = (k > k0 || ks) ? 1u : 0u;
          mma_bf16(tmem_base, w0 + (sw + ks * wstep), x0 + (sx + ks * 2), g.idesc, acc);
          if (kTwo) mma_bf16(tmem_base + 128, w0 + (sw + 1024 + ks * wstep), x0 + (sx + ks * 2), g.idesc, acc);
        }
        mma_commit(&tail->empty[s]);
        if (++s == stages) { s = 0; ph ^= 1u; }
      }
      mma_commit(&tail->acc_full);
      mbar_drain(&tail->acc_full, 0);
    }
  } else {
    wait_stage(&tail->acc_full, 0, ctl);
  }
  // Everything this CTA issued is done.  Where the sums have no room of their
  // own they go into the rings, which then have to be idle in the whole cluster.
  // An aborted CTA takes part in the barriers all the same.
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (g.split > 1) {
    cluster_wait();                              // of the arrival at the start: every CTA is there
    if (!g.own_room) cluster_sync_all();
  }
  tc_fence_after();

  // Exchange: rank d finishes tokens [d per, (d + 1) per).  Every CTA sends its
  // fp32 sums of them to block `rank` of d's room: [plane][token / 4][row][4
  // tokens], rows swizzled so that both the lanes' writes (a row each) and
  // their reads (four rows each) spread over the banks.
  const int per = few_share(g.nt, g.split), ncols = (kTwo ? 2 : 1) * g.nt;
  const int block = (kTwo ? 2 : 1) * per * 128;            // fp32 values of one CTA's sums
  float* room = reinterpret_cast<float*>(smem + (g.own_room ? g.ring : 0));
  if (warp >= 2) {
    const int q = warp & 3;
    float* mine = room + (size_t)rank * block + swz_row(q * 32 + lane) * 4;
    for (int c = 0; c < ncols; c += 16) {
      float v[16];
      const int plane = c < g.nt ? 0 : 1, n0 = c - plane * g.nt;
      tmem_ld16(tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(plane * 128 + n0), v);
#pragma unroll
      for (int e = 0; e < 16; e += 4) {
        const int n = n0 + e, d = n / per;
        float* at = mine + (size_t)(plane * per + n - d * per) * 128;
        const float4 w = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
        if (g.split == 1) *reinterpret_cast<float4*>(at) = w;
        else st_dsmem_v4(at, (uint32_t)d, w);
      }
    }
  }
  if (g.split > 1) cluster_sync_all();
  else __syncthreads();
  pdl_wait();                                    // outputs may be what earlier launches still read
  for (int n = warp * 4; n < per && rank * per + n < g.T; n += 4 * (kFewThreads / 32)) {
    float m[2][4][4];                            // [plane][row][token]
#pragma unroll
    for (int p = 0; p < (kTwo ? 2 : 1); ++p) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float* at = room + (size_t)(p * per + n) * 128 + swz_row(4 * lane + i) * 4;
        float4 v = *reinterpret_cast<const float4*>(at);
        for (int r = 1; r < g.split; ++r) {
          const float4 w = *reinterpret_cast<const float4*>(at + (size_t)r * block);
          v.x += w.x;
          v.y += w.y;
          v.z += w.z;
          v.w += w.w;
        }
        m[p][i][0] = v.x;
        m[p][i][1] = v.y;
        m[p][i][2] = v.z;
        m[p][i][3] = v.w;
      }
    }
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      if (rank * per + n + t >= g.T) break;
      const float4 v = make_float4(m[0][0][t], m[0][1][t], m[0][2][t], m[0][3][t]);
      const float4 u = kTwo ? make_float4(m[1][0][t], m[1][1][t], m[1][2][t], m[1][3][t]) : v;
      epi.token(rank * per + n + t, tile, v, u, lane);
    }
  }

  // ---- teardown
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(kTmemCols) : "memory");
  }
}

// The few-token shape of a product whose weights have `rows` rows.
inline FewShape few_shape(const GemmShape& g, const FfnCall& call, int rows, int T, bool f16, bool w_mn, bool first,
                          bool last) {
  FewShape w = {};
  w.T = T;
  w.nt = (T + 15) & ~15;
  w.tiles = (rows + kFewRows - 1) / kFewRows;
  w.kiters = g.kiters;
  w.a_mn = w_mn ? 1 : 0;
  w.idesc = f16 ? idesc_f16(kFewRows, w.nt) : idesc_bf16(kFewRows, w.nt);
  if (w_mn) w.idesc |= 1u << 15;
  w.err = call.err;
  w.wait_ns = call.wait_ns;
  w.withhold = last ? call.withhold : 0;
  w.first = first ? 1 : 0;
  return w;
}

// Ring, room and shared memory of a launch with `split` CTAs per tile.
inline size_t few_layout(FewShape& g, bool two, int split) {
  const int stage = few_stage_bytes(two, g.nt), room = few_room_bytes(two, g.nt, split);
  g.split = split;
  g.own_room = split > 1 && g.nt <= 64;
  g.ring = (two ? kFewRingTwo : kFewRingOne) - (g.own_room ? room : 0);
  if (g.ring < kFewMinStages * stage) g.ring = kFewMinStages * stage;
  g.stages = g.ring / stage < kFewMaxStages ? g.ring / stage : kFewMaxStages;
  return (size_t)g.ring + (g.own_room ? room : 0) + sizeof(FewTail) + 1024;
}

// A kernel of the same launch shape that uses no tensor memory: the runtime
// counts one CTA per SM for those that do, whatever they allocate.
static __global__ void __launch_bounds__(kFewThreads) few_shape_kernel() {}

// Clusters of each size that the device holds at once, with the shared memory of
// two CTAs per SM (first row) or of one; looked up once per device.
struct FewClusters {
  int n[2][kFewMostSplit + 1];
};
inline cudaError_t few_clusters(int dev, FewClusters* out) {
  static std::mutex mu;
  static FewClusters known[64];
  static bool have[64];
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lk(mu);
  if (!have[dev]) {
    cudaError_t e = cudaFuncSetAttribute(few_shape_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kFewMostSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.blockDim = dim3(kFewThreads);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    for (int c = 0; c < 2; ++c) {
      for (int i = 2; i <= kFewMostSplit; ++i) {
        attr[0].val.clusterDim.x = (unsigned)i;
        cfg.gridDim = dim3(1024u * i);
        cfg.dynamicSmemBytes = c == 0 ? kFewHalfSm : kFewMostSmem;
        if ((e = cudaOccupancyMaxActiveClusters(&known[dev].n[c][i], few_shape_kernel, &cfg)) != cudaSuccess) return e;
      }
    }
    have[dev] = true;
  }
  *out = known[dev];
  return cudaSuccess;
}

// CTAs per tile: the most whose clusters the device holds all at once, with
// four chunks of the depth each at least (D = 1024, F = 4096, one token: 14.4 us,
// with eight chunks 15.1, one CTA per tile 29.6).  Clusters that start as SMs fall
// free pack less tightly than on an empty device, so a sixteenth stays free (one
// token, D = 7168, F = 8192, second product: 56 clusters of 5, of at most 58, 72
// us, of 4 65.4).  Against sizes of 2, 4 and 8 alone: one token, D = 4424, F =
// 5192: 38.5 -> 34.5 us; 64 tokens, D = 7168, F = 2048: 32.8 -> 30.5.
template <class Epi>
cudaError_t launch_few(const CUtensorMap& tw, const CUtensorMap& tx, FewShape g, const Epi& epi, cudaStream_t s) {
  auto* k = ffn_few_kernel<Epi>;
  static std::atomic<bool> ready[64];                      // per device: the shared-memory limit is set
  int dev = 0;
  FewClusters fit;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (e = few_clusters(dev, &fit)) != cudaSuccess) return e;
  if (!ready[dev].load(std::memory_order_relaxed)) {
    if ((e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kFewMostSmem)) != cudaSuccess) return e;
    ready[dev].store(true, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.blockDim = dim3(kFewThreads);
  cfg.stream = s;
  cfg.attrs = attr;
  size_t smem = few_layout(g, Epi::kTwo, 1);
  for (int split = kFewMostSplit; split > 1; --split) {
    FewShape w = g;
    const size_t bytes = few_layout(w, Epi::kTwo, split);
    const int most = fit.n[bytes > kFewHalfSm ? 1 : 0][split];
    if (bytes > (size_t)kFewMostSmem || g.kiters < 4 * split || g.tiles > most - (g.first ? 0 : most / 16)) continue;
    g = w;
    smem = bytes;
    break;
  }
  attr[0].val.clusterDim.x = (unsigned)g.split;
  cfg.gridDim = dim3((unsigned)(g.tiles * g.split));
  cfg.dynamicSmemBytes = smem;
  cfg.numAttrs = g.first ? 1 : 2;
  return cudaLaunchKernelEx(&cfg, k, tw, tx, (const FewShape)g, epi);
}

}  // namespace mhc
