// mhc_ffn_gemm.cuh -- the matrix product of the feed-forward block on the
// tensor cores, with a fused epilogue.
//
// Persistent CTAs take output tiles of 128 x 256.  One warp streams operand
// chunks of 64 along the depth into a ring of shared-memory stages (TMA, 128-
// byte swizzle), one thread issues tcgen05.mma on them into one of two tensor-
// memory accumulators, and two groups of four warps read the accumulators back
// alternately and run the epilogue, so that a tile's epilogue overlaps the next
// tile's products.
#pragma once

#include "mhc_ffn.cuh"

namespace mhc {

constexpr int kGemmThreads = 320;          // producer, MMA issuer, 2 x 4 epilogue warps
constexpr int kGemmStages = 4;
constexpr int kGemmABytes = kFfnTileM * kFfnTileK * 2, kGemmBBytes = kFfnTileN * kFfnTileK * 2;
constexpr int kGemmStageBytes = kGemmABytes + kGemmBBytes;

struct GemmTail {
  uint64_t full[kGemmStages], empty[kGemmStages];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t mma_done;
  uint32_t tmem_base;
  uint32_t abort;
};
constexpr size_t kGemmSmem = (size_t)kGemmStages * kGemmStageBytes + sizeof(GemmTail) + 1024;

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

// Tile t of the persistent loop: bands of kBand tile rows, column by column
// inside a band, so that the CTAs running at one time share operand rows in L2.
constexpr int kBand = 16;
__device__ __forceinline__ void tile_coords(const GemmShape& g, int t, int& tm, int& tn) {
  const int band = t / (kBand * g.tiles_n), first = band * kBand;
  const int rows = min(kBand, g.tiles_m - first);
  const int r = t - band * kBand * g.tiles_n;
  tm = first + r % rows;
  tn = r / rows;
}

// ------------------------------------------------------------- epilogues

// The sigmoid form of both activations: act(z) = z s(r(z)), s(r) = 1 / (1 + e^-r),
// r = z for silu and 2 sqrt(2/pi) (z + 0.044715 z^3) for gelu's tanh form.
// Fast exponential and division: their relative error of a few 2^-22 is far
// below the 16-bit rounding that follows.
__device__ __forceinline__ float act_arg(float z, int act) {
  return act == 0 ? z : 1.5957691216f * z * fmaf(0.044715f, z * z, 1.0f);
}
__device__ __forceinline__ float sigmoid_fast(float r) { return __fdividef(1.0f, 1.0f + __expf(-r)); }

template <bool F16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const typename XType<F16>::T2 v = XType<F16>::from_f2(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <bool F16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  return XType<F16>::to_f2(*reinterpret_cast<const typename XType<F16>::T2*>(&w));
}
template <bool F16>
__device__ __forceinline__ uint4 pack8v(const float* f) {
  return make_uint4(pack2<F16>(f[0], f[1]), pack2<F16>(f[2], f[3]), pack2<F16>(f[4], f[5]), pack2<F16>(f[6], f[7]));
}

// out[row, col] = round(acc)
template <bool F16>
struct EpiStore {
  uint16_t* out;
  int M, N;
  __device__ __forceinline__ void tile(uint32_t taddr, int row, int tn) const {
    const int n0 = tn * kFfnTileN;
    uint16_t* o = out + (size_t)row * N + n0;
#pragma unroll 1
    for (int c = 0; c < kFfnTileN && n0 + c < N; c += 32) {
      float v[32];
      tmem_ld32(taddr + c, v);
      if (row < M) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (n0 + c + 8 * q < N) *reinterpret_cast<uint4*>(o + c + 8 * q) = pack8v<F16>(v + 8 * q);
      }
      __syncwarp();                              // whole again before the next accumulator load
    }
  }
};

// Accumulator columns 0..127 gate, 128..255 up of the same 128 columns of F:
// a = act(g) u, and g, u kept in 16 bits (kKept 1) or 8 bits (2).
template <bool F16, int kKept>
struct EpiGateUp {
  uint16_t *a, *gate_up;
  uint8_t *codes, *scales;
  int T, F, act;
  __device__ __forceinline__ void tile(uint32_t taddr, int row, int tn) const {
    const int f0 = tn * 128;
    const bool in = row < T;
    float inv[2] = {1.0f, 1.0f};
    if constexpr (kKept == 2) {
      const int nblk = (F + kCkptBlock - 1) / kCkptBlock;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float amax = 0.0f;                       // columns beyond F hold zeros (or NaN)
#pragma unroll 1
        for (int c = 0; c < 128; c += 32) {
          float v[32];
          tmem_ld32(taddr + h * 128 + c, v);
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const float m = fabsf(v[e]);
            amax = m < __int_as_float(0x7F800000) ? fmaxf(amax, m) : amax;
          }
        }
        const int ex = ckpt_exponent<F16>(amax);
        inv[h] = pow2_f32(-ex);
        if (in) scales[((size_t)row * 2 + h) * nblk + tn] = (uint8_t)(ex + 127);
      }
    }
#pragma unroll 1
    for (int c = 0; c < 128 && f0 + c < F; c += 16) {
      float g[16], u[16], p[16];
      tmem_ld16(taddr + c, g);
      tmem_ld16(taddr + 128 + c, u);
      if (in) {
#pragma unroll
        for (int e = 0; e < 16; ++e) p[e] = g[e] * sigmoid_fast(act_arg(g[e], act)) * u[e];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int f = f0 + c + 8 * q;
          if (f >= F) break;
          *reinterpret_cast<uint4*>(a + (size_t)row * F + f) = pack8v<F16>(p + 8 * q);
          if constexpr (kKept == 1) {
            *reinterpret_cast<uint4*>(gate_up + ((size_t)row * 2) * F + f) = pack8v<F16>(g + 8 * q);
            *reinterpret_cast<uint4*>(gate_up + ((size_t)row * 2 + 1) * F + f) = pack8v<F16>(u + 8 * q);
          }
          if constexpr (kKept == 2) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float w[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float v = h ? u[8 * q + e] : g[8 * q + e];
                w[e] = fabsf(v) < __int_as_float(0x7F800000) ? v * inv[h] : __int_as_float(0x7FFFFFFF);
              }
              *reinterpret_cast<uint2*>(codes + ((size_t)row * 2 + h) * F + f) =
                  make_uint2(e4m3x4(w[0], w[1], w[2], w[3]), e4m3x4(w[4], w[5], w[6], w[7]));
            }
          }
        }
      }
      __syncwarp();
    }
  }
};

// acc = ga: with the kept g and u, gg = ga u act'(g), gu = ga act(g) and
// a = act(g) u.  act' = s + z s (1 - s) r'(z).
template <bool F16, int kKept>
struct EpiDgate {
  const uint16_t* gate_up;
  const uint8_t *codes, *scales;
  uint16_t *gg, *a;
  int T, F, act;
  __device__ __forceinline__ void tile(uint32_t taddr, int row, int tn) const {
    const int f0 = tn * kFfnTileN;
    const bool in = row < T;
    const int nblk = (F + kCkptBlock - 1) / kCkptBlock;
#pragma unroll 1
    for (int c = 0; c < kFfnTileN && f0 + c < F; c += 16) {
      float v[16];
      tmem_ld16(taddr + c, v);
      if (in) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int f = f0 + c + 8 * q;
          if (f >= F) break;
          float k[2][8], o[3][8];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const size_t r = (size_t)row * 2 + h;
            if constexpr (kKept == 1) {
              const uint4 w = *reinterpret_cast<const uint4*>(gate_up + r * F + f);
              const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float2 p = unpack2<F16>(ww[e]);
                k[h][2 * e] = p.x;
                k[h][2 * e + 1] = p.y;
              }
            } else {
              const uint2 w = *reinterpret_cast<const uint2*>(codes + r * F + f);
              const float s = ckpt_scale(scales[r * nblk + (f >> 7)]);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float2 p = e4m3x2_f2((e < 2 ? w.x : w.y) >> (16 * (e & 1)));
                k[h][2 * e] = p.x * s;
                k[h][2 * e + 1] = p.y * s;
              }
            }
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float z = k[0][e], u = k[1][e], ga = v[8 * q + e];
            const float s = sigmoid_fast(act_arg(z, act));
            const float dr = act == 0 ? 1.0f : 1.5957691216f * fmaf(3.0f * 0.044715f, z * z, 1.0f);
            const float h = z * s;
            const float dh = fmaf(h * (1.0f - s), dr, s);
            o[0][e] = ga * u * dh;
            o[1][e] = ga * h;
            o[2][e] = h * u;
          }
          *reinterpret_cast<uint4*>(gg + ((size_t)row * 2) * F + f) = pack8v<F16>(o[0]);
          *reinterpret_cast<uint4*>(gg + ((size_t)row * 2 + 1) * F + f) = pack8v<F16>(o[1]);
          *reinterpret_cast<uint4*>(a + (size_t)row * F + f) = pack8v<F16>(o[2]);
        }
      }
      __syncwarp();
    }
  }
};

// ------------------------------------------------------------------ kernel

// kPair: B's 256 rows are 128 rows of plane 0 and the same 128 of plane 1
// (gate and up); else 256 consecutive rows.
template <class Epi, bool kAMN, bool kBMN, bool kPair>
__global__ void __launch_bounds__(kGemmThreads, 1)
    ffn_gemm_kernel(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tb, const GemmShape g,
                    const Epi epi) {
  constexpr uint32_t kTmemCols = 512;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  GemmTail* tail = reinterpret_cast<GemmTail*>(smem + kGemmStages * kGemmStageBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ntiles = g.tiles_m * g.tiles_n;
  Ctl ctl{&tail->abort, g.err, g.wait_ns};

  if (threadIdx.x == 0) {
    // Cleared here rather than by a launch of its own: a wait of this call
    // sets it wait_ns after its CTA began at the earliest.
    if (g.clear_err && blockIdx.x == 0) *g.err = 0u;
    for (int s = 0; s < kGemmStages; ++s) {
      mbar_init(&tail->full[s], 1);
      mbar_init(&tail->empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tail->acc_full[b], 1);
      mbar_init(&tail->acc_empty[b], 4);
    }
    mbar_init(&tail->mma_done, 1);
    tail->abort = 0u;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    tma_prefetch_desc(&ta);
    tma_prefetch_desc(&tb);
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

  if (warp == 0) {
    // ===================================================== TMA producer
    if (lane == 0) {
      int s = 0;
      uint32_t ph = 0;
      long long iss = 0;
      bool ok = true;
      for (int t = blockIdx.x; t < ntiles && ok; t += gridDim.x) {
        int tm, tn;
        tile_coords(g, t, tm, tn);
        const int m0 = tm * kFfnTileM, n0 = tn * (kPair ? 128 : kFfnTileN);
        for (int k = 0; k < g.kiters; ++k) {
          if (!wait_bar_sleep(&tail->empty[s], ph ^ 1u, ctl, kErrWaitTimeout)) { ok = false; break; }
          // test hook: CTA 0 leaves out its last chunk, so the waits on it
          // give up (no copy is left in flight)
          if (g.withhold && blockIdx.x == 0 && k == g.kiters - 1 && t + (int)gridDim.x >= ntiles) { ok = false; break; }
          uint8_t* sa = smem + s * kGemmStageBytes;
          uint8_t* sb = sa + kGemmABytes;
          const int k0 = k * kFfnTileK;
          mbar_expect_tx(&tail->full[s], kGemmStageBytes);
          if constexpr (kAMN) {
#pragma unroll
            for (int i = 0; i < kFfnTileM / 64; ++i)
              tma_load_3d(sa + i * 8192, &ta, &tail->full[s], m0 + 64 * i, k0, 0);
          } else {
            tma_load_3d(sa, &ta, &tail->full[s], k0, m0, 0);
          }
          if constexpr (kBMN) {
#pragma unroll
            for (int i = 0; i < kFfnTileN / 64; ++i)
              tma_load_3d(sb + i * 8192, &tb, &tail->full[s], n0 + 64 * i, k0, 0);
          } else {
#pragma unroll
            for (int i = 0; i < 2; ++i)
              tma_load_3d(sb + i * 16384, &tb, &tail->full[s], k0, kPair ? n0 : n0 + 128 * i, kPair ? i : 0);
          }
          ++iss;
          if (++s == kGemmStages) { s = 0; ph ^= 1u; }
        }
      }
      for (long long q = 0; q < (iss < kGemmStages ? iss : kGemmStages); ++q) {   // let issued copies land
        if (--s < 0) { s = kGemmStages - 1; ph ^= 1u; }
        mbar_drain(&tail->full[s], ph);
      }
    }
  } else if (warp == 1) {
    // ===================================================== MMA issuer
    if (lane == 0) {
      int s = 0, n = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int t = blockIdx.x; t < ntiles && ok; t += gridDim.x, ++n) {
        const int b = n & 1;
        if (!wait_bar_sleep(&tail->acc_empty[b], ((uint32_t)(n >> 1) & 1u) ^ 1u, ctl, kErrWaitTimeout)) break;
        tc_fence_after();
        const uint32_t d = tmem_base + (uint32_t)(b * kFfnTileN);
        for (int k = 0; k < g.kiters; ++k) {
          if (!wait_bar_sleep(&tail->full[s], ph, ctl, kErrWaitTimeout)) { ok = false; break; }
          tc_fence_after();
          const uint32_t sa = smem_u32(smem + s * kGemmStageBytes), sb = sa + kGemmABytes;
#pragma unroll
          for (int ks = 0; ks < kFfnTileK / 16; ++ks) {
            const uint64_t da = kAMN ? sw128_desc_mn(sa + ks * 2048, 8192) : sw128_desc(sa + ks * 32);
            const uint64_t db = kBMN ? sw128_desc_mn(sb + ks * 2048, 8192) : sw128_desc(sb + ks * 32);
            mma_bf16(d, da, db, g.idesc, (k | ks) ? 1u : 0u);
          }
          mma_commit(&tail->empty[s]);
          if (++s == kGemmStages) { s = 0; ph ^= 1u; }
        }
        if (ok) mma_commit(&tail->acc_full[b]);
      }
      mma_commit(&tail->mma_done);
      mbar_drain(&tail->mma_done, 0);
    }
  } else {
    // ===================================================== epilogue
    const int grp = (warp - 2) >> 2, q = warp & 3;
    int n = 0;
    for (int t = blockIdx.x; t < ntiles; t += gridDim.x, ++n) {
      if ((n & 1) != grp) continue;
      int tm, tn;
      tile_coords(g, t, tm, tn);
      if (!wait_bar_sleep(&tail->acc_full[grp], (uint32_t)(n >> 1) & 1u, ctl, kErrWaitTimeout)) break;
      tc_fence_after();
      epi.tile(tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(grp * kFfnTileN), tm * kFfnTileM + q * 32 + lane, tn);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tail->acc_empty[grp]);
    }
  }

  // ---- teardown
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(kTmemCols) : "memory");
  }
}

template <bool kAMN, bool kBMN, bool kPair, class Epi>
cudaError_t launch_gemm(const CUtensorMap& ta, const CUtensorMap& tb, const GemmShape& g, const Epi& epi, int sms,
                        cudaStream_t s) {
  auto* k = ffn_gemm_kernel<Epi, kAMN, kBMN, kPair>;
  const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kGemmSmem);
  if (e != cudaSuccess) return e;
  const long long tiles = (long long)g.tiles_m * g.tiles_n;
  k<<<(unsigned)(tiles < sms ? tiles : sms), kGemmThreads, kGemmSmem, s>>>(ta, tb, g, epi);
  return cudaGetLastError();
}

}  // namespace mhc
