// mhc_ckpt.cuh -- the 8-bit form of 16-bit activations (include/mhc_ckpt.h):
// block exponent, e4m3 codes and the way back, for the kernels that write or
// read it.
#pragma once

#include "mhc_ptx.cuh"

namespace mhc {

constexpr int kCkptBlock = 128;

// Exponents inside which every value code 2^e is exact in the 16-bit type:
// the smallest step is 2^(e - 9), the largest value 448 2^e.
template <bool F16>
struct CkptRange {
  static constexpr int lo = F16 ? -15 : -100;
  static constexpr int hi = F16 ? 7 : 119;
};

// Smallest e with amax <= 448 2^e, clamped.  amax finite and >= 0: with
// amax = m 2^k, m in [1, 2), it is k - 8 for m <= 1.75 and k - 7 above;
// adding 2^23 (2 - 1.75) - 1 to the bits carries into the exponent exactly
// when m > 1.75.
template <bool F16>
__device__ __forceinline__ int ckpt_exponent(float amax) {
  const int e = (int)((__float_as_uint(amax) + 0x1FFFFFu) >> 23) - 135;
  return min(max(e, CkptRange<F16>::lo), CkptRange<F16>::hi);
}
__device__ __forceinline__ float pow2_f32(int e) { return __int_as_float((e + 127) << 23); }   // e in [-126, 127]

// Two fp32 values to two e4m3 codes (low byte: a), ties to even, capped at
// 448; NaN gives 0x7F.
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  return e4m3x2(a, b) | (e4m3x2(c, d) << 16);
}
// Two codes to fp32 (exact through fp16).
__device__ __forceinline__ float2 e4m3x2_f2(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
  return __half22float2(*reinterpret_cast<__half2*>(&h));
}

// Largest magnitude of eight 16-bit elements as raw bits of the two lanes of
// a packed word; NaN loses against a number, two NaN give NaN.
template <bool F16>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  if constexpr (F16) {
    const __half2 r = __hmax2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
  } else {
    const __nv_bfloat162 r = __hmax2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
}
template <bool F16>
__device__ __forceinline__ uint32_t absmax8(uint4 v) {
  constexpr uint32_t m = 0x7FFF7FFFu;
  return max2<F16>(max2<F16>(v.x & m, v.y & m), max2<F16>(v.z & m, v.w & m));
}
// The packed word's two lanes joined, as fp32.
template <bool F16>
__device__ __forceinline__ float max_lanes(uint32_t w) {
  using X = XType<F16>;
  const float2 f = X::to_f2(*reinterpret_cast<typename X::T2*>(&w));
  return fmaxf(f.x, f.y);
}

// Eight elements to eight codes with 1 / scale = inv.
template <bool F16>
__device__ __forceinline__ uint2 ckpt_encode8(uint4 v, float inv) {
  using X = XType<F16>;
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  float f[8];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 p = X::to_f2(*reinterpret_cast<const typename X::T2*>(&w[e]));
    f[2 * e] = p.x * inv;
    f[2 * e + 1] = p.y * inv;
  }
  return make_uint2(e4m3x4(f[0], f[1], f[2], f[3]), e4m3x4(f[4], f[5], f[6], f[7]));
}

// The same with infinities turned into NaN codes, and its absmax8 over the
// finite elements: the rare path of a block that holds an infinity or
// nothing but NaN.
template <bool F16>
__device__ __forceinline__ uint4 ckpt_mark_nonfinite(uint4 v, bool to_zero) {
  constexpr uint32_t top = F16 ? 0x7C00u : 0x7F80u;
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if ((w[e] & top) == top) w[e] = (w[e] & 0xFFFF0000u) | (to_zero ? 0u : 0x7FFFu);
    if (((w[e] >> 16) & top) == top) w[e] = (w[e] & 0x0000FFFFu) | (to_zero ? 0u : 0x7FFF0000u);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// One block held by the 16 lanes of `mask` (eight elements each, zeros beyond
// the row): its exponent in every lane and this lane's codes.
template <bool F16>
__device__ __forceinline__ int ckpt_block16(uint4 v, uint32_t mask, uint2& codes) {
  uint32_t w = absmax8<F16>(v);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) w = max2<F16>(w, __shfl_xor_sync(mask, w, o));
  float amax = max_lanes<F16>(w);
  if (!(amax < __int_as_float(0x7F800000))) {
    w = absmax8<F16>(ckpt_mark_nonfinite<F16>(v, true));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) w = max2<F16>(w, __shfl_xor_sync(mask, w, o));
    amax = max_lanes<F16>(w);
    v = ckpt_mark_nonfinite<F16>(v, false);
  }
  const int e = ckpt_exponent<F16>(amax);
  codes = ckpt_encode8<F16>(v, pow2_f32(-e));
  return e;
}

// Two rows' blocks held by the 16 lanes of `mask`: the maxima travel as one
// packed pair.  Exponents and this lane's codes.
template <bool F16>
__device__ __forceinline__ void ckpt_block16x2(uint4 v0, uint4 v1, uint32_t mask, int (&e)[2], uint2 (&codes)[2]) {
  const uint32_t a = absmax8<F16>(v0), b = absmax8<F16>(v1);
  uint32_t w = max2<F16>(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));     // (max of v0, max of v1)
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) w = max2<F16>(w, __shfl_xor_sync(mask, w, o));
  using X = XType<F16>;
  const float2 f = X::to_f2(*reinterpret_cast<typename X::T2*>(&w));
  const float inf = __int_as_float(0x7F800000);
  if (!(f.x < inf) || !(f.y < inf)) {
    e[0] = ckpt_block16<F16>(v0, mask, codes[0]);
    e[1] = ckpt_block16<F16>(v1, mask, codes[1]);
    return;
  }
  e[0] = ckpt_exponent<F16>(f.x);
  e[1] = ckpt_exponent<F16>(f.y);
  codes[0] = ckpt_encode8<F16>(v0, pow2_f32(-e[0]));
  codes[1] = ckpt_encode8<F16>(v1, pow2_f32(-e[1]));
}

// Asynchronous copies of 16 or 8 bytes to shared memory, zeros where `in` is
// false; each thread waits for its own groups and reads only what it copied.
__device__ __forceinline__ void copy16(void* dst, const void* src, bool in, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(smem_u32(dst)),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(in ? 16 : 0), "l"(policy)
               : "memory");
}
__device__ __forceinline__ void copy8(void* dst, const void* src, bool in, uint64_t policy) {
  asm volatile("cp.async.ca.shared.global.L2::cache_hint [%0], [%1], 8, %2, %3;" ::"r"(smem_u32(dst)),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(in ? 8 : 0), "l"(policy)
               : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Value of a scale byte: 2^(byte - 127).
__device__ __forceinline__ float ckpt_scale(uint32_t byte) { return __uint_as_float(byte << 23); }

}  // namespace mhc
