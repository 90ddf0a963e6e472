// mhc_ffn_gemm.cuh -- the matrix product of the feed-forward block on the
// tensor cores, with a fused epilogue.
//
// Persistent pairs of CTAs (clusters of two, one tcgen05 cta_group::2) take
// output tiles of 256 x 256 (or 192 or 128 wide, where that saves a round of tiles,
// with fewer rows of B).  Each CTA holds 128 rows of A and 128 of B, so a
// stage of depth 64 is 32 KB per SM where a tile of its own (128 x 256) would
// be 48: a third less L2 traffic and six stages instead of four.  In each CTA
// one warp streams its operand rows into the ring (TMA, 128-byte swizzle, all
// completing on the even CTA's barriers); one thread of the even CTA issues the
// products for both into one of two tensor-memory accumulators; and in each CTA
// two groups of four warps read its 128 rows back, half the columns each, and run
// the epilogue, which overlaps the next tile's products.
//
// A launch may hold several products (the backward's last).  Where their tiles
// differ in depth the pairs draw tile numbers from a counter in the workspace: the
// even CTA's producer draws them ahead and hands them to the other warps of both
// CTAs through a small ring (T = 1021, D = 2048, F = 5512: backward 134 us, with
// tiles dealt out in turn 23 more).  Which pair forms a tile does not change its bits.
//
// T = 4096, D = 4096, F = 8192, bf16: forward 455 to 495 us (1.81 to 1.67 PFLOP/s;
// 508 to 520 with gate and up kept), backward 1085 to 1105 us (1.5 PFLOP/s), at the
// card's power limit, which differs from one to the next.  Bound
// by the tensor cores: four products of a stage execute in 512 clocks and take 535
// with K-major operands, 650 to 710 with MN-major ones, whose reads leave the
// shared memory less room (with the products of a stage issued twice they take
// their 512 there too).
#pragma once

#include <atomic>

#include "mhc_ffn.cuh"

namespace mhc {

constexpr int kGemmThreads = 320;          // producer, MMA issuer, 2 x 4 epilogue warps
constexpr int kGemmStages = 6;
constexpr int kGemmHalf = 128;             // rows of A and of B that one CTA of the pair holds
constexpr int kGemmOpBytes = kGemmHalf * kFfnTileK * 2;
constexpr int kGemmStageBytes = 2 * kGemmOpBytes;

constexpr int kSchedSlots = 4;

struct GemmTail {
  uint64_t full[kGemmStages], empty[kGemmStages];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t sched_full[kSchedSlots], sched_empty[kSchedSlots];
  uint64_t mma_done;
  uint64_t sent[2];                        // even CTA: 1 + the stages that each CTA of the pair issued, once it issues no more
  uint32_t tmem_base;
  uint32_t abort;
  int sched[kSchedSlots];                  // tile numbers, -1: no more
};

// The products of one launch, in the order of their tiles.
struct GemmOperands {
  CUtensorMap a, b;
  GemmShape g;
};
template <int P>
struct GemmSet {
  GemmOperands op[P];
};
constexpr size_t kGemmSmem = (size_t)kGemmStages * kGemmStageBytes + 8 * 4096 + sizeof(GemmTail) + 1024;

// Programmatic dependent launch: let the next launch of the stream begin; wait
// until the launches before this one are complete and their writes visible.
__device__ __forceinline__ void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// The address, in the cluster's shared window, of this CTA's object `p` in
// CTA `rank`.
__device__ __forceinline__ uint32_t map_cluster(const void* p, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}
// Tiled load into this CTA's shared memory, completing on a barrier of either
// CTA of the pair (`bar`: its address in the cluster's window).
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1,
                                                 int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}
// D[256, N] += A B^T over a depth of 16, A and B halved over the pair.
__device__ __forceinline__ void mma_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Start-address field of an operand descriptor.  A shared-memory address holds
// the CTA's rank in its upper bits, which would run into the fields above.
__device__ __forceinline__ uint32_t desc_addr(const void* p) { return (smem_u32(p) & 0x3FFFFu) >> 4; }
// One lane of a whole warp.  The issuing warp stays together and elects a lane
// only for the instructions themselves: in a branch of one lane's own, four
// products and their bookkeeping took 640 clocks, 25% more than they execute
// for; so they take 535 (forward at T = 4096, D = 4096, F = 8192: 498 -> 456 us).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
  return p != 0;
}
// Arrive on the barrier at this offset in both CTAs once the products issued
// so far are done.
__device__ __forceinline__ void commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}

// 32 consecutive fp32 columns of this warp's 32 accumulator lanes: one load, one
// wait (a wait costs a few hundred clocks of an epilogue's few thousand).
__device__ __forceinline__ void acc_ld32(uint32_t taddr, float (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]),
        "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]),
        "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(taddr)
      : "memory");
}
// 16 columns of two ranges.
__device__ __forceinline__ void acc_ld16x2(uint32_t ta, uint32_t tb, float (&a)[16], float (&b)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%32];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,"
      "%26,%27,%28,%29,%30,%31}, [%33];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(a[0]), "=f"(a[1]), "=f"(a[2]), "=f"(a[3]), "=f"(a[4]), "=f"(a[5]), "=f"(a[6]), "=f"(a[7]), "=f"(a[8]),
        "=f"(a[9]), "=f"(a[10]), "=f"(a[11]), "=f"(a[12]), "=f"(a[13]), "=f"(a[14]), "=f"(a[15]),
        "=f"(b[0]), "=f"(b[1]), "=f"(b[2]), "=f"(b[3]), "=f"(b[4]), "=f"(b[5]), "=f"(b[6]), "=f"(b[7]), "=f"(b[8]),
        "=f"(b[9]), "=f"(b[10]), "=f"(b[11]), "=f"(b[12]), "=f"(b[13]), "=f"(b[14]), "=f"(b[15])
      : "r"(ta), "r"(tb)
      : "memory");
}

// Bytes of a stage that one CTA of the pair copies; an MN-major B comes in blocks
// of 64 rows.
__device__ __forceinline__ uint32_t stage_bytes_of(const GemmShape& g) {
  const int half_n = g.tile_n / 2;
  return (uint32_t)(kGemmOpBytes + (g.b_mn ? (half_n + 63) & ~63 : half_n) * kFfnTileK * 2);
}

// Completes `bytes` of a barrier's phase without a copy.
__device__ __forceinline__ void mbar_complete_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.complete_tx.relaxed.cluster.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}

// After a wait gave up, in the even CTA: every copy that the pair issued lands
// before it leaves.  Once neither CTA issues any more (each of their waits is
// bounded too), both CTAs' copies are counted on the even CTA's barriers.  These
// expect both halves of a stage; where only one CTA issued its half, the barrier
// is made to count that half alone.  The ring bounds the difference at its stages.
static __device__ __noinline__ void settle_copies(GemmTail* tail, uint64_t wait_ns, uint32_t bytes) {
  uint64_t sent[2];
  const uint64_t t0 = now_ns();
  do {
#pragma unroll
    for (int r = 0; r < 2; ++r)
      asm volatile("ld.acquire.cluster.shared::cta.b64 %0, [%1];" : "=l"(sent[r]) : "r"(smem_u32(&tail->sent[r])) : "memory");
    if (now_ns() - t0 > 2 * wait_ns + 100000000ull) return;
  } while (!sent[0] || !sent[1]);
  const long long mine = (long long)sent[0] - 1, theirs = (long long)sent[1] - 1;
  const long long both = mine < theirs ? mine : theirs, most = mine < theirs ? theirs : mine;
  for (long long k = both; k < most; ++k) {
    if (mine < theirs) mbar_expect_tx(&tail->full[k % kGemmStages], bytes);
    else mbar_complete_tx(&tail->full[k % kGemmStages], bytes);
  }
  for (long long k = most > kGemmStages ? most - kGemmStages : 0; k < most; ++k)
    mbar_drain(&tail->full[k % kGemmStages], (uint32_t)(k / kGemmStages) & 1u);
}

// Bounded wait of the product loops.  The clock is read only after a few
// probes have failed (each may sleep in the barrier for a while): reading it at
// the head of every wait costs more than a stage of products.
static __device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, const Ctl& c, uint32_t code, bool cluster) {
  uint64_t t0 = 0;
  for (uint32_t it = 1;; ++it) {
    if (cluster ? mbar_test_cluster(bar, parity) : mbar_test(bar, parity)) return true;
    if ((it & 15u) == 0) {
      if (*c.abort) return false;
      const uint64_t now = now_ns();
      if (t0 == 0) t0 = now;
      if (now - t0 > c.wait_ns) {
        atomicOr(c.err, code);
        *c.abort = 1u;
        return false;
      }
    }
  }
}
__device__ __forceinline__ bool wait_stage(uint64_t* bar, uint32_t parity, const Ctl& c) {
  return mbar_test(bar, parity) || wait_slow(bar, parity, c, kErrWaitTimeout, false);
}

// Tile t of the persistent loop: bands of g.band tile rows, column by column
// inside a band, so that the CTAs running at one time share operand rows in L2.
__device__ __forceinline__ void tile_coords(const GemmShape& g, int t, int& tm, int& tn) {
  const int band = g.by_band(t), first = band * g.band, rows = min(g.band, g.tiles_m - first);
  const int r = t - first * g.tiles_n;
  tn = rows == g.band ? g.by_rows(r) : g.by_last(r);
  tm = first + r - tn * rows;
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

// gg = ga u act'(z), gu = ga act(z) and a = act(z) u; act' = s + z s (1 - s) r'(z).
// r' is kept finite: z z overflows from |z| = 1.8e19 on, where s is 0 or 1 and the
// product with it is 0.
__device__ __forceinline__ void gate_grads(float z, float u, float ga, int act, float& gg, float& gu, float& a) {
  const float s = sigmoid_fast(act_arg(z, act));
  const float dr = act == 0 ? 1.0f : fminf(1.5957691216f * fmaf(3.0f * 0.044715f, z * z, 1.0f), 3e38f);
  const float h = z * s;
  gg = ga * u * fmaf(h * (1.0f - s), dr, s);
  gu = ga * h;
  a = h * u;
}

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

// A warp's staging buffer: 32 rows (its accumulator lanes) of 128 bytes in the
// 128-byte swizzle.  A lane holds one row, so writing rows to memory straight
// from registers would touch 32 distant lines per instruction, 16 bytes each;
// through the buffer a warp instruction covers whole rows (kept sums of the
// forward at T = 4096, D = 4096, F = 8192: 573 -> 538 us).
constexpr int kStageBuf = 4096;

// 32 rows x 128 bytes to memory: row r at base + r * pitch, the first `bytes`
// (a multiple of 16) of each row, rows below `rows`.
__device__ __forceinline__ void stage_flush(const uint8_t* buf, uint8_t* base, size_t pitch, int rows, int bytes, int lane) {
  __syncwarp();
  const int c = lane & 7;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = i * 4 + (lane >> 3);
    const uint4 v = *reinterpret_cast<const uint4*>(buf + sw128(r, c));
    if (r < rows && c * 16 < bytes) *reinterpret_cast<uint4*>(base + (size_t)r * pitch + c * 16) = v;
  }
  __syncwarp();
}
// The same for byte rows whose pitch is only a multiple of 8.
__device__ __forceinline__ void stage_flush8(const uint8_t* buf, uint8_t* base, size_t pitch, int rows, int bytes, int lane) {
  __syncwarp();
  const int c = lane & 15;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int r = i * 2 + (lane >> 4);
    const uint2 v = *reinterpret_cast<const uint2*>(buf + sw128(r, c >> 1) + (c & 1) * 8);
    if (r < rows && c * 8 < bytes) *reinterpret_cast<uint2*>(base + (size_t)r * pitch + c * 8) = v;
  }
  __syncwarp();
}

// out[row, col] = round(acc), one output per product of the launch; with slices
// of the depth their fp32 sums, part[slice][row][col], which ffn_sum_kernel joins.
struct StoreTo {
  uint16_t* out;
  int M, N;
  float* part;
};
template <bool F16, int P>
struct EpiStore {
  StoreTo to[P];
  // which, slice: the product and its part; taddr: the warp's accumulator lanes;
  // row0: the row of its lane 0; tn, cols: the tile's column and width; grp: which
  // half of them
  __device__ __forceinline__ void tile(int which, int slice, uint32_t taddr, int row0, int tn, int cols, int grp,
                                       uint8_t* buf, int lane) const {
    uint16_t* out = to[which].out;
    const int M = to[which].M, N = to[which].N;
    const int n0 = tn * cols;
    if (to[which].part) {
      float* part = to[which].part + ((size_t)slice * M + row0) * N + n0;
#pragma unroll 1
      for (int c = grp * (cols / 2); c < (grp + 1) * (cols / 2) && n0 + c < N; c += 32) {
        float v[32];
        acc_ld32(taddr + c, v);
#pragma unroll
        for (int q = 0; q < 8; ++q)
          *reinterpret_cast<float4*>(buf + sw128(lane, q)) = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
        stage_flush(buf, reinterpret_cast<uint8_t*>(part + c), (size_t)N * 4, M - row0, min(32, N - n0 - c) * 4, lane);
      }
      return;
    }
    const int end = (grp + 1) * (cols / 2);        // the last step may have 32 columns
#pragma unroll 1
    for (int c = grp * (cols / 2); c < end && n0 + c < N; c += 64) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (h && c + 32 >= end) break;
        float v[32];
        acc_ld32(taddr + c + 32 * h, v);
#pragma unroll
        for (int q = 0; q < 4; ++q) *reinterpret_cast<uint4*>(buf + sw128(lane, h * 4 + q)) = pack8v<F16>(v + 8 * q);
      }
      stage_flush(buf, reinterpret_cast<uint8_t*>(out + (size_t)row0 * N + n0 + c), (size_t)N * 2, M - row0,
                  min(min(64, end - c), N - n0 - c) * 2, lane);
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
  __device__ __forceinline__ void tile(int, int, uint32_t taddr, int row0, int tn, int, int grp, uint8_t* buf, int lane) const {
    const int f0 = tn * 128, rows = T - row0, c = grp * 64;
    if (f0 + c < F) {
      const int bytes = min(64, F - f0 - c) * 2;
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        float g[16], u[16];
        acc_ld16x2(taddr + c + 16 * h, taddr + 128 + c + 16 * h, g, u);
#pragma unroll
        for (int e = 0; e < 16; ++e) u[e] *= g[e] * sigmoid_fast(act_arg(g[e], act));
#pragma unroll
        for (int q = 0; q < 2; ++q) *reinterpret_cast<uint4*>(buf + sw128(lane, h * 2 + q)) = pack8v<F16>(u + 8 * q);
      }
      stage_flush(buf, reinterpret_cast<uint8_t*>(a + (size_t)row0 * F + f0 + c), (size_t)F * 2, rows, bytes, lane);
      if constexpr (kKept == 1) {
#pragma unroll 1
        for (int p = 0; p < 2; ++p) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float v[32];
            acc_ld32(taddr + p * 128 + c + 32 * h, v);
#pragma unroll
            for (int q = 0; q < 4; ++q) *reinterpret_cast<uint4*>(buf + sw128(lane, h * 4 + q)) = pack8v<F16>(v + 8 * q);
          }
          stage_flush(buf, reinterpret_cast<uint8_t*>(gate_up + ((size_t)row0 * 2 + p) * F + f0 + c), (size_t)F * 4, rows,
                      bytes, lane);
        }
      }
    }
    if constexpr (kKept == 2) {
      const int nblk = (F + kCkptBlock - 1) / kCkptBlock;
      {
        const int p = grp;                       // one group the gate's blocks, the other the up's
        float amax = 0.0f;                       // columns beyond F hold zeros (or NaN)
#pragma unroll 1
        for (int c = 0; c < 128; c += 32) {
          float v[32];
          acc_ld32(taddr + p * 128 + c, v);
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const float m = fabsf(v[e]);
            amax = m < __int_as_float(0x7F800000) ? fmaxf(amax, m) : amax;
          }
        }
        const int ex = ckpt_exponent<F16>(amax);
        const float inv = pow2_f32(-ex);
        if (lane < rows) scales[((size_t)(row0 + lane) * 2 + p) * nblk + tn] = (uint8_t)(ex + 127);
#pragma unroll 1
        for (int c = 0; c < 128; c += 32) {
          float v[32];
          acc_ld32(taddr + p * 128 + c, v);
#pragma unroll
          for (int e = 0; e < 32; ++e)
            v[e] = fabsf(v[e]) < __int_as_float(0x7F800000) ? v[e] * inv : __int_as_float(0x7FFFFFFF);
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const float* w = v + 16 * q;
            *reinterpret_cast<uint4*>(buf + sw128(lane, (c >> 4) + q)) =
                make_uint4(e4m3x4(w[0], w[1], w[2], w[3]), e4m3x4(w[4], w[5], w[6], w[7]),
                           e4m3x4(w[8], w[9], w[10], w[11]), e4m3x4(w[12], w[13], w[14], w[15]));
          }
        }
        uint8_t* base = codes + ((size_t)row0 * 2 + p) * F + f0;
        const int bytes = min(128, F - f0);
        if (F % 16 == 0) stage_flush(buf, base, (size_t)F * 2, rows, bytes, lane);
        else stage_flush8(buf, base, (size_t)F * 2, rows, bytes, lane);
      }
    }
  }
};

// acc = ga: gg, gu and a from the kept g and u.  Thirty-two columns at a time:
// the kept sums come in over the buffer (g in the first half of its 128-byte
// rows, u in the second), loaded one step ahead.
template <bool F16, int kKept>
struct EpiDgate {
  const uint16_t* gate_up;
  const uint8_t *codes, *scales;
  uint16_t *gg, *a;
  int T, F, act;

  // g and u of columns [f, f + 32) for eight rows per instruction (lane / 4,
  // eight columns each): 16 bytes, or 8 from codes
  struct Kept {
    uint4 v[2][4];
    uint32_t s[2];
  };
  __device__ __forceinline__ void load(Kept& k, int row0, int f, int lane) const {
    const int c = (lane & 3) * 8;
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      k.s[p] = 127;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = row0 + i * 8 + (lane >> 2);
        k.v[p][i] = make_uint4(0, 0, 0, 0);
        if (r < T && f + c < F) {
          const size_t at = ((size_t)r * 2 + p) * F + f + c;
          if constexpr (kKept == 1) {
            k.v[p][i] = *reinterpret_cast<const uint4*>(gate_up + at);
          } else {
            const uint2 w = *reinterpret_cast<const uint2*>(codes + at);
            k.v[p][i].x = w.x;
            k.v[p][i].y = w.y;
          }
        }
      }
      if constexpr (kKept == 2) {
        const int r = row0 + lane;
        if (r < T && f < F) k.s[p] = scales[((size_t)r * 2 + p) * ((F + kCkptBlock - 1) / kCkptBlock) + (f >> 7)];
      }
    }
  }

  __device__ __forceinline__ void tile(int, int, uint32_t taddr, int row0, int tn, int cols, int grp, uint8_t* buf,
                                       int lane) const {
    const int f0 = tn * cols, rows = T - row0, c0 = grp * (cols / 2), c1 = c0 + cols / 2;
    Kept k;
    load(k, row0, f0 + c0, lane);
#pragma unroll 1
    for (int c = c0; c < c1 && f0 + c < F; c += 32) {
      const int f = f0 + c;
      __syncwarp();
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<uint4*>(buf + sw128(i * 8 + (lane >> 2), p * 4 + (lane & 3))) = k.v[p][i];
      const float s0 = ckpt_scale(k.s[0]), s1 = ckpt_scale(k.s[1]);
      if (c + 32 < c1) load(k, row0, f + 32, lane);
      float ga[32];
      acc_ld32(taddr + c, ga);
      __syncwarp();
      uint4 o[3][4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float z[8], u[8];
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const uint4 w = *reinterpret_cast<const uint4*>(buf + sw128(lane, p * 4 + q));
          float* d = p ? u : z;
          if constexpr (kKept == 1) {
            const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 t = unpack2<F16>(ww[e]);
              d[2 * e] = t.x;
              d[2 * e + 1] = t.y;
            }
          } else {
            const float s = p ? s1 : s0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 t = e4m3x2_f2((e < 2 ? w.x : w.y) >> (16 * (e & 1)));
              d[2 * e] = t.x * s;
              d[2 * e + 1] = t.y * s;
            }
          }
        }
        float og[8], ou[8], oa[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) gate_grads(z[e], u[e], ga[8 * q + e], act, og[e], ou[e], oa[e]);
        o[0][q] = pack8v<F16>(og);
        o[1][q] = pack8v<F16>(ou);
        o[2][q] = pack8v<F16>(oa);
      }
      __syncwarp();
      // gg and gu side by side, then a
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        *reinterpret_cast<uint4*>(buf + sw128(lane, q)) = o[0][q];
        *reinterpret_cast<uint4*>(buf + sw128(lane, 4 + q)) = o[1][q];
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = i * 4 + (lane >> 3), p = (lane >> 2) & 1, cc = (lane & 3) * 8;
        const uint4 v = *reinterpret_cast<const uint4*>(buf + sw128(r, lane & 7));
        if (r < rows && f + cc < F) *reinterpret_cast<uint4*>(gg + ((size_t)(row0 + r) * 2 + p) * F + f + cc) = v;
      }
      __syncwarp();
#pragma unroll
      for (int q = 0; q < 4; ++q) *reinterpret_cast<uint4*>(buf + sw128(lane, q)) = o[2][q];
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = i * 8 + (lane >> 2), cc = (lane & 3) * 8;
        const uint4 v = *reinterpret_cast<const uint4*>(buf + sw128(r, lane & 3));
        if (r < rows && f + cc < F) *reinterpret_cast<uint4*>(a + (size_t)(row0 + r) * F + f + cc) = v;
      }
    }
    __syncwarp();
  }
};

// ------------------------------------------------------------------ kernel

// kPair: B's 256 rows are 128 rows of plane 0 (in the even CTA) and the same
// 128 of plane 1 (gate and up); else 256 consecutive rows.  A tile's operands
// may each be K-major or MN-major (g.a_mn, g.b_mn): a stage holds 128 rows of
// 128 bytes along the depth, or two blocks of 64 depths x 64 rows.
// kDraw: tiles are drawn from the counter, else dealt out in turn (products of
// one depth: nothing to balance, and no wait for the counter).
template <class Epi, bool kPair, int P, bool kDraw>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGemmThreads, 1)
    ffn_gemm_kernel(const __grid_constant__ GemmSet<P> set, const FfnCall call, const int first, const int withhold,
                    const __grid_constant__ Epi epi) {
  constexpr uint32_t kTmemCols = 512;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* bufs = smem + kGemmStages * kGemmStageBytes;          // one staging buffer per epilogue warp
  GemmTail* tail = reinterpret_cast<GemmTail*>(bufs + 8 * kStageBuf);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  int ntiles = 0;
#pragma unroll
  for (int i = 0; i < P; ++i) ntiles += gemm_tiles(set.op[i].g);
  Ctl ctl{&tail->abort, call.err, call.wait_ns};

  if (threadIdx.x == 0) {
    // Cleared here rather than by a launch of its own: a wait of this call
    // sets the word wait_ns after its CTA began at the earliest, and the tile
    // counter serves a later launch of the call.
    if (first && blockIdx.x == 0) call.err[0] = call.err[1] = 0u;
    for (int s = 0; s < kGemmStages; ++s) {
      mbar_init(&tail->full[s], 1);
      mbar_init(&tail->empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tail->acc_full[b], 1);
      mbar_init(&tail->acc_empty[b], 16);        // eight warps of each CTA
    }
    for (int b = 0; b < kSchedSlots; ++b) {
      mbar_init(&tail->sched_full[b], 1);
      mbar_init(&tail->sched_empty[b], 18);      // MMA issuer, the other producer, eight epilogue warps of each CTA
    }
    mbar_init(&tail->mma_done, 1);
    tail->abort = 0u;
    tail->sent[0] = tail->sent[1] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
#pragma unroll
    for (int i = 0; i < P; ++i) {
      tma_prefetch_desc(&set.op[i].a);
      tma_prefetch_desc(&set.op[i].b);
    }
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tail->tmem_base)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();                            // the peer's barriers exist
  tc_fence_after();
  const uint32_t tmem_base = tail->tmem_base;
  pdl_trigger();
  pdl_wait();                                    // operands, and the counter, are earlier launches'

  // The n-th tile of this pair as the roles see it: its number, or -1 after the
  // last (and when the wait for it gave up).  One call per n and role.
  auto tile_of = [&](int n, bool whole_warp) -> int {
    if constexpr (!kDraw) {
      const long long t = pair + (long long)n * pairs;
      return t < ntiles ? (int)t : -1;
    } else {
      const int slot = n % kSchedSlots;
      int t = -1;
      if (mbar_test_cluster(&tail->sched_full[slot], (uint32_t)(n / kSchedSlots) & 1u) ||
          wait_slow(&tail->sched_full[slot], (uint32_t)(n / kSchedSlots) & 1u, ctl, kErrClusterWait, true))
        t = *reinterpret_cast<volatile int*>(&tail->sched[slot]);
      if (whole_warp) t = __shfl_sync(0xFFFFFFFFu, t, 0);
      if (!whole_warp || lane == 0) mbar_arrive_remote(&tail->sched_empty[slot], 0);
      return t;
    }
  };
  // Tile t: its product, slice, row and column.
  auto locate = [&](int t, int& slice, int& tm, int& tn) -> int {
    int which = 0;
#pragma unroll
    for (int i = 0; i + 1 < P; ++i) {
      const int tiles = gemm_tiles(set.op[i].g);
      if (which == i && t >= tiles) {
        t -= tiles;
        which = i + 1;
      }
    }
    const int area = set.op[which].g.tiles_m * set.op[which].g.tiles_n;
    slice = set.op[which].g.by_area(t);
    tile_coords(set.op[which].g, t - slice * area, tm, tn);
    return which;
  };

  if (warp == 0) {
    // ===================================================== TMA producer
    if (lane == 0) {
      int s = 0;
      uint32_t ph = 0;
      long long iss = 0;
      bool ok = true;
      // Hands tile number t out as the pair's n-th.
      auto publish = [&](int n, int t) -> bool {
        const int slot = n % kSchedSlots;
        if (!wait_slow(&tail->sched_empty[slot], ((uint32_t)(n / kSchedSlots) & 1u) ^ 1u, ctl, kErrClusterWait, true)) return false;
        *reinterpret_cast<volatile int*>(&tail->sched[slot]) = t;
        asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(map_cluster(&tail->sched[slot], 1)), "r"(t) : "memory");
        mbar_arrive(&tail->sched_full[slot]);
        mbar_arrive_remote(&tail->sched_full[slot], 1);
        return true;
      };
      auto draw = [&]() -> int {
        const unsigned t = (unsigned)pairs + atomicAdd(call.err + 1, 1u);
        return t < (unsigned)ntiles ? (int)t : -1;
      };
      int cur = -1, next = -1;                   // the numbers of tiles n and n + 1, handed out already
      if (kDraw && rank == 0) {
        cur = pair;
        next = draw();
        ok = publish(0, cur) && publish(1, next);
      }
      for (int n = 0; ok; ++n) {
        const int t = kDraw && rank == 0 ? cur : tile_of(n, false);
        if (t < 0) break;
        int slice, tm, tn;
        const int which = locate(t, slice, tm, tn);
        const GemmShape& g = set.op[which].g;
        const CUtensorMap* ta = &set.op[which].a;
        const CUtensorMap* tb = &set.op[which].b;
        const int m0 = tm * kFfnTileM + (int)rank * kGemmHalf;
        const int half_n = g.tile_n / 2;
        const int n0 = kPair ? tn * kGemmHalf : tn * g.tile_n + (int)rank * half_n;
        const int plane = kPair ? (int)rank : 0, a_mn = g.a_mn, b_mn = g.b_mn;
        const uint32_t bytes = 2u * stage_bytes_of(g);
        const int kbeg = slice * g.kslice, kiters = min(g.kslice, g.kiters - kbeg);
        // test hook: the first two pairs leave out the last chunk of their first
        // tile, so the waits on it give up; the first pair's odd CTA and the
        // second pair's even one also leave out the one before it
        const int kend = withhold && pair < 2 && n == 0 ? max(kiters - 1 - (int)(rank ^ (uint32_t)pair), 0) : kiters;
        int after = -1;                          // tile n + 2, drawn under this tile's copies
        if (kDraw && rank == 0 && next >= 0) after = draw();
        for (int k = 0; k < kend; ++k) {
          if (!wait_stage(&tail->empty[s], ph ^ 1u, ctl)) { ok = false; break; }
          const uint32_t sa = smem_u32(smem + s * kGemmStageBytes), sb = sa + kGemmOpBytes;
          const uint32_t bar = map_cluster(&tail->full[s], 0);
          const int k0 = (kbeg + k) * kFfnTileK;
          if (rank == 0) mbar_expect_tx(&tail->full[s], bytes);
          if (a_mn) {
            tma_load_3d_pair(sa, ta, bar, m0, k0, 0);
            tma_load_3d_pair(sa + 8192, ta, bar, m0 + 64, k0, 0);
          } else {
            tma_load_3d_pair(sa, ta, bar, k0, m0, 0);
          }
          if (b_mn) {
            tma_load_3d_pair(sb, tb, bar, n0, k0, 0);
            if (half_n > 64) tma_load_3d_pair(sb + 8192, tb, bar, n0 + 64, k0, 0);
          } else {
            tma_load_3d_pair(sb, tb, bar, k0, n0, plane);
          }
          ++iss;
          if (++s == kGemmStages) { s = 0; ph ^= 1u; }
        }
        ok = ok && kend == kiters;
        if (kDraw && rank == 0) {                // after the last tile: -1
          ok = ok && publish(n + 2, after);
          cur = next;
          next = after;
        }
      }
      asm volatile("st.release.cluster.shared::cluster.b64 [%0], %1;" ::"r"(map_cluster(&tail->sent[rank], 0)), "l"(iss + 1)
                   : "memory");
    }
  } else if (warp == 1) {
    // ===================================================== MMA issuer
    if (rank == 0) {
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int n = 0; ok; ++n) {
        const int t = tile_of(n, true);
        if (t < 0) break;
        int slice, tm, tn;
        const GemmShape& g = set.op[locate(t, slice, tm, tn)].g;
        // byte step of sixteen depths, and the distance of the next 64 rows
        const uint64_t a0 = g.a_mn ? sw128_desc_mn(0, 8192) : sw128_desc(0), b0 = g.b_mn ? sw128_desc_mn(0, 8192) : sw128_desc(0);
        const uint32_t astep = (g.a_mn ? 2048u : 32u) >> 4, bstep = (g.b_mn ? 2048u : 32u) >> 4, idesc = g.idesc;
        const int b = n & 1, kiters = min(g.kslice, g.kiters - slice * g.kslice);
        if (!wait_slow(&tail->acc_empty[b], ((uint32_t)(n >> 1) & 1u) ^ 1u, ctl, kErrClusterWait, true)) break;
        tc_fence_after();
        const uint32_t d = tmem_base + (uint32_t)(b * kFfnTileN);
        for (int k = 0; k < kiters; ++k) {
          if (!wait_stage(&tail->full[s], ph, ctl)) { ok = false; break; }
          tc_fence_after();
          const uint32_t sa = desc_addr(smem + s * kGemmStageBytes), sb = sa + (kGemmOpBytes >> 4);
          if (elect_one()) {
#pragma unroll
            for (int ks = 0; ks < kFfnTileK / 16; ++ks)
              mma_pair(d, a0 + (sa + ks * astep), b0 + (sb + ks * bstep), idesc, (k | ks) ? 1u : 0u);
            commit_pair(&tail->empty[s]);
          }
          __syncwarp();
          if (++s == kGemmStages) { s = 0; ph ^= 1u; }
        }
        if (ok && elect_one()) commit_pair(&tail->acc_full[b]);
        __syncwarp();
      }
      if (elect_one()) asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                       smem_u32(&tail->mma_done))
                   : "memory");
      __syncwarp();
      mbar_drain(&tail->mma_done, 0);
      // Products that were all formed have consumed all copies.  The products of
      // a launch have tiles of one width and one layout of B.
      if ((!ok || *ctl.abort) && lane == 0) settle_copies(tail, ctl.wait_ns, stage_bytes_of(set.op[0].g));
      __syncwarp();
    }
  } else {
    // ===================================================== epilogue
    const int grp = (warp - 2) >> 2, q = warp & 3;
    for (int n = 0;; ++n) {
      const int t = tile_of(n, true);
      if (t < 0) break;
      int slice, tm, tn;
      const int which = locate(t, slice, tm, tn), b = n & 1;
      if (!__all_sync(0xFFFFFFFFu, wait_stage(&tail->acc_full[b], (uint32_t)(n >> 1) & 1u, ctl))) break;
      tc_fence_after();
      epi.tile(which, slice, tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(b * kFfnTileN),
               tm * kFfnTileM + (int)rank * kGemmHalf + q * 32, tn, set.op[which].g.tile_n, grp,
               bufs + (warp - 2) * kStageBuf, lane);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(&tail->acc_empty[b], 0);
    }
  }

  // ---- teardown: the pair leaves together
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(kTmemCols) : "memory");
  }
}

// out = round(sum of the slices), in their order; eight values a thread.
template <bool F16>
__global__ void __launch_bounds__(256) ffn_sum_kernel(const float* part, int slices, long long count, uint16_t* out) {
  pdl_wait();
  for (long long i = ((long long)blockIdx.x * 256 + threadIdx.x) * 8; i < count; i += (long long)gridDim.x * 2048) {
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 0.0f;
    for (int s = 0; s < slices; ++s) {
      const float4 a = *reinterpret_cast<const float4*>(part + s * count + i);
      const float4 b = *reinterpret_cast<const float4*>(part + s * count + i + 4);
      v[0] += a.x;
      v[1] += a.y;
      v[2] += a.z;
      v[3] += a.w;
      v[4] += b.x;
      v[5] += b.y;
      v[6] += b.z;
      v[7] += b.w;
    }
    *reinterpret_cast<uint4*>(out + i) = pack8v<F16>(v);
  }
}
template <bool F16>
cudaError_t launch_sum(const StoreTo& to, int slices, int sms, cudaStream_t s) {
  const long long count = (long long)to.M * to.N, blocks = (count + 2047) / 2048;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)(blocks < 8ll * sms ? blocks : 8ll * sms));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, ffn_sum_kernel<F16>, (const float*)to.part, (int)slices, (long long)count, to.out);
}

// first: the call's first launch (ordered behind everything before it, clears
// the error word); later ones start as SMs fall free.  last: takes the test hook.
template <bool kPair, bool kDraw, int P, class Epi>
cudaError_t launch_gemm(const GemmSet<P>& set, const FfnCall& call, const Epi& epi, bool first, bool last, cudaStream_t s) {
  auto* k = ffn_gemm_kernel<Epi, kPair, P, kDraw>;
  // per device: the shared-memory limit is set, and the pairs that fit at once
  // counted (some SMs may have no partner)
  static std::atomic<int> known[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.blockDim = dim3(kGemmThreads);
  cfg.dynamicSmemBytes = kGemmSmem;
  int pairs = known[dev].load(std::memory_order_relaxed);
  if (pairs == 0) {
    e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kGemmSmem);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3((unsigned)(call.sms & ~1));
    if ((e = cudaOccupancyMaxActiveClusters(&pairs, k, &cfg)) != cudaSuccess) return e;
    if (pairs < 1) return cudaErrorInvalidConfiguration;
    known[dev].store(pairs, std::memory_order_relaxed);
  }
  long long tiles = 0;
  for (int i = 0; i < P; ++i) tiles += gemm_tiles(set.op[i].g);
  cfg.gridDim = dim3((unsigned)(2 * (tiles < pairs ? tiles : pairs)));
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = first ? 0 : 1;
  return cudaLaunchKernelEx(&cfg, k, set, call, (const int)first, (const int)(last ? call.withhold : 0), epi);
}

}  // namespace mhc
