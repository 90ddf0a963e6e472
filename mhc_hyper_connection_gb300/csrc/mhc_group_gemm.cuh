// mhc_group_gemm.cuh -- matrix products whose tiles a job describes: the routed
// experts' products (groups of rows whose sizes only the device knows) and the
// products of the orthogonalisation (many small matrices, symmetric results).
//
// The kernel is built as the feed-forward block's (mhc_ffn_gemm.cuh): persistent
// pairs of CTAs, one tcgen05 cta_group::2 product of 256 rows of A by up to 256 of
// B per step, operands by TMA through a ring of stages, two tensor-memory
// accumulators so that epilogues overlap the next tile's products.  What differs:
// a job maps a tile number to operands, width and depth (each tile's own), stages
// are as many as the job's operands leave room for, and a tile deeper than
// kGrpDeepest chunks is formed in parts that the epilogue joins in fp32.  Large products
// keep the tensor pipe 80 to 88% busy (products whose epilogues read as much as they write
// 70 to 75%) and are then held by the power limit.
#pragma once

#include "mhc_ffn_gemm.cuh"

namespace mhc {

constexpr int kGrpThreads = 352;                     // producer, MMA issuer, 2 x 4 epilogue warps, scheduler
constexpr int kGrpMaxStages = 12;
constexpr int kGrpRing = 6 * 32768;                  // bytes of the ring of stages
constexpr int kGrpDeepest = 512;                     // chunks of the depth that one accumulator sums at most

// A tile of a job.  e < 0: no more tiles.
struct __align__(16) GTile {
  int e;                       // group (expert, matrix)
  int tm, tn;                  // tile row and, where the job has them, column
  int row0, rows;              // first row of the group's part and its rows that count
  int width;                   // rows of B, a multiple of 32
  int kiters;                  // chunks of the depth (0: nothing to sum)
  int kind;                    // which of the job's products
};

struct GrpTail {
  uint64_t full[kGrpMaxStages], empty[kGrpMaxStages];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t sched_full[kSchedSlots], sched_empty[kSchedSlots];
  uint64_t mma_done;
  uint64_t sent[2];                        // as in GemmTail
  uint32_t sent_bytes[2][kGrpMaxStages];   // bytes of each CTA's last copies into a stage
  uint32_t tmem_base;
  uint32_t abort;
  uint32_t handed;                         // tiles that the scheduler handed out, the last one's -1 among them
  GTile sched[kSchedSlots];
};
constexpr size_t kGrpSmem = (size_t)kGrpRing + 8 * kStageBuf + sizeof(GrpTail) + 1024;
static_assert(kGrpSmem <= 232448, "shared memory of a CTA");

struct GrpCall {
  uint32_t* err;               // device error word
  uint32_t* counter;           // tiles drawn so far, zero at the launch (jobs that draw)
  uint64_t wait_ns;
  int withhold;                // test hook
  int stages, stage_bytes;     // of the ring, per CTA
};

__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
      : "memory");
}
__device__ __forceinline__ void tma_load_4d_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1,
                                                 int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}
__device__ __forceinline__ void tma_load_5d_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1,
                                                 int c2, int c3, int c4) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4)
      : "memory");
}
// 16 bytes to a CTA of the cluster, completing 16 bytes of a barrier there: the waiter sees
// them without a release by the sender (one costs a thousand clocks or two).
__device__ __forceinline__ void st_async_v4(uint32_t addr, int4 v, uint32_t bar) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(addr), "r"(v.x),
               "r"(v.y), "r"(v.z), "r"(v.w), "r"(bar)
               : "memory");
}
__device__ __forceinline__ void expect_tx_relaxed(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.relaxed.cluster.shared::cluster.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
// Arrive on CTA 0's barrier without a release: what it hands back (tensor memory, a
// scheduler slot) was only read, and the reads are complete.  A release would first wait
// for the epilogue's global stores, a microsecond a tile.
__device__ __forceinline__ void arrive_relaxed(uint64_t* bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(map_cluster(bar, 0)) : "memory");
}
__device__ __forceinline__ int4 ld_slot(const void* p) {
  int4 v;
  asm volatile("ld.volatile.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(smem_u32(p)) : "memory");
  return v;
}

// As settle_copies of mhc_ffn_gemm.cuh, for stages whose bytes differ: both CTAs
// copy the same number of bytes into a stage and leave behind what they last
// copied into each.
static __device__ __noinline__ void grp_settle(GrpTail* tail, uint64_t wait_ns, int stages) {
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
    const int s = (int)(k % stages);
    if (mine < theirs) mbar_expect_tx(&tail->full[s], *(volatile uint32_t*)&tail->sent_bytes[1][s]);
    else mbar_complete_tx(&tail->full[s], *(volatile uint32_t*)&tail->sent_bytes[0][s]);
  }
  for (long long k = most > stages ? most - stages : 0; k < most; ++k)
    mbar_drain(&tail->full[k % stages], (uint32_t)(k / stages) & 1u);
}

__host__ __device__ constexpr uint32_t grp_idesc(bool f16, bool a_mn, bool b_mn, int width) {
  return (f16 ? (1u << 4) : ((1u << 4) | (1u << 7) | (1u << 10))) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) |
         ((uint32_t)(width >> 3) << 17) | ((uint32_t)(kFfnTileM >> 4) << 24);
}

// Job:
//   kAMn, kBMn           operands stored MN-major
//   kEarly               tiles, Raw and A do not depend on the launches that this one overlaps
//   kDraw                tiles are drawn from the counter (their work differs), else dealt out in turn
//   int tiles() const    their number (read once earlier launches are complete)
//   Raw fetch(int t)     what tile t needs from memory, loaded ahead of its use
//   GTile make(int t, const Raw&)
//   int bytes(const GTile&)                       bytes that one CTA copies into a stage
//   void load_a(tile, k, sa, bar, rank), load_b   chunk k of the depth into a stage
//   int steps(tile, k)                            products of depth 16 in chunk k
//   uint32_t idesc(tile)
//   void prefetch()                               tensor-map descriptors
// Epi:
//   Pre, void pre(tile, Pre&, rank, q, grp, lane)   loads ahead of a tile's sums
//   void tile(tile, Pre&, part, parts, taddr, rank, q, grp, buf, lane, pair)
template <class Job, class Epi>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGrpThreads, 1)
    group_gemm_kernel(const __grid_constant__ Job job, const GrpCall call, const __grid_constant__ Epi epi) {
  constexpr uint32_t kTmemCols = 512;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* bufs = smem + kGrpRing;
  GrpTail* tail = reinterpret_cast<GrpTail*>(bufs + 8 * kStageBuf);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int stages = call.stages, stage_bytes = call.stage_bytes;
  Ctl ctl{&tail->abort, call.err, call.wait_ns};

  if (threadIdx.x == 0) {
    for (int s = 0; s < kGrpMaxStages; ++s) {
      mbar_init(&tail->full[s], 1);
      mbar_init(&tail->empty[s], 1);
      tail->sent_bytes[0][s] = tail->sent_bytes[1][s] = 0;
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tail->acc_full[b], 1);
      mbar_init(&tail->acc_empty[b], 16);
    }
    for (int b = 0; b < kSchedSlots; ++b) {
      mbar_init(&tail->sched_full[b], 1);
      mbar_init(&tail->sched_empty[b], 19);      // MMA issuer, both producers, eight epilogue warps of each CTA
    }
    mbar_init(&tail->mma_done, 1);
    tail->abort = tail->handed = 0u;
    tail->sent[0] = tail->sent[1] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    job.prefetch();
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
  // Operands and the counter are earlier launches'.  The producers of a job whose A is not
  // (an expert's weights) begin with it before they wait.
  const bool scheduler = warp == 10;
  if (!Job::kEarly || (warp != 0 && !scheduler)) pdl_wait();
  const int ntiles = job.tiles();

  // The n-th tile of this pair as the roles see it (e = -1 after the last, and when
  // the wait for it gave up).  One call per n and role.
  auto tile_of = [&](int n, bool whole_warp) -> GTile {
    GTile g;
    g.e = -1;
    if constexpr (!Job::kDraw) {
      const long long t = pair + (long long)n * pairs;
      if (t < ntiles) g = job.make((int)t, job.fetch((int)t));
      return g;
    } else {
      const int slot = n % kSchedSlots;
      const uint32_t par = (uint32_t)(n / kSchedSlots) & 1u;
      bool ok = mbar_test_cluster(&tail->sched_full[slot], par) ||
                wait_slow(&tail->sched_full[slot], par, ctl, kErrClusterWait, true);
      if (whole_warp) ok = __all_sync(0xFFFFFFFFu, ok);
      bool read = true;
      if (ok) {
        const int4 lo = ld_slot(&tail->sched[slot]), hi = ld_slot(&tail->sched[slot].rows);
        read = lo.x >= -1 && hi.w >= 0;          // always
        g.e = lo.x;
        g.tm = lo.y;
        g.tn = lo.z;
        g.row0 = lo.w;
        g.rows = hi.x;
        g.width = hi.y;
        g.kiters = hi.z;
        g.kind = hi.w;
      }
      // The arrival orders nothing by itself, and the scheduler's next write of the slot must
      // not meet loads still under way: whether it is made goes by a value of each load, so no
      // thread issues it before these are there, nor lane 0 before all lanes' are.
      if (whole_warp) read = __all_sync(0xFFFFFFFFu, read);
      if (!read) g.e = -1;
      else if (!whole_warp || lane == 0) arrive_relaxed(&tail->sched_empty[slot]);
      return g;
    }
  };

  if (warp == 0) {
    // ===================================================== TMA producer
    if (lane == 0) {
      int s = 0;
      uint32_t ph = 0;
      long long iss = 0;
      bool ok = true;
      GTile first;                               // the pair's first tile, known without the scheduler
      int early = 0;                             // chunks of it whose A is on its way
      const uint32_t ring = smem_u32(smem), full0 = map_cluster(&tail->full[0], 0);
      if constexpr (Job::kEarly) {
        first.e = -1;
        if (pair < ntiles) first = job.make(pair, job.fetch(pair));
        if (first.e >= 0 && !call.withhold) {
          early = min(stages, first.kiters);
          for (int k = 0; k < early; ++k) {
            if (rank == 0) mbar_expect_tx(&tail->full[k], 2u * (uint32_t)job.bytes(first));
            job.load_a(first, k, ring + k * stage_bytes, full0 + 8 * k, (int)rank);
          }
        }
        pdl_wait();
      }
      for (int n = 0; ok; ++n) {
        GTile g = tile_of(n, false);
        if (n == 0 && early) g = first;          // its copies are completed whatever became of that wait
        if (g.e < 0) break;
        const uint32_t bytes = (uint32_t)job.bytes(g);
        // test hook, as in ffn_gemm_kernel
        const int kend = call.withhold && pair < 2 && n == 0 ? max(g.kiters - 1 - (int)(rank ^ (uint32_t)pair), 0) : g.kiters;
        for (int k = 0; k < kend; ++k) {
          if (!wait_stage(&tail->empty[s], ph ^ 1u, ctl)) { ok = false; break; }
          const uint32_t sa = ring + s * stage_bytes, bar = full0 + 8 * s;
          if (n > 0 || k >= early) {
            if (rank == 0) mbar_expect_tx(&tail->full[s], 2u * bytes);
            job.load_a(g, k, sa, bar, (int)rank);
          }
          job.load_b(g, k, sa + kGemmOpBytes, bar, (int)rank);
          tail->sent_bytes[rank][s] = bytes;     // for grp_settle; the odd CTA's are sent over below
          ++iss;
          if (++s == stages) { s = 0; ph ^= 1u; }
        }
        ok = ok && kend == g.kiters;
      }
      if (rank == 1) {
        const uint32_t at = map_cluster(&tail->sent_bytes[1][0], 0);
        for (int i = 0; i < stages; ++i)
          asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(at + 4 * i), "r"(tail->sent_bytes[1][i]) : "memory");
      }
      asm volatile("st.release.cluster.shared::cluster.b64 [%0], %1;" ::"r"(map_cluster(&tail->sent[rank], 0)), "l"(iss + 1)
                   : "memory");
    }
  } else if (warp == 1) {
    // ===================================================== MMA issuer
    if (rank == 0) {
      int s = 0, acc = 0;
      uint32_t ph = 0;
      bool ok = true;
      const uint64_t a0 = Job::kAMn ? sw128_desc_mn(0, 8192) : sw128_desc(0), b0 = Job::kBMn ? sw128_desc_mn(0, 8192) : sw128_desc(0);
      constexpr uint32_t astep = (Job::kAMn ? 2048u : 32u) >> 4, bstep = (Job::kBMn ? 2048u : 32u) >> 4;
      for (int n = 0; ok; ++n) {
        const GTile g = tile_of(n, true);
        if (g.e < 0) break;
        const uint32_t idesc = job.idesc(g);
        for (int k0 = 0; k0 < g.kiters && ok; k0 += kGrpDeepest, ++acc) {
          const int b = acc & 1, k1 = min(k0 + kGrpDeepest, g.kiters);
          if (!wait_slow(&tail->acc_empty[b], ((uint32_t)(acc >> 1) & 1u) ^ 1u, ctl, kErrClusterWait, true)) { ok = false; break; }
          tc_fence_after();
          const uint32_t d = tmem_base + (uint32_t)(b * kFfnTileN);
          for (int k = k0; k < k1; ++k) {
            if (!wait_stage(&tail->full[s], ph, ctl)) { ok = false; break; }
            tc_fence_after();
            const uint32_t sa = desc_addr(smem + s * stage_bytes), sb = sa + (kGemmOpBytes >> 4);
            const int steps = job.steps(g, k);
            if (elect_one()) {
#pragma unroll
              for (int ks = 0; ks < kFfnTileK / 16; ++ks)
                if (ks < steps) mma_pair(d, a0 + (sa + ks * astep), b0 + (sb + ks * bstep), idesc, (k > k0 || ks) ? 1u : 0u);
              commit_pair(&tail->empty[s]);
            }
            __syncwarp();
            if (++s == stages) { s = 0; ph ^= 1u; }
          }
          if (ok && elect_one()) commit_pair(&tail->acc_full[b]);
          __syncwarp();
        }
      }
      if (elect_one()) asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                       smem_u32(&tail->mma_done))
                   : "memory");
      __syncwarp();
      mbar_drain(&tail->mma_done, 0);
      if ((!ok || *ctl.abort) && lane == 0) grp_settle(tail, ctl.wait_ns, stages);
      __syncwarp();
    }
  } else if (scheduler) {
    // ===================================================== scheduler
    // A warp of its own: in the producer, drawing and handing out a tile held up copies for
    // a thousand clocks a tile, and its code for half a stage in every stage.
    if (Job::kDraw && rank == 0 && lane == 0) {
      GTile none;
      none.e = -1;
      none.tm = none.tn = none.row0 = none.rows = none.width = none.kiters = none.kind = 0;
      auto publish = [&](int n, const GTile& g) -> bool {
        const int slot = n % kSchedSlots;
        if (!wait_slow(&tail->sched_empty[slot], ((uint32_t)(n / kSchedSlots) & 1u) ^ 1u, ctl, kErrClusterWait, true)) return false;
        const int4 lo = make_int4(g.e, g.tm, g.tn, g.row0), hi = make_int4(g.rows, g.width, g.kiters, g.kind);
#pragma unroll
        for (uint32_t r = 0; r < 2; ++r) {
          const uint32_t at = map_cluster(&tail->sched[slot], r), bar = map_cluster(&tail->sched_full[slot], r);
          expect_tx_relaxed(bar, 32u);
          st_async_v4(at, lo, bar);
          st_async_v4(at + 16, hi, bar);
        }
        return true;
      };
      // The first two tiles of a pair are dealt out, the others drawn.
      int t = pair;
      bool more = true;
      uint32_t handed = 0;
      for (int n = 0; more; ++n) {
        GTile g = none;
        if (t < ntiles) g = job.make(t, job.fetch(t));
        const bool sent = publish(n, g);
        handed += sent ? 1u : 0u;
        more = sent && g.e >= 0;
        if (n == 0) t = pair + pairs;
        if (n == 1 && Job::kEarly) pdl_wait();   // the counter is the first launch's
        if (n >= 1 && more) {
          const unsigned drawn = 2u * (unsigned)pairs + atomicAdd(call.counter, 1u);
          t = drawn < (unsigned)ntiles ? (int)drawn : ntiles;
        }
      }
#pragma unroll
      for (uint32_t r = 0; r < 2; ++r)
        asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(map_cluster(&tail->handed, r)), "r"(handed) : "memory");
    }
  } else {
    // ===================================================== epilogue
    const int grp = (warp - 2) >> 2, q = warp & 3;
    uint8_t* buf = bufs + (warp - 2) * kStageBuf;
    int acc = 0;
    bool ok = true;
    for (int n = 0; ok; ++n) {
      const GTile g = tile_of(n, true);
      if (g.e < 0) break;
      const int parts = (g.kiters + kGrpDeepest - 1) / kGrpDeepest;
      typename Epi::Pre pre;
      epi.pre(g, pre, (int)rank, q, grp, lane);
      if (parts == 0) epi.tile(g, pre, 0, 0, 0u, (int)rank, q, grp, buf, lane, pair);
      for (int p = 0; p < parts; ++p, ++acc) {
        const int b = acc & 1;
        if (!__all_sync(0xFFFFFFFFu, wait_stage(&tail->acc_full[b], (uint32_t)(acc >> 1) & 1u, ctl))) { ok = false; break; }
        tc_fence_after();
        epi.tile(g, pre, p, parts, tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(b * kFfnTileN), (int)rank, q, grp, buf, lane,
                 pair);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_relaxed(&tail->acc_empty[b]);
      }
    }
  }

  // ---- teardown: the pair leaves together
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  // Tiles are sent asynchronously.  Roles read all of them, up to the last one's -1, but where
  // a wait of theirs gave up: then this CTA does not leave before the last ones are there.
  if (Job::kDraw && scheduler && lane == 0 && *ctl.abort) {
    const int handed = (int)*(volatile uint32_t*)&tail->handed;
    for (int n = max(handed - kSchedSlots, 0); n < handed; ++n) {
      const uint32_t par = (uint32_t)(n / kSchedSlots) & 1u;
      if (!mbar_test(&tail->sched_full[n % kSchedSlots], par)) mbar_drain(&tail->sched_full[n % kSchedSlots], par);
    }
  }
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(kTmemCols) : "memory");
  }
}

// Launch: at most `most` tiles; started as SMs fall free of the launch before.
template <class Job, class Epi>
cudaError_t launch_group(const Job& job, const GrpCall& call, const Epi& epi, long long most, int sms, bool dependent,
                         cudaStream_t s) {
  auto* k = group_gemm_kernel<Job, Epi>;
  static std::atomic<int> known[64];             // as in launch_gemm
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.blockDim = dim3(kGrpThreads);
  cfg.dynamicSmemBytes = kGrpSmem;
  int pairs = known[dev].load(std::memory_order_relaxed);
  if (pairs == 0) {
    e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kGrpSmem);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3((unsigned)(sms & ~1));
    if ((e = cudaOccupancyMaxActiveClusters(&pairs, k, &cfg)) != cudaSuccess) return e;
    if (pairs < 1) return cudaErrorInvalidConfiguration;
    known[dev].store(pairs, std::memory_order_relaxed);
  }
  cfg.gridDim = dim3((unsigned)(2 * (most < pairs ? most : pairs)));
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = dependent ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, k, job, call, epi);
}

// The ring for stages of 128 rows of A and `b_rows` of B per CTA.
inline void grp_ring(GrpCall* c, int b_rows) {
  c->stage_bytes = kGemmOpBytes + b_rows * kFfnTileK * 2;
  c->stages = kGrpRing / c->stage_bytes;
  if (c->stages > kGrpMaxStages) c->stages = kGrpMaxStages;
}

// ------------------------------------------------ epilogues' shared pieces

// Nothing to load ahead.
struct NoPre {};

// A warp's part of an accumulator as the fragments of 8 x 8 blocks: with t = lane, element
// (row 8 i + t / 4, column 8 b + 2 (t % 4) + e) for i in 0..3 and b in 0..kB - 1 is v[i][b][e].
// Two columns of a row then pack into a word of a 16-bit matrix fragment, which stmatrix
// writes as rows or, transposed, as columns, and ldmatrix reads: an epilogue that stored
// and loaded its lanes' elements one by one took 24000 to 30000 clocks for a tile of gate
// gradients of 205 tokens and takes 17000 so, time that a tile of few products cannot hide.
template <int kB>
__device__ __forceinline__ void frag_ld(uint32_t taddr, float (&v)[4][kB][2]) {
  static_assert(kB == 2 || kB == 4, "16 or 32 columns");
#pragma unroll
  for (int h = 0; h < 2; ++h) {                  // 16 of the warp's 32 lanes
    float r[4 * kB];
    const uint32_t at = taddr + ((uint32_t)(h * 16) << 16);
    if constexpr (kB == 4) {
      asm volatile(
          "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
          : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
            "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
          : "r"(at)
          : "memory");
    } else {
      asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                   : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7])
                   : "r"(at)
                   : "memory");
    }
#pragma unroll
    for (int b = 0; b < kB; ++b) {
      v[2 * h][b][0] = r[4 * b];
      v[2 * h][b][1] = r[4 * b + 1];
      v[2 * h + 1][b][0] = r[4 * b + 2];
      v[2 * h + 1][b][1] = r[4 * b + 3];
    }
  }
  // no use of the values moves above the wait
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int b = 0; b < kB; b += 2) {
      if (i == 0 && b == 0)
        asm volatile("tcgen05.wait::ld.sync.aligned;" : "+f"(v[0][0][0]), "+f"(v[0][0][1]), "+f"(v[0][1][0]), "+f"(v[0][1][1])::"memory");
      else
        asm volatile("" : "+f"(v[i][b][0]), "+f"(v[i][b][1]), "+f"(v[i][b + 1][0]), "+f"(v[i][b + 1][1])::"memory");
    }
}
// Four 8 x 8 blocks of 16-bit elements, one word of each per lane; lane 8 n + r gives the
// address of row r of block n (16 bytes).
__device__ __forceinline__ void frag_st(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ void frag_st_t(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}
__device__ __forceinline__ void frag_lds(uint32_t addr, uint32_t (&v)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void frag_lds_t(uint32_t addr, uint32_t (&v)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
               : "r"(addr)
               : "memory");
}
// Pitches of staged rows of 64, 32 and 128 bytes: eight rows in sequence lie in eight
// different sixteen-byte columns of the banks.
constexpr int kPitch64 = 80, kPitch32 = 48, kPitch128 = 144;

// Staged rows of 64 (or 32) bytes to memory: row r at base + r pitch, 16-byte pieces below
// `pieces`, rows below `rows`.
template <int kRows>
__device__ __forceinline__ void flush64(const uint8_t* buf, uint8_t* base, size_t pitch, int rows, int pieces, int lane) {
  const int c = lane & 3;
#pragma unroll
  for (int i = 0; i < kRows / 8; ++i) {
    const int r = i * 8 + (lane >> 2);
    const uint4 w = *reinterpret_cast<const uint4*>(buf + r * kPitch64 + c * 16);
    if (r < rows && c < pieces) *reinterpret_cast<uint4*>(base + (size_t)r * pitch + c * 16) = w;
  }
}
__device__ __forceinline__ void flush32(const uint8_t* buf, uint8_t* base, size_t pitch, int rows, int pieces, int lane) {
  const int c = lane & 1;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = i * 16 + (lane >> 1);
    const uint4 w = *reinterpret_cast<const uint4*>(buf + r * kPitch32 + c * 16);
    if (r < rows && c < pieces) *reinterpret_cast<uint4*>(base + (size_t)r * pitch + c * 16) = w;
  }
}

}  // namespace mhc
