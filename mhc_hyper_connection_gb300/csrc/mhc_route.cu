// mhc_route.cu -- routing of tokens to experts (include/mhc_route.h): scores,
// choice and weights, the weights' gradient, and the counting sort of the slots.
//
// Routing and its gradient read and write each score once; a row is a warp's, its
// scores in registers, E / 32 consecutive ones a lane.  Bound by the warp's instructions
// (keys, sorting, the groups and a maximum over the warp for each choice: 1270 a row of
// 256 experts, 8 of 4 groups of 8), not by memory: 16384 such rows take 38 us, their bytes 2.6.
// Up to 256 experts a lane's scores are sorted; more are searched (8192 rows of 512: 27 us
// without a bias or groups, 66 with both).
#include <math.h>

#include "mhc_experts.cuh"
#include "mhc_ffn_gemm.cuh"
#include "mhc_host.cuh"
#include "../../include/mhc_route.h"

namespace mhc {
namespace {

constexpr uint32_t kFull = 0xFFFFFFFFu;
constexpr int kRouteWarps = 4;

struct RouteArgs {
  const void* logits;
  const float* bias;
  int* experts;
  float* weights;
  long long T;
  int E, k, sigmoid, groups, top_groups, top2, renorm;
  float scale;
};

// fp32 and fp64 as unsigned numbers of the same order, NaN above all, -0 below +0; and back.
__device__ __forceinline__ uint32_t order(float v) {
  const uint32_t b = __float_as_uint(v);
  return v != v ? 0xFFFFFFFFu : b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ unsigned long long order(double v) {
  const unsigned long long b = (unsigned long long)__double_as_longlong(v);
  return v != v ? ~0ull : b ^ ((b >> 63) ? ~0ull : 1ull << 63);
}
// Of the result of an fp32 sum, whose NaN is 0x7FFFFFFF.
__device__ __forceinline__ uint32_t order_sum(float v) {
  const uint32_t b = __float_as_uint(v);
  return b ^ ((uint32_t)((int)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ unsigned long long order_sum(double v) { return order(v); }
__device__ __forceinline__ float unorder(uint32_t u) {
  return u == 0xFFFFFFFFu ? NAN : __uint_as_float(u ^ ((u >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}
__device__ __forceinline__ double unorder(unsigned long long u) {
  return u == ~0ull ? (double)NAN : __longlong_as_double((long long)(u ^ ((u >> 63) ? 1ull << 63 : ~0ull)));
}
template <class K>
struct Ordered;
template <>
struct Ordered<float> {
  using U = uint32_t;
  static constexpr U kOut = 0x007FFFFFu;                   // order(-inf): an expert that is out
};
template <>
struct Ordered<double> {
  using U = unsigned long long;
  static constexpr U kOut = 0x000FFFFFFFFFFFFFull;
};

__device__ __forceinline__ uint32_t warp_max(uint32_t v) { return __reduce_max_sync(kFull, v); }
__device__ __forceinline__ unsigned long long warp_max(unsigned long long v) {
  const uint32_t hi = warp_max((uint32_t)(v >> 32));
  const uint32_t lo = warp_max((uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
  return ((unsigned long long)hi << 32) | lo;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}
__device__ __forceinline__ float sigmoid32(float l) { return 1.0f / (1.0f + expf(-l)); }

template <int kType>
__device__ __forceinline__ float load_logit(const void* p, long long at) {
  if constexpr (kType == MHC_DTYPE_FP32) return static_cast<const float*>(p)[at];
  else if constexpr (kType == MHC_DTYPE_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[at]);
  else return __half2float(static_cast<const __half*>(p)[at]);
}

// What the scores of a row's logits share: the largest logit and the sum of exponentials.
template <class K>
struct RowSum {
  float top;
  K sum;
};
// Score of a logit.  In fp32 only to be compared: fast exponential and division, a few 2^-23
// of it off.
__device__ __forceinline__ float score_of(const RouteArgs& a, float l, const RowSum<float>& r) {
  return a.sigmoid ? __fdividef(1.0f, 1.0f + __expf(-l)) : __fdividef(expf(l - r.top), r.sum);
}
__device__ __forceinline__ double score_of(const RouteArgs& a, double l, const RowSum<double>& r) {
  return a.sigmoid ? 1.0 / (1.0 + exp(-l)) : exp(l - (double)r.top) / r.sum;
}

// (u, id) of a lane in descending order of u, equal ones by id: id's low byte first.
template <class U, int V>
__device__ __forceinline__ void sort_lane(U (&u)[V], int (&id)[V]) {
  // Batcher's odd-even merges
#pragma unroll
  for (int p = 1; p < V; p *= 2) {
#pragma unroll
    for (int k = p; k > 0; k /= 2) {
#pragma unroll
      for (int j = k % p; j + k < V; j += 2 * k) {
#pragma unroll
        for (int i = 0; i < k; ++i) {
          if (i + j + k < V && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
            U &x = u[i + j], &y = u[i + j + k];
            int &xi = id[i + j], &yi = id[i + j + k];
            const bool swap = y > x || (y == x && yi < xi);
            const U t = swap ? y : x;
            y = swap ? x : y;
            x = t;
            const int ti = swap ? yi : xi;
            yi = swap ? xi : yi;
            xi = ti;
          }
        }
      }
    }
  }
}

// Groups of the marks (group g's in lane g): the top_groups best, as bits.  size: of the keys
// that a mark is the sum of (with a bias they may cancel).  close: were every mark off by `tol`
// of that and smax, a group left out might be ahead of one taken.
template <class K>
__device__ __forceinline__ uint32_t choose_groups(K mark, K size, const RouteArgs& a, float smax, float tol, int lane, bool& close) {
  using U = typename Ordered<K>::U;
  U u = lane < a.groups ? order(mark) : (U)0;
  uint32_t stays = 0;
  for (int i = 0; i < a.top_groups; ++i) {
    const U mu = warp_max(u);
    const int w = __ffs(__ballot_sync(kFull, u == mu && lane < a.groups && !((stays >> lane) & 1u))) - 1;
    stays |= 1u << w;
    if (lane == w) u = 0;
  }
  close = false;
  if (sizeof(K) == 4) {
    const float m = (float)mark, off = tol * (smax + (float)size);
    const bool any = lane < a.groups && m != -INFINITY, taken = (stays >> lane) & 1u;
    close = warp_max(order(any && !taken ? m + off : -INFINITY)) >= __reduce_min_sync(kFull, order(any && taken ? m - off : INFINITY));
  }
  return stays;
}

// Lane j < n has the j-th of a row's experts by fp32 keys, `after` is the next one (or -1):
// the n first of them by fp64 keys.  Sigmoid scores with a bias.
template <int kType>
__device__ __noinline__ int reorder64(const RouteArgs& a, long long row, int mine, int after, int n, int lane) {
  auto key_of = [&](int e) {
    return 1.0 / (1.0 + exp(-(double)load_logit<kType>(a.logits, row * a.E + e))) + (double)a.bias[e];
  };
  const double key = lane < n ? key_of(mine) : 0.0;
  const double key2 = after >= 0 ? key_of(after) : 0.0;
  int rank = 0, rank2 = 0;                       // how many stand before
  for (int i = 0; i < n; ++i) {
    const double o = __shfl_sync(kFull, key, i);
    const int e = __shfl_sync(kFull, mine, i);
    rank += order(o) > order(key) || (order(o) == order(key) && e < mine);
    rank2 += order(o) > order(key2) || (order(o) == order(key2) && e < after);
  }
  if (after >= 0) rank += order(key2) > order(key) || (order(key2) == order(key) && after < mine);
  int got = -1;
  for (int i = 0; i < n; ++i) {
    const int r = __shfl_sync(kFull, rank, i), e = __shfl_sync(kFull, mine, i);
    if (r == lane) got = e;
  }
  if (after >= 0 && rank2 == lane) got = after;
  return lane < n ? got : -1;
}

// The choice from keys of type K: experts lane * V + i are a lane's.  Returns, in lane j <
// k, the j-th expert (or -1).  With K = float, `unsure` is set where two keys that decide
// something are so close that they may stand in the wrong order: closer than tol (smax +
// max(|a|, |b|)), smax the largest score; of groups as choose_groups says.  room: E values of
// this warp.
// Up to eight scores a lane are sorted first, so that a round takes a lane's next instead
// of searching it (T = 16384, E = 256, k = 8 of 4 groups of 8: 63 -> 48 us).
template <int kType, class K, int V>
__device__ __forceinline__ int choose(const RouteArgs& a, long long row, const float (&l)[V], const K (&key)[V],
                                      const RowSum<K>& sums, float smax, float tol, K* room, int lane, bool& unsure) {
  using U = typename Ordered<K>::U;
  constexpr U kOut = Ordered<K>::kOut;
  constexpr bool kCheck = sizeof(K) == 4, kSorted = V <= 8;
  const int E = a.E, k = a.k, e0 = lane * V, per = E / a.groups;
  const bool by_key = a.bias != nullptr;
  // Logits are ordered with + 0, which makes one number of the zeros; a key is no -0, being a
  // sum with a score, nor are marks.
  U u[V];
  int id[V];
  bool close = false;
  // whole lanes in a group, and a power of two of them
  const int lanes = per / V;
  const bool whole = kSorted && per % V == 0 && (lanes & (lanes - 1)) == 0;
  if (a.groups > 1 && !whole) {
    __syncwarp();
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (e0 + i < E) room[e0 + i] = key[i];
    __syncwarp();
    K best = (K)-INFINITY, next = (K)-INFINITY;
    // as many lanes as there are for a group, each with every so many-th expert
    int span = 32 / a.groups;
    span = 1 << (31 - __clz(span));
    const int g = lane / span, off = lane - g * span;
    if (g < a.groups) {
      // started at different places, so that the lanes' reads spread over the banks
      const int n = (per - off + span - 1) / span;
      int at = n > 0 ? g % n : 0;
      for (int i = 0; i < n; ++i) {
        const K v = room[g * per + off + at * span];
        if (order(v) > order(best)) {
          next = best;
          best = v;
        } else if (order(v) > order(next)) {
          next = v;
        }
        if (++at == n) at = 0;
      }
    }
    for (int o = 1; o < span; o <<= 1) {
      const K b2 = __shfl_xor_sync(kFull, best, o), n2 = __shfl_xor_sync(kFull, next, o);
      if (order(b2) > order(best)) {
        next = order(best) > order(n2) ? best : n2;
        best = b2;
      } else {
        next = order(b2) > order(next) ? b2 : next;
      }
    }
    const bool two = a.top2 && next != (K)-INFINITY;
    const K m = two ? best + next : best, size = two ? fabs(best) + fabs(next) : fabs(best);
    const int from = min(lane * span, 31);
    const uint32_t stays =
        choose_groups<K>(__shfl_sync(kFull, m, from), __shfl_sync(kFull, size, from), a, smax, tol, lane, close);
    int grp = e0 / per, grp_end = (grp + 1) * per;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (e0 + i >= grp_end) {
        ++grp;
        grp_end += per;
      }
      u[i] = e0 + i < E && ((stays >> (grp & 31)) & 1u) ? order(by_key ? key[i] : (K)l[i] + (K)0) : kOut;
    }
  } else if (by_key) {                           // -inf, of a logit too, is kOut
#pragma unroll
    for (int i = 0; i < V; ++i) u[i] = order_sum(key[i]);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) u[i] = order((K)l[i] + (K)0);
  }
  uint32_t ids = 0;                              // the sorted ones' places in the lane, four bits each
  if constexpr (kSorted) {
#pragma unroll
    for (int i = 0; i < V; ++i) id[i] = i;
    sort_lane(u, id);
#pragma unroll
    for (int i = 0; i < V; ++i) ids |= (uint32_t)id[i] << (4 * i);
    if (a.groups > 1 && whole) {
      // a lane's two best; without a bias in the order of the logits, their scores then
      U b = u[0], n = V > 1 ? u[V > 1 ? 1 : 0] : kOut;
      for (int o = 1; o < lanes; o <<= 1) {
        const U b2 = __shfl_xor_sync(kFull, b, o), n2 = __shfl_xor_sync(kFull, n, o);
        n = b2 > b ? (b > n2 ? b : n2) : (b2 > n ? b2 : n);
        b = b2 > b ? b2 : b;
      }
      K best, next;
      if (by_key) {
        best = unorder(b);
        next = unorder(n);
      } else {
        best = b == kOut ? (K)-INFINITY : score_of(a, unorder(b), sums);
        next = n == kOut ? (K)-INFINITY : score_of(a, unorder(n), sums);
      }
      const bool two = a.top2 && next != (K)-INFINITY;
      const K m = two ? best + next : best, size = two ? fabs(best) + fabs(next) : fabs(best);
      const int from = (lane * lanes) & 31;
      const uint32_t stays =
          choose_groups<K>(__shfl_sync(kFull, m, from), __shfl_sync(kFull, size, from), a, smax, tol, lane, close);
      if (!((stays >> (lane / lanes)) & 1u)) {
#pragma unroll
        for (int i = 0; i < V; ++i) u[i] = kOut;
      }
    }
  }
  unsure = kCheck && close;
  U best = kOut;
  if constexpr (!kSorted) {
#pragma unroll
    for (int i = 0; i < V; ++i) best = u[i] > best ? u[i] : best;
  }
  // the largest that is left: its key and expert; false: none
  auto take = [&](U& m, int& e) -> bool {
    if constexpr (kSorted) best = u[0];
    m = warp_max(best);
    if (m == kOut) return false;
    const int w = __ffs(__ballot_sync(kFull, best == m)) - 1;
    e = 0;
    if constexpr (kSorted) {
      e = __shfl_sync(kFull, e0 + (int)(ids & 15u), w);
      if (lane == w) {
        ids >>= 4;
#pragma unroll
        for (int i = 0; i + 1 < V; ++i) u[i] = u[i + 1];
        u[V - 1] = kOut;
      }
    } else {
      if (lane == w) {
        bool done = false;
        best = kOut;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          if (!done && u[i] == m) {
            done = true;
            u[i] = kOut;
            e = e0 + i;
          }
          best = u[i] > best ? u[i] : best;
        }
      }
      e = __shfl_sync(kFull, e, w);
    }
    return true;
  };
  // lane j's; of the two behind the chosen (kCheck) in every lane
  int mine = -1, found = 0, after = -1, third = -1;
  U mykey = kOut, afterkey = kOut, thirdkey = kOut;
  {
    U m;
    int e;
    while (found < k && take(m, e)) {
      if (lane == found) {
        mine = e;
        mykey = m;
      }
      ++found;
    }
    if (kCheck && by_key && found == k) {
#pragma unroll 1
      while (found < k + 2 && take(m, e)) {
        if (found == k) {
          after = e;
          afterkey = m;
        }
        third = e;
        thirdkey = m;
        ++found;
      }
    }
  }
  if constexpr (kCheck) {
    if (by_key && found > 1 && !unsure) {
      // lane j against the next one, the last against the first that was left out
      const int chosen = min(k, found), pairs = min(k, found - 1);
      int ne = __shfl_down_sync(kFull, mine, 1);
      U nk = __shfl_down_sync(kFull, mykey, 1);
      if (lane == k - 1) {
        ne = after;
        nk = afterkey;
      }
      const float x = unorder(mykey), y = unorder(nk);
      const bool close2 = lane < pairs && x - y <= tol * (smax + fmaxf(fabsf(x), fabsf(y)));
      if (__any_sync(kFull, close2)) {
        // equal numbers in give equal keys: the index decides
        auto equal = [&](int p, int q) {
          return load_logit<kType>(a.logits, row * E + p) == load_logit<kType>(a.logits, row * E + q) && a.bias[p] == a.bias[q];
        };
        const bool same = close2 && equal(mine, ne);
        const float last = unorder(__shfl_sync(kFull, mykey, chosen - 1));
        auto near_last = [&](U key) {
          const float o = unorder(key);
          return last - o <= tol * (smax + fmaxf(fabsf(last), fabsf(o)));
        };
        if (__any_sync(kFull, close2 && !same)) {
          // Where the second left out is clearly behind the last chosen, the order among the
          // chosen and the first left out is all there is to find.
          if (!a.sigmoid || (found > k + 1 && near_last(thirdkey))) unsure = true;
          else mine = reorder64<kType>(a, row, mine, found > k ? after : -1, chosen, lane);
        } else if (found > k + 1 && ((__ballot_sync(kFull, same) >> (k - 1)) & 1u)) {
          // The first left out equals the last chosen: what comes behind its equals may have
          // to stand before them.
          while (near_last(thirdkey)) {
            if (!equal(after, third)) {
              unsure = true;
              break;
            }
            if (!take(thirdkey, third)) break;
          }
        }
      }
    }
  }
  return lane < k ? mine : -1;
}

// A lane's V scores of a row, -inf behind the last.
template <int kType, int V>
__device__ __forceinline__ void load_row(const RouteArgs& a, long long row, int lane, float (&l)[V]) {
  const int E = a.E, e0 = lane * V;
  const long long base = row * E + e0;
  bool loaded = false;
  if constexpr (V % 4 == 0) {
    if (E % 4 == 0) {                          // rows stay aligned to four elements
      loaded = true;
#pragma unroll
      for (int i = 0; i < V; i += 4) {
        if (e0 + i < E) {
          if constexpr (kType == MHC_DTYPE_FP32) {
            const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(a.logits) + base + i);
            l[i] = v.x;
            l[i + 1] = v.y;
            l[i + 2] = v.z;
            l[i + 3] = v.w;
          } else {
            const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.logits) + base + i);
            constexpr bool f16 = kType == MHC_DTYPE_FP16;
            const float2 p = XType<f16>::to_f2(*reinterpret_cast<const typename XType<f16>::T2*>(&v.x));
            const float2 q = XType<f16>::to_f2(*reinterpret_cast<const typename XType<f16>::T2*>(&v.y));
            l[i] = p.x;
            l[i + 1] = p.y;
            l[i + 2] = q.x;
            l[i + 3] = q.y;
          }
        } else {
          l[i] = l[i + 1] = l[i + 2] = l[i + 3] = -INFINITY;
        }
      }
    }
  }
  if (!loaded) {
#pragma unroll
    for (int i = 0; i < V; ++i) l[i] = e0 + i < E ? load_logit<kType>(a.logits, base + i) : -INFINITY;
  }
}

// The choice once more with keys in fp64, for rows where fp32 left two keys too close: two to
// ten of ten thousand ordinary rows with groups, or of softmax scores with a bias.
template <int kType, int V>
__device__ __noinline__ int choose64(const RouteArgs& a, long long row, float top, double* room, int lane) {
  const int e0 = lane * V;
  float l[V];
  load_row<kType, V>(a, row, lane, l);
  double key[V];
  RowSum<double> r = {top, 0.0};
#pragma unroll
  for (int i = 0; i < V; ++i) {
    key[i] = l[i] == -INFINITY ? 0.0 : a.sigmoid ? 1.0 / (1.0 + exp(-(double)l[i])) : exp((double)l[i] - (double)top);
    r.sum += key[i];
  }
  r.sum = warp_sum(r.sum);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if (!a.sigmoid) key[i] /= r.sum;
    if (a.bias && e0 + i < a.E) key[i] += (double)a.bias[e0 + i];
    if (l[i] == -INFINITY) key[i] = -INFINITY;
  }
  bool unsure = false;
  return choose<kType, double, V>(a, row, l, key, r, 0.0f, 0.0f, room, lane, unsure);
}

// Warps of a block, and blocks of an SM.
__host__ __device__ constexpr int route_warps(int V) { return V <= 8 ? 8 : 4; }
__host__ __device__ constexpr int route_blocks(int V) { return V <= 4 ? 4 : V <= 8 ? 3 : V <= 16 ? 4 : 2; }

// V: consecutive scores of a lane.  A block's warps take its rows in turn as they come free:
// a row whose keys are formed again takes several others' time, and the code for it comes
// into an SM for a row or two.
template <int kType, int V>
__global__ void __launch_bounds__(route_warps(V) * 32, route_blocks(V)) route_kernel(const RouteArgs a) {
  extern __shared__ double route_keys[];
  __shared__ unsigned taken;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int E = a.E, k = a.k, e0 = lane * V;
  double* keys64 = route_keys + (size_t)warp * E;
  float bias[V];
#pragma unroll
  for (int i = 0; i < V; ++i) bias[i] = a.bias && e0 + i < E ? a.bias[e0 + i] : 0.0f;
  const long long first = a.T * blockIdx.x / gridDim.x, last = a.T * (blockIdx.x + 1) / gridDim.x;
  if (threadIdx.x == 0) taken = 0;
  __syncthreads();
  auto draw = [&]() -> long long {
    const unsigned n = lane == 0 ? atomicAdd(&taken, 1u) : 0u;
    return first + __shfl_sync(kFull, n, 0);
  };
  for (long long row = draw(); row < last; row = draw()) {
    float l[V];
    load_row<kType, V>(a, row, lane, l);
    // Scores; softmax: top and sum of the row.
    float top = 0.0f;
    if (!a.sigmoid) {
      uint32_t topu = Ordered<float>::kOut;
#pragma unroll
      for (int i = 0; i < V; ++i) topu = max(topu, order(l[i]));
      topu = warp_max(topu);
      if (topu != Ordered<float>::kOut) top = unorder(topu);
    }
    const bool scores = a.bias != nullptr || a.groups > 1;
    float smax = 1.0f;
    RowSum<float> r = {top, 0.0f};
    float key[V];
    if (a.sigmoid) {
      if (scores) {
#pragma unroll
        for (int i = 0; i < V; ++i) key[i] = score_of(a, l[i], r);
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        key[i] = l[i] == -INFINITY ? 0.0f : expf(l[i] - top);
        r.sum += key[i];
      }
      r.sum = warp_sum(r.sum);
      if (scores) {
        smax = 1.0f / r.sum;
#pragma unroll
        for (int i = 0; i < V; ++i) key[i] = key[i] * smax;
      }
    }
    if (scores) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        key[i] += bias[i];
        if (l[i] == -INFINITY) key[i] = -INFINITY;
      }
    }
    // How far two keys may be off against one another, of the largest score and their own
    // size.  Sigmoid: fast exponential (2 + 1.2 |l| units of 2^-23 of itself, which counts s
    // (1 - s), at most 0.8 of 2^-23 in all), the sum and the division 2^-22 each: 2^-21.
    // Softmax: exponential and rounding of l - top 2^-22 of the largest, reciprocal and
    // division 2^-22, its sum V + 5 roundings, the same for all.  A key with a bias 2^-24 of
    // itself.  Twice that for two keys, and as much again.
    const float tol = a.sigmoid ? 0x1p-19f : (V + 24) * 0x1p-23f;
    bool unsure = false;
    int mine = choose<kType, float, V>(a, row, l, key, r, smax, tol, reinterpret_cast<float*>(keys64), lane, unsure);
    if (unsure) mine = choose64<kType, V>(a, row, top, keys64, lane);
    const float myl = mine >= 0 ? load_logit<kType>(a.logits, row * E + mine) : -INFINITY;
    const float sum = r.sum;
    // Weights: lane j has slot j.
    float w;
    if (a.renorm) {
      float mx = myl;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o));
      if (mx == -INFINITY) mx = 0.0f;
      float s;
      if (a.sigmoid) {
        // all far below 0: the common factor e^mx is left out
        const float c = fminf(mx, 0.0f);
        s = mx < 0.0f ? expf(myl - c) / (1.0f + expf(myl)) : sigmoid32(myl);
      } else {
        s = expf(myl - mx);
      }
      if (mine < 0) s = 0.0f;
      const float total = warp_sum(s);
      w = total == 0.0f ? 0.0f : s / total;
      if (!a.sigmoid && sum != sum) w = NAN;     // a NaN or infinity among the scores, chosen or not
    } else {
      w = a.sigmoid ? sigmoid32(myl) : expf(myl - top) / sum;
    }
    if (lane < k) {
      a.experts[row * k + lane] = mine;
      a.weights[row * k + lane] = mine < 0 ? 0.0f : w * a.scale;
    }
    __syncwarp();
  }
}

struct RouteBwdArgs {
  const void* logits;
  const int* experts;
  const float* grad_weights;
  void* grad_logits;
  long long T;
  int E, k, sigmoid, renorm;
  float scale;
};

// A warp per row; lane j < k has slot j.
template <int kType>
__global__ void __launch_bounds__(kRouteWarps * 32) route_backward_kernel(const RouteBwdArgs a) {
  extern __shared__ float route_row[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int E = a.E, k = a.k;
  float* g = route_row + (size_t)warp * E;
  for (long long row = (long long)blockIdx.x * kRouteWarps + warp; row < a.T; row += (long long)gridDim.x * kRouteWarps) {
    int e = lane < k ? a.experts[row * k + lane] : -1;
    if (e >= E) e = -1;
    const float d = e >= 0 ? a.grad_weights[row * k + lane] * a.scale : 0.0f;
    const float l = e >= 0 ? load_logit<kType>(a.logits, row * E + e) : -INFINITY;
    float v, dot = 0.0f, top = 0.0f, sum = 1.0f;
    const bool dense = !a.sigmoid && !a.renorm;
    if (a.renorm) {
      float mx = l;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o));
      if (mx == -INFINITY) mx = 0.0f;
      float s, h = 1.0f;
      if (a.sigmoid) {
        s = mx < 0.0f ? expf(l - mx) / (1.0f + expf(l)) : sigmoid32(l);
        h = 1.0f / (1.0f + expf(l));             // 1 - sigmoid, without its cancellation
      } else {
        s = expf(l - mx);
      }
      if (e < 0) s = 0.0f;
      const float total = warp_sum(s);
      const float w = total == 0.0f ? 0.0f : s / total;
      dot = warp_sum(d * w);
      v = w * (d - dot) * h;
    } else if (a.sigmoid) {
      const float s = sigmoid32(l);
      v = d * s * (1.0f / (1.0f + expf(l)));
    } else {
      top = -INFINITY;
      bool bad = false;
      for (int i = lane; i < E; i += 32) {
        const float x = load_logit<kType>(a.logits, row * E + i);
        g[i] = x;
        bad |= x != x;
        top = fmaxf(top, x);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
      if (top == -INFINITY) top = 0.0f;
      sum = 0.0f;
      for (int i = lane; i < E; i += 32) {
        const float s = g[i] == -INFINITY ? 0.0f : expf(g[i] - top);
        g[i] = s;
        sum += s;
      }
      sum = warp_sum(sum);
      if (__any_sync(kFull, bad)) sum = NAN;
      const float s = e >= 0 && sum != 0.0f ? expf(l - top) / sum : 0.0f;
      v = d * s;
      dot = warp_sum(v);
    }
    if (e < 0) v = 0.0f;
    if (dense) {
      const float f = sum == 0.0f ? 0.0f : dot / sum;
      __syncwarp();
      for (int i = lane; i < E; i += 32) g[i] = -g[i] * f;
    } else {
      for (int i = lane; i < E; i += 32) g[i] = 0.0f;
    }
    __syncwarp();
    // an expert given twice: its first lane adds the others' parts, in their order
    const uint32_t same = __match_any_sync(kFull, e);
    const bool first = e >= 0 && (__ffs(same) - 1) == lane;
    if (__any_sync(kFull, e >= 0 && !first)) {
      float add = 0.0f;
      for (int j = 0; j < k; ++j) {
        const float o = __shfl_sync(kFull, v, j);
        if ((same >> j) & 1u) add += o;
      }
      v = add;
    }
    if (first) g[e] += v;
    __syncwarp();
    if (kType == MHC_DTYPE_FP32) {
      float* out = static_cast<float*>(a.grad_logits) + row * E;
      if (E % 4 == 0) {
        for (int i = lane * 4; i < E; i += 128)
          *reinterpret_cast<float4*>(out + i) = *reinterpret_cast<const float4*>(g + i);
      } else {
        for (int i = lane; i < E; i += 32) out[i] = g[i];
      }
    } else {
      uint16_t* out = static_cast<uint16_t*>(a.grad_logits) + row * E;
      constexpr bool f16 = kType == MHC_DTYPE_FP16;
      if (E % 2 == 0) {
        for (int i = lane * 2; i < E; i += 64) {
          const typename XType<f16>::T2 p = XType<f16>::from_f2(g[i], g[i + 1]);
          *reinterpret_cast<uint32_t*>(out + i) = *reinterpret_cast<const uint32_t*>(&p);
        }
      } else {
        for (int i = lane; i < E; i += 32) {
          const typename XType<f16>::T2 p = XType<f16>::from_f2(g[i], 0.0f);
          out[i] = (uint16_t)*reinterpret_cast<const uint32_t*>(&p);
        }
      }
    }
    __syncwarp();
  }
}

// ------------------------------------------------------------------ the plan

constexpr int kPlanThreads = 1024, kPlanWarps = 32;

struct PlanArgs {
  const int* experts;
  PlanView p;
  int slots, E, chunk;         // slots of a block
};

// Shared memory of the plan's kernels: the warps' counters.
__host__ __device__ inline size_t plan_smem(int E) { return (size_t)kPlanWarps * E * 2; }

// f(slot, its expert or -1) for a warp's slots of the block's [first, last), 32 at a time,
// eight loads in flight.
template <class F>
__device__ __forceinline__ void plan_slots(const PlanArgs& a, int first, int last, int warp, int lane, F f) {
  const int per = (((last - first) + kPlanWarps - 1) / kPlanWarps + 31) & ~31;
  const int b = first + warp * per, n = min(b + per, last);
  for (int i = b; i < n; i += 256) {
    int e[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int at = i + 32 * u + lane;
      e[u] = at < n ? a.experts[at] : -1;
    }
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (i + 32 * u < n) f(i + 32 * u + lane, e[u] < 0 || e[u] >= a.E ? -1 : e[u], n);
  }
}

// Counts of each expert among each warp's slots of this block.
__device__ __forceinline__ void plan_count(const PlanArgs& a, uint16_t* hist, int first, int last, int warp, int lane) {
  const int E = a.E;
  for (int i = threadIdx.x; i < kPlanWarps * E; i += kPlanThreads) hist[i] = 0;
  __syncthreads();
  plan_slots(a, first, last, warp, lane, [&](int, int e, int) {
    const uint32_t same = __match_any_sync(kFull, e);
    if (e >= 0 && (__ffs(same) - 1) == lane) hist[warp * E + e] += (uint16_t)__popc(same);
    __syncwarp();
  });
  __syncthreads();
}
// The counters as what lies before each warp's slots; returns expert e's count.
__device__ __forceinline__ int plan_prefix(uint16_t* hist, int E, int e) {
  int c[kPlanWarps], run = 0;
#pragma unroll
  for (int w = 0; w < kPlanWarps; ++w) c[w] = hist[w * E + e];
#pragma unroll
  for (int w = 0; w < kPlanWarps; ++w) {
    hist[w * E + e] = (uint16_t)run;
    run += c[w];
  }
  return run;
}
// Exclusive sum over the block; every thread gets it, *total the whole.
__device__ __forceinline__ int plan_scan(int v, int* sums, int* total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kFull, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int s = sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(kFull, s, o);
      if (lane >= o) s += y;
    }
    sums[lane] = s;
  }
  __syncthreads();
  const int before = warp ? sums[warp - 1] : 0;
  *total = sums[31];
  __syncthreads();
  return before + x - v;
}
// Counts -> starts, padding rows, tiles.  Thread e has expert e's count.
__device__ __forceinline__ void plan_finish(const PlanArgs& a, int count, int* sums, int* tile_at, int* start_at, int* count_at) {
  const int e = threadIdx.x, E = a.E, width = a.p.width;
  int rows, tiles;
  const int padded = (count + kPlanPad - 1) & ~(kPlanPad - 1);
  const int start = plan_scan(padded, sums, &rows);
  const int nt = (count + width - 1) / width;
  const int t0 = plan_scan(nt, sums, &tiles);
  if (e < E) {
    a.p.counts[e] = count;
    a.p.starts[e] = start;
    for (int i = count; i < padded; ++i) a.p.rows[start + i] = -1;
  }
  tile_at[e] = t0;
  start_at[e] = start;
  count_at[e] = count;
  if (e == 0) {
    a.p.starts[E] = rows;
    a.p.head[1] = rows;
    a.p.head[2] = tiles;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < tiles; i += kPlanThreads) {
    int lo = 0, hi = E - 1;                      // the last expert whose first tile is at most i
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (tile_at[mid] <= i) lo = mid;
      else hi = mid - 1;
    }
    // tiles of one expert differ by 32 rows at most
    const int units = (count_at[lo] + 31) >> 5, n = (count_at[lo] + width - 1) / width, base = units / n, wide = units - base * n;
    const int j = i - tile_at[lo], band = j / kPlanBand * kPlanBand, in_band = min(kPlanBand, n - band);
    const int first = 32 * (band * base + min(band, wide)), w = min(max(wide - band, 0), in_band);
    a.p.table[2 * i] = make_int4(lo, tile_at[lo] + band, in_band, start_at[lo] + first);
    a.p.table[2 * i + 1] = make_int4(min(32 * (in_band * base + w), count_at[lo] - first), 32 * base, w, 0);
  }
}
// Rows of the block's slots: base[e] + what lies before them.
__device__ __forceinline__ void plan_place(const PlanArgs& a, uint16_t* hist, const int* base, int first, int last, int warp,
                                           int lane) {
  const int E = a.E;
  plan_slots(a, first, last, warp, lane, [&](int at, int e, int n) {
    const uint32_t same = __match_any_sync(kFull, e);
    int row = -1;
    if (e >= 0) row = base[e] + hist[warp * E + e] + __popc(same & ((1u << lane) - 1u));
    __syncwarp();
    if (e >= 0 && (__ffs(same) - 1) == lane) hist[warp * E + e] += (uint16_t)__popc(same);
    __syncwarp();
    if (at < n) {
      a.p.places[at] = row;
      if (row >= 0) a.p.rows[row] = at;
    }
  });
}

// All in one block: about 5 us for the slots of a few tokens.
__global__ void __launch_bounds__(kPlanThreads) plan_alone_kernel(const PlanArgs a) {
  extern __shared__ uint16_t plan_hist[];
  __shared__ int sums[32], tile_at[kMostExperts], start_at[kMostExperts], count_at[kMostExperts];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  plan_count(a, plan_hist, 0, a.slots, warp, lane);
  const int count = (int)threadIdx.x < a.E ? plan_prefix(plan_hist, a.E, threadIdx.x) : 0;
  plan_finish(a, count, sums, tile_at, start_at, count_at);
  __syncthreads();
  plan_place(a, plan_hist, start_at, 0, a.slots, warp, lane);
}
// Many slots: counts of each block's, then the sums over blocks, then the rows.  Each kernel
// starts beside the one before; what the placing one counts again does not wait for it.
// Bound by their starts and the latency of dependent loads: 32768 slots take 8.9 us (18.7 one
// after the other with 4096 slots a block), 8192 take 8.5 (20 in one block alone).
__global__ void __launch_bounds__(kPlanThreads) plan_count_kernel(const PlanArgs a) {
  extern __shared__ uint16_t plan_hist[];
  pdl_trigger();
  const int first = blockIdx.x * a.chunk, last = min(first + a.chunk, a.slots);
  plan_count(a, plan_hist, first, last, threadIdx.x >> 5, threadIdx.x & 31);
  if ((int)threadIdx.x < a.E) a.p.scratch[(size_t)blockIdx.x * a.E + threadIdx.x] = plan_prefix(plan_hist, a.E, threadIdx.x);
}
__global__ void __launch_bounds__(kPlanThreads) plan_sum_kernel(const PlanArgs a, const int blocks) {
  __shared__ int sums[32], tile_at[kMostExperts], start_at[kMostExperts], count_at[kMostExperts];
  pdl_trigger();
  pdl_wait();
  int count = 0;
  if ((int)threadIdx.x < a.E) {
    for (int b0 = 0; b0 < blocks; b0 += 16) {
      int c[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) c[i] = b0 + i < blocks ? a.p.scratch[(size_t)(b0 + i) * a.E + threadIdx.x] : 0;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        if (b0 + i < blocks) a.p.scratch[(size_t)(b0 + i) * a.E + threadIdx.x] = count;
        count += c[i];
      }
    }
  }
  plan_finish(a, count, sums, tile_at, start_at, count_at);
}
__global__ void __launch_bounds__(kPlanThreads) plan_place_kernel(const PlanArgs a) {
  extern __shared__ uint16_t plan_hist[];
  __shared__ int base[kMostExperts];
  const int first = blockIdx.x * a.chunk, last = min(first + a.chunk, a.slots);
  plan_count(a, plan_hist, first, last, threadIdx.x >> 5, threadIdx.x & 31);
  if ((int)threadIdx.x < a.E) plan_prefix(plan_hist, a.E, threadIdx.x);
  pdl_wait();
  if ((int)threadIdx.x < a.E) {
    base[threadIdx.x] = a.p.starts[threadIdx.x] + a.p.scratch[(size_t)blockIdx.x * a.E + threadIdx.x];
  }
  __syncthreads();
  plan_place(a, plan_hist, base, first, last, threadIdx.x >> 5, threadIdx.x & 31);
}

// --------------------------------------------------------------------- host

mhc_status_t check_route(int64_t T, int64_t E, int64_t k) {
  if (T < 0 || T > (int64_t(1) << 20)) return fail(MHC_ERR_PARAM_INVALID, "T must be in [0, 2^20] (got %lld)", (long long)T);
  if (E < 1 || E > kMostExperts) return fail(MHC_ERR_PARAM_INVALID, "E must be in [1, 1024] (got %lld)", (long long)E);
  if (k < 1 || k > kMostChoices || k > E)
    return fail(MHC_ERR_PARAM_INVALID, "k must be in [1, min(E, 32)] (got %lld)", (long long)k);
  if (T * k > (int64_t(1) << 22)) return fail(MHC_ERR_PARAM_INVALID, "T k must be at most 2^22 (got %lld)", (long long)(T * k));
  return MHC_OK;
}
mhc_status_t check_kind(int32_t dtype, int32_t score, int32_t renorm, float scale) {
  if (dtype != MHC_DTYPE_BF16 && dtype != MHC_DTYPE_FP16 && dtype != MHC_DTYPE_FP32)
    return fail(MHC_ERR_PARAM_INVALID, "dtype must be MHC_DTYPE_BF16, _FP16 or _FP32 (got %d)", (int)dtype);
  if (score != MHC_SCORE_SOFTMAX && score != MHC_SCORE_SIGMOID)
    return fail(MHC_ERR_PARAM_INVALID, "score must be MHC_SCORE_SOFTMAX or MHC_SCORE_SIGMOID (got %d)", (int)score);
  if (renorm != 0 && renorm != 1) return fail(MHC_ERR_PARAM_INVALID, "renormalise must be 0 or 1");
  if (!isfinite(scale)) return fail(MHC_ERR_PARAM_INVALID, "scale must be finite");
  return MHC_OK;
}
mhc_status_t route_device(int* sms) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return fail(MHC_ERR_RUNTIME, "no CUDA device");
  const DeviceInfo di = device_info(dev);
  if (!di.ok) return fail(MHC_ERR_RUNTIME, "device %d is not an sm_103 GPU", dev);
  *sms = di.sms;
  return MHC_OK;
}
unsigned row_blocks(int64_t T, int sms) {
  const int64_t b = (T + kRouteWarps - 1) / kRouteWarps, most = (int64_t)sms * 16;
  return (unsigned)(b < most ? b : most);
}
size_t elem_bytes(int32_t dtype) { return dtype == MHC_DTYPE_FP32 ? 4 : 2; }
// Vector loads of four logits and stores of four fp32 or two 16-bit gradients.
size_t logits_align(int32_t dtype, int64_t E) { return E % 4 == 0 ? 4 * elem_bytes(dtype) : E % 2 == 0 ? 2 * elem_bytes(dtype) : elem_bytes(dtype); }

// Scores of a lane: as few as hold the row (E = 160: five in 32 lanes, 17 us for 16384 rows,
// with eight in 20 22), but first of all so that a group is whole lanes (8 groups: 23 and 39).
int route_width(int E, int groups) {
  constexpr int kWidths[] = {1, 2, 3, 4, 5, 6, 8, 16, 32};
  int least = 0;
  for (int v : kWidths) {
    if (32 * v < E) continue;
    if (!least) least = v;
    const int per = E / groups, lanes = per / v;
    if (groups > 1 && v <= 8 && per % v == 0 && (lanes & (lanes - 1)) == 0) return v;
  }
  return least;
}

template <int kType>
cudaError_t launch_route(const RouteArgs& a, int sms, cudaStream_t s) {
  // where no key is formed again and no group is marked nothing is kept in shared memory
  auto run = [&](auto* k, int v) {
    const int warps = route_warps(v);
    const int64_t rows = (a.T + warps - 1) / warps, most = (int64_t)sms * route_blocks(v);
    const size_t smem = a.bias || a.groups > 1 ? (size_t)warps * a.E * 8 : 0;
    k<<<(unsigned)(rows < most ? rows : most), warps * 32, smem, s>>>(a);
  };
  switch (route_width(a.E, a.groups)) {
    case 1: run(route_kernel<kType, 1>, 1); break;
    case 2: run(route_kernel<kType, 2>, 2); break;
    case 3: run(route_kernel<kType, 3>, 3); break;
    case 4: run(route_kernel<kType, 4>, 4); break;
    case 5: run(route_kernel<kType, 5>, 5); break;
    case 6: run(route_kernel<kType, 6>, 6); break;
    case 8: run(route_kernel<kType, 8>, 8); break;
    case 16: run(route_kernel<kType, 16>, 16); break;
    default: run(route_kernel<kType, 32>, 32);
  }
  return cudaGetLastError();
}

}  // namespace
}  // namespace mhc

using namespace mhc;

extern "C" {

mhc_status_t mhc_route_run(const mhc_route_args* a, void* stream) {
  clear_error();
  if (!a) return fail(MHC_ERR_NULLPTR, "args must be non-NULL");
  mhc_status_t st = check_route(a->T, a->E, a->k);
  if (st == MHC_OK) st = check_kind(a->dtype, a->score, a->renormalise, a->scale);
  if (st != MHC_OK) return st;
  if (a->groups < 1 || a->groups > kMostGroups || a->E % a->groups != 0)
    return fail(MHC_ERR_PARAM_INVALID, "groups must divide E and be in [1, 32] (got %d)", (int)a->groups);
  if (a->top_groups < 1 || a->top_groups > a->groups)
    return fail(MHC_ERR_PARAM_INVALID, "top_groups must be in [1, groups] (got %d)", (int)a->top_groups);
  if (a->k > a->E / a->groups * a->top_groups)
    return fail(MHC_ERR_PARAM_INVALID, "k must be at most the experts of top_groups groups (got %lld)", (long long)a->k);
  if (a->group_score != MHC_GROUP_MAX && a->group_score != MHC_GROUP_TOP2)
    return fail(MHC_ERR_PARAM_INVALID, "group_score must be MHC_GROUP_MAX or MHC_GROUP_TOP2 (got %d)", (int)a->group_score);
  if (a->T == 0) return MHC_OK;
  if (!a->logits || !a->experts || !a->weights) return fail(MHC_ERR_NULLPTR, "logits, experts and weights are required");
  if (!aligned(a->logits, logits_align(a->dtype, a->E)) || !aligned(a->bias, 4) || !aligned(a->experts, 4) || !aligned(a->weights, 4))
    return fail(MHC_ERR_PARAM_INVALID, "tensors must be aligned to their elements, logits to the largest of one, two and four elements that divides a row");
  const size_t lb = (size_t)a->T * a->E * elem_bytes(a->dtype), kb = (size_t)a->T * a->k * 4;
  if ((st = check_apart({{"experts", a->experts, kb}, {"weights", a->weights, kb}},
                        {{"logits", a->logits, lb}, {"bias", a->bias, (size_t)a->E * 4}})) != MHC_OK)
    return st;
  int sms = 0;
  if ((st = route_device(&sms)) != MHC_OK) return st;
  RouteArgs r = {a->logits, a->bias, a->experts, a->weights, a->T, (int)a->E, (int)a->k, a->score == MHC_SCORE_SIGMOID,
                 a->groups, a->top_groups, a->group_score == MHC_GROUP_TOP2, a->renormalise, a->scale};
  if (r.top_groups == r.groups) r.groups = r.top_groups = 1;             // every group stays
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = a->dtype == MHC_DTYPE_FP32   ? launch_route<MHC_DTYPE_FP32>(r, sms, s)
                        : a->dtype == MHC_DTYPE_BF16 ? launch_route<MHC_DTYPE_BF16>(r, sms, s)
                                                     : launch_route<MHC_DTYPE_FP16>(r, sms, s);
  if (e != cudaSuccess) return fail(MHC_ERR_RUNTIME, "routing launch failed: %s", cudaGetErrorString(e));
  return MHC_OK;
}

mhc_status_t mhc_route_backward_run(const mhc_route_bwd_args* a, void* stream) {
  clear_error();
  if (!a) return fail(MHC_ERR_NULLPTR, "args must be non-NULL");
  mhc_status_t st = check_route(a->T, a->E, a->k);
  if (st == MHC_OK) st = check_kind(a->dtype, a->score, a->renormalise, a->scale);
  if (st != MHC_OK || a->T == 0) return st;
  if (!a->logits || !a->experts || !a->grad_weights || !a->grad_logits)
    return fail(MHC_ERR_NULLPTR, "logits, experts, grad_weights and grad_logits are required");
  if (!aligned(a->logits, elem_bytes(a->dtype)) || !aligned(a->grad_logits, logits_align(a->dtype, a->E)) || !aligned(a->experts, 4) ||
      !aligned(a->grad_weights, 4))
    return fail(MHC_ERR_PARAM_INVALID, "tensors must be aligned to their elements, grad_logits to the largest of one, two and four elements that divides a row");
  const size_t lb = (size_t)a->T * a->E * elem_bytes(a->dtype), kb = (size_t)a->T * a->k * 4;
  if ((st = check_apart({{"grad_logits", a->grad_logits, lb}},
                        {{"logits", a->logits, lb}, {"experts", a->experts, kb}, {"grad_weights", a->grad_weights, kb}})) != MHC_OK)
    return st;
  int sms = 0;
  if ((st = route_device(&sms)) != MHC_OK) return st;
  const RouteBwdArgs r = {a->logits, a->experts, a->grad_weights, a->grad_logits, a->T, (int)a->E, (int)a->k,
                          a->score == MHC_SCORE_SIGMOID, a->renormalise, a->scale};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const unsigned grid = row_blocks(a->T, sms);
  const size_t smem = (size_t)kRouteWarps * ((a->E + 3) & ~int64_t(3)) * 4;
  if (a->dtype == MHC_DTYPE_FP32) route_backward_kernel<MHC_DTYPE_FP32><<<grid, kRouteWarps * 32, smem, s>>>(r);
  else if (a->dtype == MHC_DTYPE_BF16) route_backward_kernel<MHC_DTYPE_BF16><<<grid, kRouteWarps * 32, smem, s>>>(r);
  else route_backward_kernel<MHC_DTYPE_FP16><<<grid, kRouteWarps * 32, smem, s>>>(r);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(MHC_ERR_RUNTIME, "routing backward launch failed: %s", cudaGetErrorString(e));
  return MHC_OK;
}

mhc_status_t mhc_expert_plan_size(int64_t T, int64_t k, int64_t E, size_t* bytes) {
  clear_error();
  if (!bytes) return fail(MHC_ERR_NULLPTR, "bytes must be non-NULL");
  const mhc_status_t st = check_route(T, E, k);
  if (st != MHC_OK) return st;
  *bytes = (size_t)plan_layout(T, k, E).total * 4;
  return MHC_OK;
}

mhc_status_t mhc_expert_plan_rows(int64_t T, int64_t k, int64_t E, int64_t* rows) {
  clear_error();
  if (!rows) return fail(MHC_ERR_NULLPTR, "rows must be non-NULL");
  const mhc_status_t st = check_route(T, E, k);
  if (st != MHC_OK) return st;
  *rows = plan_layout(T, k, E).cap_rows;
  return MHC_OK;
}

mhc_status_t mhc_expert_plan_run(int64_t T, int64_t k, int64_t E, const int32_t* experts, void* plan, size_t plan_bytes,
                                 void* stream) {
  clear_error();
  mhc_status_t st = check_route(T, E, k);
  if (st != MHC_OK) return st;
  if (!plan || (T && !experts)) return fail(MHC_ERR_NULLPTR, "experts and plan are required");
  if (!aligned(experts, 4) || !aligned(plan, 256))
    return fail(MHC_ERR_PARAM_INVALID, "experts must be 4-byte and the plan 256-byte aligned");
  const PlanLayout l = plan_layout(T, k, E);
  if (plan_bytes < (size_t)l.total * 4)
    return fail(MHC_ERR_PARAM_INVALID, "plan too small: %zu bytes given, %zu needed", plan_bytes, (size_t)l.total * 4);
  if ((st = check_apart({{"plan", plan, (size_t)l.total * 4}}, {{"experts", experts, (size_t)l.slots * 4}})) != MHC_OK) return st;
  int sms = 0;
  if ((st = route_device(&sms)) != MHC_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (T == 0) {
    const cudaError_t z = cudaMemsetAsync(plan, 0, (size_t)l.total * 4, s);
    return z == cudaSuccess ? MHC_OK : fail(MHC_ERR_RUNTIME, "clearing the plan failed: %s", cudaGetErrorString(z));
  }
  PlanArgs a = {experts, plan_view(l, E, plan), (int)l.slots, (int)E, (int)plan_chunk(l.slots)};
  const size_t smem = plan_smem((int)E);
  cudaError_t e = cudaSuccess;
  if (smem > 32 * 1024) {                        // beside the static arrays more than a kernel has by default
    for (const void* f : {(const void*)plan_alone_kernel, (const void*)plan_count_kernel, (const void*)plan_place_kernel})
      if (e == cudaSuccess) e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)plan_smem(kMostExperts));
    if (e != cudaSuccess) return fail(MHC_ERR_RUNTIME, "plan kernels: %s", cudaGetErrorString(e));
  }
  if (l.slots <= kPlanAlone) {
    plan_alone_kernel<<<1, kPlanThreads, smem, s>>>(a);
  } else {
    const int blocks = (int)((l.slots + a.chunk - 1) / a.chunk);
    plan_count_kernel<<<blocks, kPlanThreads, smem, s>>>(a);
    e = cudaGetLastError();
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(kPlanThreads);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, plan_sum_kernel, a, blocks);
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.dynamicSmemBytes = smem;
    if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, plan_place_kernel, a);
  }
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return fail(MHC_ERR_RUNTIME, "plan launch failed: %s", cudaGetErrorString(e));
  return MHC_OK;
}

}  // extern "C"
