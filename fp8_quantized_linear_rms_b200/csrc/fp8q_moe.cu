// fp8q_moe.cu -- routing to experts and what surrounds their products: the
// router (scores, selection, weights), the plan that orders (token, expert)
// pairs by expert, the weighted sum of the experts' rows, and the whole pass.
#include <cuda_bf16.h>

#include <atomic>

#include "fp8q_common.cuh"
#include "fp8q_fp4_math.cuh"
#include "fp8q_sm100.cuh"

namespace fp8q {
namespace {

constexpr int kMaxExperts = 512;
constexpr int kMaxTopk = 32;
constexpr unsigned kAll = 0xFFFFFFFFu;

// ------------------------------------------------------------------- router
struct RouteParams {
  const void* logits;        // fp32 or bf16 [T, E], leading dimension ld
  int64_t T, ld;
  int E, bf16, vec, vec_bias, sigmoid;  // vec: rows, the biases, begin at 16-byte boundaries
  const float* bias;         // [E] or null
  int groups, topg, topk, renorm;
  float scale;
  float* w;                  // [T, topk]
  int* ids;                  // [T, topk]
};

// A NaN counts as -inf (masked); -0 as 0, so that keys are equal where values are.
__device__ __forceinline__ float route_logit(const RouteParams& p, int64_t t, int e) {
  const int64_t i = t * p.ld + e;
  const float v = p.bf16 ? __bfloat162float(__ldg(static_cast<const __nv_bfloat16*>(p.logits) + i))
                         : __ldg(static_cast<const float*>(p.logits) + i);
  return fmaxf(v, -INFINITY) + 0.0f;
}

// Bounds of what the errors of the keys' fp32 scores make of the difference of
// two groups' sums (of two keys: half).  With u = 2^-23, exp_approx(-d) is good
// to (2 + d) u (ex2.approx to 2 u, the product with log2 e to 0.8 u d) and
// rcp.approx to u, relative.  A sigmoid, with e = exp(-x): s (1 - s) (2 + |x|) u
// + s u / 2 + s u < 2.2 u; four of them are below 9 u.  A softmax, its
// argument, reciprocal and product rounded too: p (4 + 1.5 d) u < 4.5 u, and the
// common factor 1 / z, whose sum of at most 16 terms a lane and 5 levels is good
// to 2^-19.2 of a difference of at most 1: together below 2^-18 for two, 2^-17
// for four.  (The roundings of the keys and sums are counted with them.)
constexpr float kSigmoidError = 0x1.2p-20f;
constexpr float kSoftmaxError = 0x1p-17f;

__device__ __forceinline__ float exp_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * 1.4426950408889634f));
  return r;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// e^(a - b), a <= b: what the difference's rounding leaves is added to first order.
__device__ __forceinline__ float exp_diff(float a, float b) {
  const float d = a - b;
  if (!(d > -INFINITY)) return a == b ? 1.0f : 0.0f;         // infinite, or of two infinities
  const float t = d - a, lo = (a - (d - t)) - (b + t), e = expf(d);
  return fmaf(e, lo, e);
}

// A lane's V logits of token t: experts [V lane, V lane + V), -inf beyond E.
template <int V, bool BF16>
__device__ __forceinline__ void load_logits(const RouteParams& p, int64_t t, int lane, float* l) {
  constexpr int BYTES = V * (BF16 ? 2 : 4);
  if constexpr (BYTES >= 8) {
    // whole lanes, 8 or 16 bytes at a time, where rows allow it
    constexpr int W = BYTES % 16 == 0 ? 16 : 8;
    const uint8_t* row = static_cast<const uint8_t*>(p.logits) + (t * p.ld + V * lane) * (BF16 ? 2 : 4);
    if (p.vec && V * lane + V <= p.E) {
      uint32_t w[BYTES / 4];
#pragma unroll
      for (int i = 0; i < BYTES; i += W) {
        if constexpr (W == 16) {
          const uint4 q = __ldg(reinterpret_cast<const uint4*>(row + i));
          w[i / 4] = q.x, w[i / 4 + 1] = q.y, w[i / 4 + 2] = q.z, w[i / 4 + 3] = q.w;
        } else {
          const uint2 q = __ldg(reinterpret_cast<const uint2*>(row + i));
          w[i / 4] = q.x, w[i / 4 + 1] = q.y;
        }
      }
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float x = __uint_as_float(BF16 ? (v & 1 ? w[v / 2] & 0xFFFF0000u : w[v / 2] << 16) : w[v]);
        l[v] = fmaxf(x, -INFINITY) + 0.0f;
      }
      return;
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) l[v] = V * lane + v < p.E ? route_logit(p, t, V * lane + v) : -INFINITY;
}

// The biases of the lane's experts.
template <int V>
__device__ __forceinline__ void load_bias(const RouteParams& p, int lane, float* b) {
  if constexpr (V >= 4) {
    if (p.vec_bias && V * lane + V <= p.E) {
#pragma unroll
      for (int v = 0; v < V; v += 4) {
        const float4 q = __ldg(reinterpret_cast<const float4*>(p.bias + V * lane + v));
        b[v] = q.x, b[v + 1] = q.y, b[v + 2] = q.z, b[v + 3] = q.w;
      }
      return;
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) b[v] = V * lane + v < p.E ? __ldg(p.bias + V * lane + v) : 0.0f;
}

// Order-preserving integers of floating numbers; 0 is below all of them.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t u = __float_as_uint(v);
  return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ uint64_t order_key(double v) {
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(v));
  return (u >> 63) ? ~u : u | 0x8000000000000000ull;
}
__device__ __forceinline__ float key_float(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k & 0x7FFFFFFFu : ~k);
}
__device__ __forceinline__ double key_double(uint64_t k) {
  return __longlong_as_double(static_cast<long long>((k >> 63) ? k & 0x7FFFFFFFFFFFFFFFull : ~k));
}

// Maximum over the warp.
__device__ __forceinline__ uint32_t warp_max(uint32_t v) { return __reduce_max_sync(kAll, v); }
__device__ __forceinline__ uint64_t warp_max(uint64_t v) {
  const uint32_t hi = static_cast<uint32_t>(v >> 32);
  const uint32_t mh = __reduce_max_sync(kAll, hi);
  const uint32_t ml = __reduce_max_sync(kAll, hi == mh ? static_cast<uint32_t>(v) : 0u);
  return (static_cast<uint64_t>(mh) << 32) | ml;
}

// The keys of a lane in falling order (odd-even merge sort).
template <int V, typename Key>
__device__ __forceinline__ void sort_keys(Key (&k)[V]) {
#pragma unroll
  for (int p = 1; p < V; p *= 2)
#pragma unroll
    for (int d = p; d >= 1; d /= 2)
#pragma unroll
      for (int j = d % p; j + d < V; j += 2 * d)
#pragma unroll
        for (int i = j; i < j + d && i + d < V; ++i)
          if (i / (2 * p) == (i + d) / (2 * p)) {
            const Key a = k[i], b = k[i + d];
            k[i] = a > b ? a : b;
            k[i + d] = a > b ? b : a;
          }
}

// Keys a >= b are apart: |a - b| above the error of both.  32-bit keys of scores
// with a bias (ROUGH) have an error; that of a sum of two grows with their
// magnitudes, `mag`.
template <bool ROUGH, typename Key>
__device__ __forceinline__ bool route_apart(const RouteParams& p, Key a, Key b, float mag) {
  if constexpr (ROUGH) {
    if (b <= order_key(-INFINITY)) return true;            // masked or excluded: exact
    const float x = key_float(a), y = key_float(b);
    return x - y > (p.sigmoid ? kSigmoidError : kSoftmaxError) + 0x1p-23f * (fabsf(x) + fabsf(y) + mag);
  }
  return true;
}

// Whether a group's experts fill whole lanes, a power of two of them.
template <int V>
__device__ __forceinline__ bool whole_groups(const RouteParams& p) {
  const int size = p.E / p.groups, span = size / V;
  return span * V == size && (span & (span - 1)) == 0;
}

// One warp a token: lane holds the keys of experts [V lane, V lane + V).  A group
// counts with its largest key, or (TOP2) the sum of its two largest; equal groups
// go to the lowest.  Returns the lanes' bits: of the lanes whose group is among
// the best topg, or of lane g for group g where groups do not fill lanes
// (route_keep reads it).  `sure` is cleared where 32-bit keys leave it open.
template <int V, typename Key, bool TOP2>
__device__ __forceinline__ uint32_t route_groups(const RouteParams& p, const Key (&key)[V], int lane, bool& sure) {
  constexpr bool ROUGH = TOP2 && sizeof(Key) == 4;
  const int size = p.E / p.groups, span = size / V;
  const bool whole = whole_groups<V>(p);
  const int own = whole ? lane / span : lane;              // this lane's group, below p.groups
  Key t1 = 0, t2 = 0;                                      // the two largest keys of group `own`
  if (whole) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const Key k = key[v], low = k < t1 ? k : t1;
      t1 = k > t1 ? k : t1;
      t2 = low > t2 ? low : t2;
    }
    for (int o = 1; o < span; o <<= 1) {
      const Key u1 = __shfl_xor_sync(kAll, t1, o), u2 = __shfl_xor_sync(kAll, t2, o);
      const Key low = u1 < t1 ? u1 : t1, high = u2 > t2 ? u2 : t2;
      t1 = u1 > t1 ? u1 : t1;
      t2 = low > high ? low : high;
    }
  } else {
    for (int g = 0; g < p.groups; ++g) {
      Key a = 0, b = 0;                                    // of this lane
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int e = V * lane + v;
        if (e >= g * size && e < (g + 1) * size) {
          if (key[v] > a) { b = a; a = key[v]; }
          else if (key[v] > b) b = key[v];
        }
      }
      const Key first = warp_max(a);
      const int owner = __ffs(__ballot_sync(kAll, a == first)) - 1;
      const Key second = warp_max(lane == owner ? b : a);
      if (lane == g) { t1 = first; t2 = second; }
    }
  }
  Key mine = t1;
  float mag = 0.0f;
  if constexpr (TOP2) {
    if (size > 1) {
      if constexpr (ROUGH) {
        const float x = key_float(t1), y = key_float(t2);
        mine = order_key(x + y + 0.0f);
        // a sum may be far smaller than the two, and the errors with them
        if (own < p.groups && y > -INFINITY) mag = fabsf(x) + fabsf(y);
      } else {
        mine = order_key(key_double(t1) + key_double(t2) + 0.0);
      }
    }
  }
  // how many groups come before this lane's
  const int step = whole ? span : 1;
  int rank = 0;
  for (int g = 0; g < p.groups; ++g) {
    const Key other = __shfl_sync(kAll, mine, g * step);
    rank += g < own ? other >= mine : other > mine;
  }
  if (own >= p.groups) rank = p.groups;
  if constexpr (ROUGH) {
    const Key last = __shfl_sync(kAll, mine, __ffs(__ballot_sync(kAll, rank == p.topg - 1)) - 1);
    const Key next = __shfl_sync(kAll, mine, __ffs(__ballot_sync(kAll, rank == p.topg)) - 1);
    mag = __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(mag)));     // not negative: ordered as integers
    sure = sure && route_apart<ROUGH>(p, last, next, mag);
  }
  return __ballot_sync(kAll, rank < p.topg);
}

// Experts outside the groups of route_groups' bits get key 0.
template <int V, typename Key>
__device__ __forceinline__ void route_keep(const RouteParams& p, Key (&key)[V], int lane, uint32_t bits) {
  const int size = p.E / p.groups;
  const bool whole = whole_groups<V>(p);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int from = whole ? lane : min(31, (V * lane + v) / size);
    if (!((bits >> from) & 1u)) key[v] = 0;
  }
}

// The k largest keys; equal ones go to the lowest expert: the first lane's, and
// its first.  Returns lane j's j-th expert.
//
// ROUGH keys: the experts go on until one is apart from the next: `count` of
// them, whose order is only sure if `ordered`; `sure` is cleared where 32 do not
// settle the set.
//
// A lane sorts its keys once; a round then takes the largest head and moves its
// owner's keys up; which experts they were is looked up for all at the end.
// (Searching the lane's keys every round, with the groups' maxima one group
// after another, took 1740 instructions a token and 23 us at 8192 tokens of 256
// experts in 8 groups; now 1040 and 11.)
template <int V, typename Key, bool ROUGH>
__device__ __forceinline__ int route_select(const RouteParams& p, const Key (&key)[V], int lane, bool& sure, int& count,
                                            bool& ordered) {
  Key head[V];
#pragma unroll
  for (int v = 0; v < V; ++v) head[v] = key[v];
  sort_keys<V>(head);
  int owner = 0;                        // lane j: of the j-th key, `chosen`
  Key chosen = 0, before = 0;
  count = 0;
  for (;;) {
    const Key best = warp_max(head[0]);
    if (count >= p.topk) {
      if (!ROUGH || route_apart<ROUGH>(p, before, best, 0.0f)) break;
      if (count == 32) {
        sure = false;
        break;
      }
    }
    const int o = __ffs(__ballot_sync(kAll, head[0] == best)) - 1;
    if (lane == count) {
      owner = o;
      chosen = best;
    }
    if (lane == o) {
#pragma unroll
      for (int v = 0; v + 1 < V; ++v) head[v] = head[v + 1];
      head[V - 1] = 0;
    }
    before = best;
    ++count;
  }
  // equal keys of a lane follow one another: the how many-th of them this is
  const Key above = __shfl_up_sync(kAll, chosen, 1);
  const int owner_above = __shfl_up_sync(kAll, owner, 1);
  const uint32_t firsts = __ballot_sync(kAll, lane == 0 || above != chosen || owner_above != owner);
  int nth = lane - (31 - __clz(firsts & (0xFFFFFFFFu >> (31 - lane)))), id = 0;
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (__shfl_sync(kAll, key[v], owner) == chosen && nth-- == 0) id = V * owner + v;
  ordered = true;
  if constexpr (ROUGH) {
    const Key next = __shfl_down_sync(kAll, chosen, 1);
    ordered = __all_sync(kAll, lane + 1 >= count || route_apart<ROUGH>(p, chosen, next, 0.0f));
  }
  return id;
}

constexpr int kRouteWarps = 4;          // tokens of a CTA

// One warp a token.  Without a bias both scores grow with the logit, so the
// order of the logits is the exact one.  With a bias the selection is decided
// by score + bias in fp32 where the keys are further apart than its error
// (above, and their rounding), else again in fp64, for the experts in question
// where that settles it: there two biased scores that differ in exact arithmetic
// differ too, but for accidents below 2^-50.  (fp64 for every token took 42 us
// at 8192 tokens of 256 experts.)
template <int V, bool BIASED, bool BF16>
__global__ void __launch_bounds__(32 * kRouteWarps, V <= 8 ? 8 : 4) route_kernel(const RouteParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kRouteWarps + (threadIdx.x >> 5);
  griddep_wait();
  griddep_launch_dependents();
  if (t >= p.T) return;

  float l[V];
  load_logits<V, BF16>(p, t, lane, l);
  // softmax: the largest logit and the sum of exponentials (terms equal to the
  // maximum count 1, infinite ones too); no sum where every logit is masked
  float m = 0.0f, z = 1.0f;
  if (!p.sigmoid) {
    uint32_t top = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) top = max(top, order_key(l[v]));
    m = key_float(warp_max(top));
    z = 0.0f;
    if (fabsf(m) < INFINITY) {
#pragma unroll
      for (int v = 0; v < V; ++v) z += expf(l[v] - m);
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) z += l[v] > -INFINITY && l[v] == m ? 1.0f : 0.0f;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(kAll, z, o);
  }
  uint32_t key[V];
  if constexpr (BIASED) {
    float b[V];
    load_bias<V>(p, lane, b);
    if (p.sigmoid) {
#pragma unroll
      for (int v = 0; v < V; ++v) b[v] += rcp_approx(1.0f + exp_approx(-l[v]));
    } else {
      const float r = 1.0f / z;
#pragma unroll
      for (int v = 0; v < V; ++v) b[v] += l[v] == m ? r : exp_approx(l[v] - m) * r;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) key[v] = order_key(l[v] > -INFINITY ? b[v] + 0.0f : -INFINITY);
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) key[v] = order_key(l[v]);
  }
  if (V * lane + V > p.E) {
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (V * lane + v >= p.E) key[v] = 0;
  }

  // fp64: the softmax's sum, an expert's key, the lane's keys
  auto exact_sum = [&]() {
    double zd = 1.0;
    if (!p.sigmoid) {
      zd = 0.0;
#pragma unroll 1
      for (int v = 0; v < V; ++v) {
        const float x = V * lane + v < p.E ? route_logit(p, t, V * lane + v) : -INFINITY;
        if (x > -INFINITY) zd += x == m ? 1.0 : exp(static_cast<double>(x) - static_cast<double>(m));
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) zd += __shfl_xor_sync(kAll, zd, o);
    }
    return zd;
  };
  auto exact = [&](float v, int e, double zd) {
    double c = -INFINITY;
    if (v > -INFINITY) {
      const double x = v;
      const double s = p.sigmoid ? 1.0 / (1.0 + exp(-x)) : (v == m ? 1.0 : exp(x - static_cast<double>(m))) / zd;
      c = s + static_cast<double>(__ldg(p.bias + e)) + 0.0;
    }
    return order_key(c);
  };
  auto exact_keys = [&](uint64_t (&k)[V], double zd) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = V * lane + v;
      k[v] = e < p.E ? exact(l[v], e, zd) : 0;
    }
  };

  bool sure = true, ordered = true;
  uint32_t bits = kAll;
  if (p.topg < p.groups) {
    bits = route_groups<V, uint32_t, BIASED>(p, key, lane, sure);
    if constexpr (BIASED) {
      if (!sure) {
        uint64_t k[V];
        exact_keys(k, exact_sum());
        bits = route_groups<V, uint64_t, true>(p, k, lane, sure);
        sure = true;
      }
    }
    route_keep<V>(p, key, lane, bits);
  }
  int count, id = route_select<V, uint32_t, BIASED>(p, key, lane, sure, count, ordered);
  if constexpr (BIASED) {
    if (!sure || !ordered) {
      const double zd = exact_sum();
      if (sure) {
        // the right experts, in an order that is not sure
        const uint64_t mine = lane < count ? exact(route_logit(p, t, id), id, zd) : 0;
        int rank = 0, from = 0;
        for (int j = 0; j < count; ++j) {
          const uint64_t other = __shfl_sync(kAll, mine, j);
          const int e = __shfl_sync(kAll, id, j);
          rank += other > mine || (other == mine && e < id);
        }
        for (int j = 0; j < count; ++j)
          if (__shfl_sync(kAll, rank, j) == lane) from = j;
        id = __shfl_sync(kAll, id, from);
      } else {
        uint64_t k[V];
        exact_keys(k, zd);
        if (p.topg < p.groups) route_keep<V>(p, k, lane, bits);
        id = route_select<V, uint64_t, false>(p, k, lane, sure, count, ordered);
      }
    }
  }

  // Weights.  A score below fp64's range counts as 0.  Renormalized, scores are
  // taken relative to the largest selected logit (the sigmoid's: if negative),
  // so that none is lost to fp32's range, however small they all are.
  const float x = lane < p.topk ? route_logit(p, t, id) : -INFINITY;
  const bool live = x > -INFINITY && (p.sigmoid ? x > -709.0f : x == m || x - m > -745.0f);
  float top = p.sigmoid ? 0.0f : m;
  if (p.renorm) {
    const uint32_t k = warp_max(live ? order_key(x) : 0u);
    if (k) top = p.sigmoid ? fminf(key_float(k), 0.0f) : key_float(k);
  }
  float s = 0.0f;
  if (live) {
    if (!p.sigmoid) s = p.renorm ? exp_diff(x, top) : exp_diff(x, top) / z;
    else s = x >= 0.0f ? 1.0f / (1.0f + expf(-x)) : exp_diff(x, top) / (1.0f + expf(x));
  }
  if (p.renorm) {
    float sum = s;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
    s = sum > 0.0f ? s / sum : 0.0f;    // no selected expert has a score: no weight
  }
  if (lane < p.topk) {
    p.w[t * p.topk + lane] = s * p.scale;
    p.ids[t * p.topk + lane] = id;
  }
}

// --------------------------------------------------------------------- plan
// A stable counting sort of n (token, slot) entries by expert, in entry order
// within an expert, without atomics on results: every count and rank comes
// from a fixed order.  A block takes up to kPlanBlock entries, a warp a
// contiguous part of them; a ballot for each bit of the expert gives the ranks
// inside 32 entries (__match_any_sync, whose cost grows with the number of
// distinct values, took 17 us for 32768 entries of 128 experts).
constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kPlanBlock = 4096;
constexpr int kPlanCluster = 8;
constexpr int64_t kMaxEntries = int64_t{1} << 25;   // every block reads all blocks' counts: a cost that grows with n^2

struct PlanParams {
  const int* ids;
  int n, E, blocks;
  int bits;          // that tell E experts and none (all ones) apart
  int* offsets;      // [E + 1]
  int* sf_offsets;   // [E + 1]
  int* pos;          // [n]
  int* sf_row;       // [n]
  int* hist;         // [blocks, E] counts of the blocks (blocks > 1)
};

// A warp's part of a block: kPlanSteps steps of 32 entries, read at once (a
// load a step would wait out the latency of each).  Every id outside [0, E)
// becomes -1, whose low bits are no expert's: same_lanes looks at those only,
// so another negative id (ids less the first expert that is here) would count
// as the expert whose low bits it has.
constexpr int kPlanSteps = kPlanBlock / kPlanWarps / 32;

__device__ __forceinline__ void plan_load(const PlanParams& p, int i0, int lane, int* e) {
#pragma unroll
  for (int k = 0; k < kPlanSteps; ++k) {
    const int i = i0 + 32 * k + lane;
    e[k] = i < p.n ? __ldg(p.ids + i) : -1;
  }
#pragma unroll
  for (int k = 0; k < kPlanSteps; ++k)
    if (static_cast<unsigned>(e[k]) >= static_cast<unsigned>(p.E)) e[k] = -1;
}

// Lanes of the warp with the same value of the low `bits` bits.
__device__ __forceinline__ unsigned same_lanes(int e, int bits) {
  unsigned m = kAll;
  for (int b = 0; b < bits; ++b) {
    const bool set = (e >> b) & 1;
    const unsigned v = __ballot_sync(kAll, set);
    m &= set ? v : ~v;
  }
  return m;
}

// Counts of the warp's entries into cnt[E] (shared, the warp's own).
__device__ __forceinline__ void warp_count(const int* e, int steps, int bits, int* cnt, int lane) {
#pragma unroll
  for (int k = 0; k < kPlanSteps; ++k) {
    if (k >= steps) break;
    const unsigned same = same_lanes(e[k], bits);
    if (e[k] >= 0 && lane == __ffs(same) - 1) cnt[e[k]] += __popc(same);
    __syncwarp();
  }
}

// A block's entries of expert e: the sum of its warps' counts, by eight lanes.
__device__ __forceinline__ int block_count(const int* cnt, int E, int e, int sub) {
  int s = 0;
#pragma unroll
  for (int w = 0; w < kPlanWarps / 8; ++w) s += e < E ? cnt[(sub * (kPlanWarps / 8) + w) * (E + 1) + e] : 0;
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) s += __shfl_xor_sync(kAll, s, o);
  return s;
}

__global__ void __launch_bounds__(kPlanThreads) plan_count_kernel(const PlanParams p) {
  extern __shared__ int cnt[];                          // [warps][E + 1]: no two of 32 neighbours in a bank
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < kPlanWarps * (p.E + 1); i += kPlanThreads) cnt[i] = 0;
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();
  const int i0 = static_cast<int>(blockIdx.x) * kPlanBlock + warp * 32 * kPlanSteps;
  const int steps = (p.n - i0 + 31) >> 5;               // with entries; none where negative
  int id[kPlanSteps];
  plan_load(p, i0, lane, id);
  warp_count(id, steps, p.bits, cnt + warp * (p.E + 1), lane);
  __syncthreads();
  // eight lanes an expert, four warps' counts each
  const int sub = threadIdx.x & 7;
  for (int e0 = 0; e0 < p.E; e0 += kPlanThreads / 8) {
    const int e = e0 + (threadIdx.x >> 3);
    const int s = block_count(cnt, p.E, e, sub);
    if (sub == 0 && e < p.E) p.hist[blockIdx.x * p.E + e] = s;
  }
}

// CLUSTER: the blocks are one cluster and read each other's counts (32768
// entries of 128 experts, 8 blocks: 8.4 us; with the counts in a launch of their
// own, as for more blocks, 12.5).
template <bool CLUSTER>
__global__ void __launch_bounds__(kPlanThreads) plan_place_kernel(const PlanParams p) {
  extern __shared__ int cnt[];                          // [warps][E + 1]: counts, then first ranks of the warps
  __shared__ int first[kMaxExperts + 1], sf_first[kMaxExperts + 1], own[CLUSTER ? kMaxExperts : 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < kPlanWarps * (p.E + 1); i += kPlanThreads) cnt[i] = 0;
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();
  const int i0 = static_cast<int>(blockIdx.x) * kPlanBlock + warp * 32 * kPlanSteps;
  const int steps = (p.n - i0 + 31) >> 5;               // with entries; none where negative
  int id[kPlanSteps];
  plan_load(p, i0, lane, id);
  warp_count(id, steps, p.bits, cnt + warp * (p.E + 1), lane);
  __syncthreads();
  // Eight lanes an expert: its entries in the blocks before this one and in
  // all (each lane every eighth block), and before each warp (four warps each).
  const int sub = threadIdx.x & 7;
  if constexpr (CLUSTER) {
    for (int e0 = 0; e0 < p.E; e0 += kPlanThreads / 8) {
      const int e = e0 + (threadIdx.x >> 3);
      const int s = block_count(cnt, p.E, e, sub);
      if (sub == 0 && e < p.E) own[e] = s;
    }
    sm100::cluster_sync();
  }
  for (int e0 = 0; e0 < p.E; e0 += kPlanThreads / 8) {
    const int e = e0 + (threadIdx.x >> 3);
    const bool in = e < p.E;
    int before = 0, total = 0;
    if (p.blocks > 1 && in) {
      for (int b = sub; b < p.blocks; b += 8) {
        int c;
        if constexpr (CLUSTER)
          asm volatile("ld.shared::cluster.s32 %0, [%1];"
                       : "=r"(c) : "r"(sm100::mapa_shared(sm100::smem_u32(own + e), b)) : "memory");
        else c = __ldg(p.hist + b * p.E + e);
        if (b < static_cast<int>(blockIdx.x)) before += c;
        total += c;
      }
    }
    int c[kPlanWarps / 8], mine = 0;
#pragma unroll
    for (int w = 0; w < kPlanWarps / 8; ++w) {
      c[w] = in ? cnt[(sub * (kPlanWarps / 8) + w) * (p.E + 1) + e] : 0;
      mine += c[w];
    }
    int run = mine;                                     // inclusive over the lanes
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
      const int v = __shfl_up_sync(kAll, run, o, 8);
      if (sub >= o) run += v;
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
      before += __shfl_xor_sync(kAll, before, o);
      total += __shfl_xor_sync(kAll, total, o);
    }
    if (in) {
      if (sub == 7) first[e + 1] = p.blocks > 1 ? total : run;
      int at = before + run - mine;
#pragma unroll
      for (int w = 0; w < kPlanWarps / 8; ++w) {
        cnt[(sub * (kPlanWarps / 8) + w) * (p.E + 1) + e] = at;
        at += c[w];
      }
    }
  }
  if constexpr (CLUSTER) sm100::cluster_sync();         // no block leaves while its counts are read
  else __syncthreads();
  if (warp == 0) {                                      // sums over experts
    int rows = 0, blocks = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const int c = e0 + lane < p.E ? first[e0 + lane + 1] : 0;
      int v = c, b = (c + 127) >> 7;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v2 = __shfl_up_sync(kAll, v, o), b2 = __shfl_up_sync(kAll, b, o);
        if (lane >= o) { v += v2; b += b2; }
      }
      if (e0 + lane < p.E) {
        first[e0 + lane + 1] = rows + v;
        sf_first[e0 + lane + 1] = blocks + b;
      }
      rows += __shfl_sync(kAll, v, 31);
      blocks += __shfl_sync(kAll, b, 31);
    }
    if (lane == 0) first[0] = sf_first[0] = 0;
  }
  __syncthreads();
  if (blockIdx.x == 0)
    for (int e = threadIdx.x; e <= p.E; e += kPlanThreads) {
      p.offsets[e] = first[e];
      p.sf_offsets[e] = sf_first[e];
    }
  int* mine = cnt + warp * (p.E + 1);
#pragma unroll
  for (int k = 0; k < kPlanSteps; ++k) {
    if (k >= steps) break;
    const int i = i0 + 32 * k + lane, e = id[k];
    const unsigned same = same_lanes(e, p.bits);
    const int rank = e >= 0 ? mine[e] + __popc(same & ((1u << lane) - 1u)) : 0;
    __syncwarp();
    if (e >= 0 && lane == __ffs(same) - 1) mine[e] += __popc(same);
    __syncwarp();
    if (i < p.n) {
      p.pos[i] = e >= 0 ? first[e] + rank : -1;
      p.sf_row[i] = e >= 0 ? sf_first[e] * 128 + rank : -1;
    }
  }
}

// ------------------------------------------------------------------ combine
// y[t] = bf16(sum_j w[t, j] o[pos[t, j]]), fp32, j in order; 8 columns a thread.
__global__ void __launch_bounds__(256) combine_kernel(const uint16_t* o, int64_t ldo, const int* pos, const float* w,
                                                      int64_t T, int topk, int64_t H, uint16_t* y, int64_t ldy) {
  griddep_wait();
  griddep_launch_dependents();
  const int64_t cols = H >> 3, total = T * cols;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t t = i / cols;
    const int64_t c = (i - t * cols) * 8;
    float acc[8] = {};
    for (int j0 = 0; j0 < topk; j0 += 8) {
      uint4 v[8];
      float s[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int r = j0 + j < topk ? __ldg(pos + t * topk + j0 + j) : -1;
        s[j] = r >= 0 ? __ldg(w + t * topk + j0 + j) : 0.0f;
        v[j] = r >= 0 ? __ldg(reinterpret_cast<const uint4*>(o + r * ldo + c)) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t u[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          acc[2 * k] = fmaf(s[j], __uint_as_float(u[k] << 16), acc[2 * k]);
          acc[2 * k + 1] = fmaf(s[j], __uint_as_float(u[k] & 0xFFFF0000u), acc[2 * k + 1]);
        }
      }
    }
    uint32_t r[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(acc[2 * k], acc[2 * k + 1]);
      r[k] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(y + t * ldy + c) = make_uint4(r[0], r[1], r[2], r[3]);
  }
}

template <int V>
fp8q_status launch_route_v(const RouteParams& p, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>((p.T + kRouteWarps - 1) / kRouteWarps));
  const dim3 block(32 * static_cast<unsigned>(p.T < kRouteWarps ? p.T : kRouteWarps));
  auto kern = p.bias ? (p.bf16 ? route_kernel<V, true, true> : route_kernel<V, true, false>)
                     : (p.bf16 ? route_kernel<V, false, true> : route_kernel<V, false, false>);
  return launch_kernel(kern, grid, block, 0, s, 1, p);
}

fp8q_status launch_route(const RouteParams& p, cudaStream_t s) {
  if (p.E <= 32) return launch_route_v<1>(p, s);
  if (p.E <= 64) return launch_route_v<2>(p, s);
  if (p.E <= 128) return launch_route_v<4>(p, s);
  if (p.E <= 256) return launch_route_v<8>(p, s);
  return launch_route_v<16>(p, s);
}

int64_t plan_blocks(int64_t n) { return n <= kPlanBlock ? 1 : (n + kPlanBlock - 1) / kPlanBlock; }

// The pieces of the experts' workspace, each 256-byte aligned.
struct ExpertsSpace {
  size_t pos, sf_row, offsets, sf_offsets, hist, xq, xsf, hq, hsf, o, total;
};
ExpertsSpace experts_space(int64_t T, int64_t topk, int64_t E, int64_t H, int64_t I, int format) {
  ExpertsSpace w{};
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t r = at;
    at += (bytes + 255) / 256 * 256;
    return r;
  };
  // scale block rows: every expert's last may be ragged
  const int64_t R = T * topk, blocks = R / 128 + (R < E ? R : E);
  w.pos = take(R * 4);
  w.sf_row = take(R * 4);
  w.offsets = take((E + 1) * 4);
  w.sf_offsets = take((E + 1) * 4);
  w.hist = take(fp8q_moe_plan_workspace_bytes(R, E));
  w.xq = take(R * (H / 2));
  w.xsf = take(blocks * fp4_kblocks(format, H) * 512);
  w.hq = take(R * (I / 2));
  w.hsf = take(blocks * fp4_kblocks(format, I) * 512);
  w.o = take(R * H * 2);
  w.total = at;
  return w;
}

bool experts_sizes(int64_t T, int topk, int64_t E, int64_t H, int64_t I, int format) {
  return (format == FP8Q_FP4_NV || format == FP8Q_FP4_MX) && T >= 0 && topk > 0 && topk <= kMaxTopk && E > 0 &&
         E <= kMaxExperts && H > 0 && H % 32 == 0 && I > 0 && H <= (1 << 24) && I <= (1 << 24) &&
         T * topk <= kMaxEntries;
}

}  // namespace
}  // namespace fp8q

using namespace fp8q;

extern "C" fp8q_status fp8q_moe_route(const void* logits, int logits_bf16, int64_t T, int64_t E, int64_t ldl, int topk,
                                      int scoring, const float* bias, int num_groups, int topk_groups, int renormalize,
                                      float scale, float* weights, int* ids, void* stream) {
  if (T < 0 || E <= 0 || ldl < E || topk <= 0 || num_groups <= 0 || topk_groups <= 0) return FP8Q_ERR_INVALID_ARG;
  if (logits_bf16 != 0 && logits_bf16 != 1) return FP8Q_ERR_INVALID_ARG;
  if (scoring != FP8Q_ROUTE_SOFTMAX && scoring != FP8Q_ROUTE_SIGMOID) return FP8Q_ERR_INVALID_ARG;
  if (renormalize != 0 && renormalize != 1) return FP8Q_ERR_INVALID_ARG;
  if (E > kMaxExperts || topk > kMaxTopk || num_groups > 32) return FP8Q_ERR_UNSUPPORTED;
  if (E % num_groups != 0 || topk_groups > num_groups || topk > E / num_groups * topk_groups)
    return FP8Q_ERR_INVALID_ARG;
  if (T >= (int64_t{1} << 31)) return FP8Q_ERR_INVALID_ARG;
  if (T == 0) return FP8Q_OK;
  if (!logits || !weights || !ids) return FP8Q_ERR_INVALID_ARG;
  if (!aligned(logits, logits_bf16 ? 2 : 4) || !aligned(bias, 4) || !aligned(weights, 4) || !aligned(ids, 4))
    return FP8Q_ERR_INVALID_ARG;
  const int vec = aligned(logits, 16) && ldl * (logits_bf16 ? 2 : 4) % 16 == 0;
  const RouteParams p{logits, T, ldl, static_cast<int>(E), logits_bf16, vec, aligned(bias, 16),
                      scoring == FP8Q_ROUTE_SIGMOID, bias, num_groups, topk_groups, topk, renormalize, scale, weights, ids};
  return launch_route(p, static_cast<cudaStream_t>(stream));
}

extern "C" size_t fp8q_moe_plan_workspace_bytes(int64_t n, int64_t E) {
  if (n <= 0 || E <= 0) return 0;
  const int64_t b = plan_blocks(n);
  return b > 1 ? static_cast<size_t>(b) * static_cast<size_t>(E) * 4 : 0;
}

extern "C" fp8q_status fp8q_moe_plan(const int* ids, int64_t n, int64_t E, int* offsets, int* sf_offsets, int* pos,
                                     int* sf_row, void* workspace, size_t ws_bytes, void* stream) {
  if (n < 0 || E <= 0 || n >= (int64_t{1} << 30)) return FP8Q_ERR_INVALID_ARG;
  if (E > kMaxExperts || n > kMaxEntries) return FP8Q_ERR_UNSUPPORTED;
  if (!offsets || !sf_offsets || !aligned(offsets, 4) || !aligned(sf_offsets, 4)) return FP8Q_ERR_INVALID_ARG;
  if (n > 0 && (!ids || !pos || !sf_row || !aligned(ids, 4) || !aligned(pos, 4) || !aligned(sf_row, 4)))
    return FP8Q_ERR_INVALID_ARG;
  const size_t need = fp8q_moe_plan_workspace_bytes(n, E);
  if (need > 0 && (!workspace || ws_bytes < need || !aligned(workspace, 4))) return FP8Q_ERR_INVALID_ARG;
  const int blocks = static_cast<int>(n > 0 ? plan_blocks(n) : 1);
  int bits = 1;
  while ((1 << bits) <= E) ++bits;
  const PlanParams p{ids, static_cast<int>(n), static_cast<int>(E), blocks, bits, offsets, sf_offsets, pos, sf_row,
                     static_cast<int*>(workspace)};
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const size_t smem = static_cast<size_t>(kPlanWarps) * static_cast<size_t>(E + 1) * 4;   // at most 65 KB
  static std::atomic<int> attr_done[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return FP8Q_ERR_CUDA;
  if (!attr_done[dev].load(std::memory_order_relaxed)) {
    for (auto k : {plan_count_kernel, plan_place_kernel<false>, plan_place_kernel<true>})
      if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kPlanWarps * (kMaxExperts + 1) * 4) !=
          cudaSuccess)
        return FP8Q_ERR_CUDA;
    attr_done[dev].store(1, std::memory_order_relaxed);
  }
  if (blocks > 1 && blocks <= kPlanCluster)
    return launch_kernel(plan_place_kernel<true>, dim3(blocks), dim3(kPlanThreads), smem, s, blocks, p);
  if (blocks > 1) {
    const fp8q_status st = launch_kernel(plan_count_kernel, dim3(blocks), dim3(kPlanThreads), smem, s, 1, p);
    if (st != FP8Q_OK) return st;
  }
  return launch_kernel(plan_place_kernel<false>, dim3(blocks), dim3(kPlanThreads), smem, s, 1, p);
}

extern "C" fp8q_status fp8q_moe_combine(const void* o, int64_t ldo, const int* pos, const float* weights, int64_t T,
                                        int topk, int64_t H, void* y, int64_t ldy, void* stream) {
  if (T < 0 || topk <= 0 || H <= 0 || H % 8 != 0 || ldo < H || ldo % 8 != 0 || ldy < H || ldy % 8 != 0)
    return FP8Q_ERR_INVALID_ARG;
  if (T == 0) return FP8Q_OK;
  if (!o || !pos || !weights || !y) return FP8Q_ERR_INVALID_ARG;
  if (!aligned(o, 16) || !aligned(y, 16) || !aligned(pos, 4) || !aligned(weights, 4)) return FP8Q_ERR_INVALID_ARG;
  const int64_t blocks = (T * (H >> 3) + 255) / 256, cap = static_cast<int64_t>(num_sms()) * 32;
  return launch_kernel(combine_kernel, dim3(static_cast<unsigned>(blocks < cap ? blocks : cap)), dim3(256), 0,
                       static_cast<cudaStream_t>(stream), 1, static_cast<const uint16_t*>(o), ldo, pos, weights, T, topk,
                       H, static_cast<uint16_t*>(y), ldy);
}

extern "C" size_t fp8q_moe_experts_fp4_workspace_bytes(int64_t T, int topk, int64_t E, int64_t H, int64_t I, int format) {
  if (!experts_sizes(T, topk, E, H, I, format) || T == 0) return 0;
  return experts_space(T, topk, E, H, I, format).total;
}

extern "C" fp8q_status fp8q_moe_experts_fp4(const void* x, int64_t T, int64_t ldx, const int* ids, const float* weights,
                                            int topk, int64_t E, int64_t H, int64_t I, int format, const void* w13,
                                            const uint8_t* w13_sf, const void* w2, const uint8_t* w2_sf,
                                            const float* x_gscale, const float* w13_gscale, const float* h_gscale,
                                            const float* w2_gscale, void* y, int64_t ldy, void* workspace,
                                            size_t ws_bytes, void* stream) {
  if (!experts_sizes(T, topk, E, H, I, format)) return FP8Q_ERR_INVALID_ARG;
  if (I % 128 != 0) return FP8Q_ERR_UNSUPPORTED;
  if (ldx < H || ldx % 8 != 0 || ldy < H || ldy % 8 != 0) return FP8Q_ERR_INVALID_ARG;
  if (format == FP8Q_FP4_MX && (x_gscale || w13_gscale || h_gscale || w2_gscale)) return FP8Q_ERR_INVALID_ARG;
  if (T == 0) return FP8Q_OK;
  if (!x || !ids || !weights || !w13 || !w13_sf || !w2 || !w2_sf || !y || !workspace) return FP8Q_ERR_INVALID_ARG;
  const ExpertsSpace sp = experts_space(T, topk, E, H, I, format);
  if (ws_bytes < sp.total || !aligned(workspace, 256)) return FP8Q_ERR_INVALID_ARG;
  uint8_t* b = static_cast<uint8_t*>(workspace);
  int* pos = reinterpret_cast<int*>(b + sp.pos);
  int* sf_row = reinterpret_cast<int*>(b + sp.sf_row);
  int* offsets = reinterpret_cast<int*>(b + sp.offsets);
  int* sf_offsets = reinterpret_cast<int*>(b + sp.sf_offsets);
  const int64_t R = T * topk;
  // every argument is checked before the first launch: what the calls below would refuse
  if (!aligned(x, 16) || !aligned(y, 16) || !aligned(ids, 4) || !aligned(weights, 4) || !aligned(w13, 16) ||
      !aligned(w13_sf, 16) || !aligned(w2, 16) || !aligned(w2_sf, 16) || !aligned(x_gscale, 4) ||
      !aligned(w13_gscale, 4) || !aligned(h_gscale, 4) || !aligned(w2_gscale, 4))
    return FP8Q_ERR_INVALID_ARG;
  constexpr int64_t kMax32 = int64_t{1} << 31;          // rows of all weights, tiles
  const int64_t tiles = R / 128 + E;
  if (E * 2 * I >= kMax32 || E * H >= kMax32 || tiles * ((2 * I + 63) / 64) >= kMax32 || tiles * ((H + 63) / 64) >= kMax32)
    return FP8Q_ERR_INVALID_ARG;
  fp8q_status st;
  if (R <= kSmallPlan) {
    st = moe_plan_quant_small(x, T, H, ldx, ids, topk, static_cast<int>(E), format, x_gscale, offsets, sf_offsets, pos,
                              sf_row, b + sp.xq, b + sp.xsf, static_cast<cudaStream_t>(stream));
  } else {
    st = fp8q_moe_plan(ids, R, E, offsets, sf_offsets, pos, sf_row, b + sp.hist, sp.xq - sp.hist, stream);
    if (st != FP8Q_OK) return st;
    st = fp8q_moe_fp4_quant(x, T, H, ldx, topk, pos, sf_row, format, x_gscale, b + sp.xq, H / 2, b + sp.xsf, stream);
  }
  if (st != FP8Q_OK) return st;
  st = fp8q_grouped_mm_fp4_silu_quant(b + sp.xq, w13, b + sp.xsf, w13_sf, format, x_gscale, w13_gscale, offsets,
                                      sf_offsets, E, R, I, H, h_gscale, b + sp.hq, b + sp.hsf, stream);
  if (st != FP8Q_OK) return st;
  st = fp8q_grouped_mm_fp4(b + sp.hq, w2, b + sp.hsf, w2_sf, format, h_gscale, w2_gscale, offsets, sf_offsets, E, R, H,
                           I, b + sp.o, H, stream);
  if (st != FP8Q_OK) return st;
  return fp8q_moe_combine(b + sp.o, H, pos, weights, T, topk, H, y, ldy, stream);
}
