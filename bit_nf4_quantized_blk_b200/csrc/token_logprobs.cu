// Log probabilities of given tokens, their entropy, the most likely
// alternatives, and the gradient (sm_100a).
//
// Per row of V logits x, with c = 1 / temperature, m = max x:
//   s = sum exp((x - m) c),   log p_j = (x_j - m) c - log s
//   H = -sum p log p = log s - (sum exp(t) t) / s,   t = (x - m) c
// in one pass over the row: every thread keeps a running (m, s, q = sum e t)
// and rescales it when its maximum grows,
//   s' = a s,  q' = a (q + (m - m') c s),  a = exp((m - m') c),
// and the threads' triples are joined the same way.  m stays the exact
// logit, and (m, log s) are returned apart: their sum would lose log s beside
// a large |m| (a row masked to the type's lowest value), their difference
// with x is exact.
//
// HBM-bound: 2 or 4 bytes per logit against about 6 instructions (packed fp32
// pairs) and one exponential.  Behind HBM the issue slots are the tightest (bf16,
// top 5: 61% of active cycles), then the exponentials (46%).  CTAs
// stay for many rows and every thread runs its own ring of asynchronous
// copies (cp.async into slots that it alone reads, so without barriers) across
// the rows' ends: the next row arrives while this one is reduced.  With few
// rows a cluster of up to 8 CTAs shares each row and joins over distributed
// shared memory, still one launch without a workspace.  Measured, bf16: 4096 x
// 50257 without alternatives 80 us (412 MB, 5.1 TB/s), with 5 of them 102 to 106,
// with 20 112; 2048 x 131072 93, 102 and 108 us; one row of 131072 6 to 12 us.
//
// The k largest come from the same pass.  The k-th largest (or a little less)
// of the threads' maxima is a bound that at least k logits reach, and only
// threads whose maximum reaches it are looked through once more (in L2): the
// one step that held it, or everything where a second step's maximum reaches
// the bound as well.  Should ties put more logits at the bound than the list
// holds, those above the bound are ranked and the rest taken from the row's
// start, where the lowest ids are; should that many be above it (the largest
// logits sitting in a few threads), they are taken one by one.
//
// The gradient  dx_j = c (g (1[j = t] - p_j) - g_H p_j (log p_j + H)) is
// elementwise from the saved m, log s and H: one read, one write; 2048 x 131072
// in 186 us (1.07 GB, 5.8 TB/s).
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "f32x2.cuh"
#include "kernels.cuh"

namespace qnf4 {

namespace {

constexpr int kLpThreads = 256;
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kLpVecs = 4;       // 16-byte vectors per thread and step
constexpr int kLpStages = 3;     // steps in flight
constexpr int kLpPerSm = 4;      // CTAs per SM (registers and shared memory)
constexpr int kLpMaxCluster = 8;
constexpr int kLpList = 256;     // logits at or above the bound that are ranked directly
constexpr int kLpRing = kLpStages * kLpVecs * kLpThreads * 16;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNegInf = -__builtin_huge_valf();

// Largest of two, NaN if either is (fmaxf drops NaN).
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// The values of one 16-byte vector.
template <typename T>
constexpr int kLpPer = 16 / static_cast<int>(sizeof(T));

template <typename T>
__device__ __forceinline__ void lp_values(const uint4& u, float (&v)[kLpPer<T>]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 2) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    } else {
      v[i] = __uint_as_float(w[i]);
    }
  }
}

template <typename T>
__device__ __forceinline__ uint4 lp_neg_inf() {
  const uint32_t w = sizeof(T) == 2 ? 0xFF80FF80u : 0xFF800000u;
  return make_uint4(w, w, w, w);
}

// Vector `vec` of a row of V logits: whole vectors by one load, the ragged
// last one value by value (nothing past V is read), past the end -inf.
template <typename T>
__device__ __forceinline__ uint4 lp_load(const T* row, int64_t V, int64_t vec) {
  constexpr int P = kLpPer<T>;
  const int64_t first = vec * P;
  if (first + P <= V) return *reinterpret_cast<const uint4*>(row + first);
  uint4 u = lp_neg_inf<T>();
  if (first >= V) return u;
  uint32_t* w = reinterpret_cast<uint32_t*>(&u);
#pragma unroll
  for (int i = 0; i < P; ++i) {
    if (first + i >= V) continue;
    if constexpr (sizeof(T) == 2)
      w[i / 2] = i % 2 ? (w[i / 2] & 0xFFFFu) | (static_cast<uint32_t>(row[first + i]) << 16)
                       : (w[i / 2] & 0xFFFF0000u) | row[first + i];
    else
      w[i] = __float_as_uint(row[first + i]);
  }
  return u;
}

// Unsigned integers in the order of the values (-0 = 0, NaN above everything; never 0).
__device__ __forceinline__ uint32_t lp_order(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);
  return v != v ? 0xFFFFFFFFu : (u >> 31) ? ~u : (u | 0x80000000u);
}

// (value, id) as one key: larger values first, the lower id first among equals.  0 is below every key.
__device__ __forceinline__ uint64_t lp_key(float v, int64_t id) {
  return (static_cast<uint64_t>(lp_order(v)) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(id));
}

__device__ __forceinline__ uint64_t max_u64(uint64_t a, uint64_t b) { return a > b ? a : b; }

__device__ __forceinline__ float lp_key_value(uint64_t key) {
  const uint32_t order = static_cast<uint32_t>(key >> 32);
  if (order == 0xFFFFFFFFu) return __uint_as_float(0x7FC00000u);
  return __uint_as_float((order >> 31) ? (order & 0x7FFFFFFFu) : ~order);
}

// A value such that everything of order `bound` or more is not below it (NaN, not below which is everything, at the top).
__device__ __forceinline__ float lp_least(uint32_t bound) {
  if (bound <= 0x007FFFFFu) return kNegInf;
  return lp_key_value(static_cast<uint64_t>(bound) << 32);
}

__device__ __forceinline__ int lp_key_id(uint64_t key) {
  return static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(key));
}

// Running sums of one thread or of several joined.
struct LpSums {
  float m, s, q;  // maximum; sum e^t; sum e^t t in base-2 units of t

  // Take the sums over to maximum `to` (>= m, or NaN).
  __device__ __forceinline__ void move(float to, float c2) {
    if (s != 0.0f) {
      const float t = max_nan((m - to) * c2, -1000.0f);  // far below: a = 0, and 0 t = 0
      const float a = ex2(t);
      q = a * fmaf(t, s, q);
      s *= a;
    }
    m = to;
  }
};

// Largest of one thread's packed or plain values.
template <typename T>
__device__ __forceinline__ float lp_max(const uint4 (&u)[kLpVecs]) {
  if constexpr (sizeof(T) == 2) {
    uint32_t m = 0xFF80FF80u;
#pragma unroll
    for (int i = 0; i < kLpVecs; ++i) {
      const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(w[j]));
    }
    return max_nan(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u));
  } else {
    float m = kNegInf;
#pragma unroll
    for (int i = 0; i < kLpVecs; ++i)
      m = max_nan(max_nan(max_nan(m, __uint_as_float(u[i].x)), __uint_as_float(u[i].y)),
                  max_nan(__uint_as_float(u[i].z), __uint_as_float(u[i].w)));
    return m;
  }
}

// The sums of the 2^n lanes around this one, in each of them: the maximum
// first, so that every lane moves its sums once.
template <int kLanes>
__device__ __forceinline__ LpSums lp_join_lanes(LpSums a, float c2) {
  float m = a.m;
#pragma unroll
  for (int d = kLanes / 2; d > 0; d >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, d));
  a.move(m, c2);
#pragma unroll
  for (int d = kLanes / 2; d > 0; d >>= 1) {
    a.s += __shfl_xor_sync(0xffffffffu, a.s, d);
    a.q += __shfl_xor_sync(0xffffffffu, a.q, d);
  }
  return a;
}

struct LpShared {
  LpSums warp[2][kLpWarps];  // alternate from row to row, as the counts do
  LpSums cta;                // this CTA's part of the row, for the cluster
  LpSums row;                // (maximum, log sum) of the whole row
  uint64_t top[kLogprobsMaxTop];  // this CTA's largest keys, largest first, for the cluster
  uint64_t list[kLpList];
  uint64_t best[kLpWarps];
  uint32_t order[kLpThreads];  // the threads' maxima, as lp_order
  uint32_t bound;
  int listed[2], deep[2], shallow[2];
  uint8_t cand[kLpThreads];  // deep ones from the front, shallow ones from the back
  int step[kLpThreads];      // of the shallow ones: the step of the maximum
};

// The same shared object in CTA `rank` of the cluster.
__device__ __forceinline__ uint64_t ld_cluster_u64(const void* p, uint32_t rank) {
  uint64_t v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(map_to_cta(p, rank)) : "memory");
  return v;
}
__device__ __forceinline__ float ld_cluster_f32(const void* p, uint32_t rank) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(map_to_cta(p, rank)) : "memory");
  return v;
}

// This CTA's vectors of a row: [first, end), of which those below `whole` lie
// within the row entirely (at most one, the row's last, does not).
struct LpSegment {
  int64_t first, end, whole;
};

// A value that at least k of the warp's 32 N values reach, found bit by bit
// from the top: the k-th largest itself, or, with `slack`, the first one on
// the way that no more than k + slack reach.
template <int N>
__device__ __forceinline__ uint32_t lp_bound(const uint32_t (&v)[N], int k, int slack) {
  uint32_t bound = 0;
  for (uint32_t bit = 0x80000000u; bit != 0; bit >>= 1) {
    const uint32_t at = bound | bit;
    int mine = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) mine += v[i] >= at;
    const int n = __reduce_add_sync(0xffffffffu, mine);
    if (n < k) continue;
    bound = at;
    if (n <= k + slack) break;
  }
  return bound;
}

// The bound of the threads' maxima, by one warp.
__device__ __forceinline__ uint32_t lp_threads_bound(const LpShared& sh, int k, int slack) {
  uint32_t v[kLpThreads / 32];
#pragma unroll
  for (int i = 0; i < kLpThreads / 32; ++i) v[i] = sh.order[i * 32 + (threadIdx.x & 31)];
  return lp_bound(v, k, slack);
}

// Adds this warp's threads with `in` to a list from sh.cand[0] on or, with
// kBack, from its end back; *count, zero before, becomes their number.
template <bool kBack>
__device__ __forceinline__ void lp_candidates(LpShared& sh, bool in, int* count) {
  const uint32_t all = __ballot_sync(0xffffffffu, in);
  if (all == 0) return;
  const int lane = threadIdx.x & 31;
  int at = 0;
  if (lane == 0) at = atomicAdd(count, __popc(all));
  at = __shfl_sync(0xffffffffu, at, 0) + __popc(all & ((1u << lane) - 1u));
  if (in) sh.cand[kBack ? kLpThreads - 1 - at : at] = static_cast<uint8_t>(threadIdx.x);
}

// f(value, id) of a vector's logits that are not below `least`.
template <typename T, typename F>
__device__ __forceinline__ void lp_scan_vector(const T* row, int64_t V, const LpSegment& seg, int64_t vec, float least,
                                               F&& f) {
  constexpr int P = kLpPer<T>;
  if (vec >= seg.end) return;
  float x[P];
  lp_values<T>(lp_load(row, V, vec), x);
  bool any = false;
#pragma unroll
  for (int j = 0; j < P; ++j) any = any || !(x[j] < least);
  if (!any) return;
#pragma unroll
  for (int j = 0; j < P; ++j)
    if (!(x[j] < least) && vec * P + j < V) f(x[j], vec * P + j);
}

// lp_scan_vector of every vector of the `cands` listed threads, by the whole
// CTA; thread c has the vectors seg.first + c, + kLpThreads, ...
template <typename T, typename F>
__device__ __forceinline__ void lp_scan(const LpShared& sh, const T* row, int64_t V, const LpSegment& seg, int cands,
                                        float least, F&& f) {
  const uint32_t per = static_cast<uint32_t>((seg.end - seg.first + kLpThreads - 1) / kLpThreads), items = cands * per;
#pragma unroll 1
  for (uint32_t i = threadIdx.x; i < items; i += kLpThreads) {
    const uint32_t c = i / per;
    lp_scan_vector(row, V, seg, seg.first + sh.cand[c] + static_cast<int64_t>(i - c * per) * kLpThreads, least, f);
  }
}

// put(rank, key) of the keys in the list that fewer than k exceed.
template <typename F>
__device__ __forceinline__ void lp_rank_list(const LpShared& sh, int n, int k, int first, int stride, F&& put) {
  for (int i = first; i < n; i += stride) {
    const uint64_t mine = sh.list[i];
    int larger = 0;
#pragma unroll 4
    for (int o = 0; o < n; ++o) larger += sh.list[o] > mine;
    if (larger < k) put(larger, mine);
  }
}

// The k largest when more logits than the list holds reach the bound.
template <typename T, typename F>
__device__ void lp_select_many(LpShared& sh, const T* row, int64_t V, const LpSegment& seg, int k, uint32_t order,
                               int turn, F&& put) {
  constexpr int P = kLpPer<T>;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  __syncthreads();  // everyone has read the count
  if (warp == 0) {
    const uint32_t exact = lp_threads_bound(sh, k, 0);
    if (lane == 0) sh.bound = exact, sh.listed[turn] = sh.deep[turn] = 0;
  }
  __syncthreads();
  const uint32_t bound = sh.bound;
  const float least = lp_least(bound);
  lp_candidates<false>(sh, order >= bound, &sh.deep[turn]);
  __syncthreads();
  const int cands = sh.deep[turn];
  lp_scan(sh, row, V, seg, cands, least, [&](float x, int64_t id) {
    if (lp_order(x) <= bound) return;
    const int at = atomicAdd(&sh.listed[turn], 1);
    if (at < kLpList) sh.list[at] = lp_key(x, id);
  });
  __syncthreads();
  int n = sh.listed[turn];
  if (n <= kLpList) {
    lp_rank_list(sh, n, k, tid, kLpThreads, put);
    if (warp == 0) {  // then the lowest ids at the bound
      for (int64_t v = seg.first + lane; n < k && v - lane < seg.end; v += 32) {
        float x[P];
        lp_values<T>(v < seg.end ? lp_load(row, V, v) : lp_neg_inf<T>(), x);
        int mine = 0;
#pragma unroll
        for (int j = 0; j < P; ++j) mine += v < seg.end && v * P + j < V && lp_order(x[j]) == bound;
        int upto = mine;  // of the lanes up to this one
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
          const int o = __shfl_up_sync(0xffffffffu, upto, d);
          if (lane >= d) upto += o;
        }
        int at = n + upto - mine;
#pragma unroll
        for (int j = 0; j < P; ++j)
          if (v < seg.end && v * P + j < V && lp_order(x[j]) == bound) {
            if (at < k) put(at, lp_key(x[j], v * P + j));
            ++at;
          }
        n += __shfl_sync(0xffffffffu, upto, 31);
      }
    }
    return;
  }
  uint64_t last = ~uint64_t{0};
  for (int rank = 0; rank < k; ++rank) {
    uint64_t best = 0;
    lp_scan(sh, row, V, seg, cands, least, [&](float x, int64_t id) {
      const uint64_t key = lp_key(x, id);
      if (key < last) best = max_u64(best, key);
    });
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) best = max_u64(best, __shfl_xor_sync(0xffffffffu, best, d));
    if (lane == 0) sh.best[warp] = best;
    __syncthreads();
    last = sh.best[0];
#pragma unroll
    for (int i = 1; i < kLpWarps; ++i) last = max_u64(last, sh.best[i]);
    if (tid == 0) put(rank, last);
    __syncthreads();
  }
}

}  // namespace

template <typename T, bool kTop, bool kCluster>
__global__ void __launch_bounds__(kLpThreads, kLpPerSm) token_logprobs_fwd_kernel(TokenLogprobsFwd p, int cluster) {
  constexpr int P = kLpPer<T>;
  extern __shared__ __align__(16) uint8_t ring[];
  LpShared& sh = *reinterpret_cast<LpShared*>(ring + kLpRing);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = kCluster ? cluster_ctarank() : 0;
  const int64_t stride = kCluster ? gridDim.x / cluster : gridDim.x;
  int64_t r = kCluster ? blockIdx.x / cluster : blockIdx.x;
  const float c2 = p.inv_temperature * kLog2e;
  LpSegment seg;
  {
    const int64_t vecs = (p.V + P - 1) / P, share = kCluster ? (vecs + cluster - 1) / cluster : vecs;
    seg.first = min(share * rank, vecs);
    seg.end = min(seg.first + share, vecs);
    seg.whole = min(seg.end, p.V / P);
  }
  const int steps = static_cast<int>((seg.end - seg.first + kLpThreads * kLpVecs - 1) / (kLpThreads * kLpVecs));
  const int full = static_cast<int>((seg.whole - seg.first) / (kLpThreads * kLpVecs));  // steps without a ragged end
  const uint32_t slots = smem_u32(ring) + tid * 16;  // this thread's; kLpThreads * 16 apart

  // The ring: step `next_step` of row `next_row` into stage `st`.
  int64_t next_row = r;
  int next_step = 0;
  const uint8_t* const start = static_cast<const uint8_t*>(p.logits) + (seg.first + tid) * 16;
  const uint8_t* src = start + r * p.ld * static_cast<int64_t>(sizeof(T));
  auto fetch = [&](int st) {
    if (next_row < p.M) {
      const uint32_t dst = slots + st * (kLpVecs * kLpThreads * 16);
      if (next_step < full) {
#pragma unroll
        for (int i = 0; i < kLpVecs; ++i)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + i * (kLpThreads * 16)),
                       "l"(src + i * (kLpThreads * 16))
                       : "memory");
      } else {
        const int64_t v0 = seg.first + static_cast<int64_t>(next_step) * (kLpThreads * kLpVecs) + tid;
#pragma unroll
        for (int i = 0; i < kLpVecs; ++i)
          if (v0 + i * kLpThreads < seg.whole)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + i * (kLpThreads * 16)),
                         "l"(src + i * (kLpThreads * 16))
                         : "memory");
      }
      src += kLpVecs * kLpThreads * 16;
      if (++next_step == steps) {
        next_step = 0, next_row += stride;
        src = start + next_row * p.ld * static_cast<int64_t>(sizeof(T));
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kLpStages; ++i) fetch(i);
  int st = 0, turn = 0;
  // Targets and their logits of 32 rows at a time, one per lane of warp 0.
  int64_t lane_t = -1;
  float lane_x = 0.0f;
  int nth = 0;

  for (; r < p.M; r += stride, turn ^= 1, nth = (nth + 1) & 31) {
    const T* row = static_cast<const T*>(p.logits) + r * p.ld;
    if (warp == 0 && rank == 0 && p.logprob != nullptr && nth == 0) {
      const int64_t mine = r + lane * stride;
      if (mine < p.M) {
        lane_t = p.targets[mine];
        if (lane_t >= 0 && lane_t < p.V) {
          const T x = static_cast<const T*>(p.logits)[mine * p.ld + lane_t];
          if constexpr (sizeof(T) == 2)
            lane_x = bf16_bits_to_float(x);
          else
            lane_x = x;
        }
      }
    }
    LpSums a{kNegInf, 0.0f, 0.0f};
    F2 s2 = splat2(0.0f), q2 = splat2(0.0f);
    float base = 0.0f;       // the maximum that t is relative to (0 while it is -inf)
    // Adds one vector; kMasked: with a lower bound on t that keeps e t = 0
    // for masked logits (t = -inf), which one more instruction per value buys.
    auto add = [&](auto masked, const uint4& u) {
      float x[P];
      lp_values<T>(u, x);
#pragma unroll
      for (int j = 0; j < P; j += 2) {
        F2 tt = mul2(add2(F2{x[j], x[j + 1]}, splat2(-base)), splat2(c2));
        if constexpr (decltype(masked)::value) tt = F2{max_nan(tt.x, -1000.0f), max_nan(tt.y, -1000.0f)};
        const F2 e{ex2(tt.x), ex2(tt.y)};
        s2 = add2(s2, e);
        q2 = fma2(e, tt, q2);
      }
    };
    float second = kNegInf;  // the largest maximum of the steps but best_step
    int best_step = 0;       // the first step with the thread's maximum
    auto raise = [&](float mx, int step) {  // take in a step's maximum
      if (mx <= a.m || a.m != a.m) {
        if (kTop) second = max_nan(second, mx);
        return;
      }
      if (kTop) second = a.m, best_step = step;
      a.s = s2.x + s2.y, a.q = q2.x + q2.y;
      a.move(mx, c2);
      s2 = F2{a.s, 0.0f}, q2 = F2{a.q, 0.0f};
      base = mx;
    };
    for (int step = 0; step < full; ++step) {
      cp_async_wait<kLpStages - 1>();
      uint4 u[kLpVecs];
#pragma unroll
      for (int i = 0; i < kLpVecs; ++i)
        u[i] = *reinterpret_cast<const uint4*>(ring + ((st * kLpVecs + i) * kLpThreads + tid) * 16);
      fetch(st);
      st = st + 1 == kLpStages ? 0 : st + 1;
      raise(lp_max<T>(u), step);
      const F2 s0 = s2, q0 = q2;
#pragma unroll
      for (int i = 0; i < kLpVecs; ++i) add(std::false_type{}, u[i]);
      if (q2.x + q2.y != q2.x + q2.y) {  // a masked logit (or a NaN, which stays one)
        s2 = s0, q2 = q0;
#pragma unroll
        for (int i = 0; i < kLpVecs; ++i) add(std::true_type{}, u[i]);
      }
    }
    if (full < steps) {  // the row's end
      const int64_t v0 = seg.first + static_cast<int64_t>(full) * (kLpThreads * kLpVecs) + tid;
      cp_async_wait<kLpStages - 1>();
#pragma unroll 1
      for (int i = 0; i < kLpVecs; ++i) {
        const int64_t vec = v0 + i * kLpThreads;
        if (vec >= seg.end) break;
        const uint4 u = vec < seg.whole
                            ? *reinterpret_cast<const uint4*>(ring + ((st * kLpVecs + i) * kLpThreads + tid) * 16)
                            : lp_load(row, p.V, vec);
        float x[P];
        lp_values<T>(u, x);
        float mx = x[0];
#pragma unroll
        for (int j = 1; j < P; ++j) mx = max_nan(mx, x[j]);
        raise(mx, full);
        add(std::true_type{}, u);
      }
      fetch(st);
      st = st + 1 == kLpStages ? 0 : st + 1;
    }
    a.s = s2.x + s2.y, a.q = q2.x + q2.y;

    const LpSums w = lp_join_lanes<32>(a, c2);
    const uint32_t order = lp_order(a.m);
    if (lane == 0) sh.warp[turn][warp] = w;
    if (kTop) sh.order[tid] = order;
    __syncthreads();
    if (warp == 0) {
      LpSums all = lp_join_lanes<kLpWarps>(sh.warp[turn][lane % kLpWarps], c2);
      if constexpr (kCluster) {
        if (lane == 0) sh.cta = all;
        __syncwarp();
        cluster_sync();  // every CTA's sums are written
        if (rank == 0) {
          all = LpSums{kNegInf, 0.0f, 0.0f};
          if (lane < cluster)
            all = LpSums{ld_cluster_f32(&sh.cta.m, lane), ld_cluster_f32(&sh.cta.s, lane), ld_cluster_f32(&sh.cta.q, lane)};
          all = lp_join_lanes<32>(all, c2);
        }
      }
      if (rank == 0) {
        const int64_t t = __shfl_sync(0xffffffffu, lane_t, nth);
        const float target = __shfl_sync(0xffffffffu, lane_x, nth);
        const bool empty = all.m == kNegInf;  // every logit is -inf
        const float log_sum = empty ? 0.0f : logf(all.s);
        const float m = empty ? 0.0f : all.m;
        if (lane == 0) {
          if (p.entropy != nullptr) p.entropy[r] = empty ? 0.0f : log_sum - all.q / all.s * kLn2;
          if (p.row_max != nullptr) p.row_max[r] = all.m;
          if (p.log_sum != nullptr) p.log_sum[r] = log_sum;
          if (p.logprob != nullptr)
            p.logprob[r] = t < 0 ? 0.0f
                           : t >= p.V ? __uint_as_float(0x7FC00000u)
                                      : (target - m) * p.inv_temperature - log_sum;
          sh.row = LpSums{m, log_sum, 0.0f};
        }
      }
    } else {
      if (kTop && warp == 1) {  // beside warp 0's joins
        const uint32_t bound = lp_threads_bound(sh, p.k, 2);
        if (lane == 0) sh.bound = bound, sh.listed[turn] = sh.deep[turn] = sh.shallow[turn] = 0;
        __syncwarp();
      }
      if constexpr (kCluster) cluster_sync();
    }
    if constexpr (kTop) {
      auto put = [&](int at, uint64_t key) {  // an alternative of the whole row
        p.top_ids[r * p.k + at] = lp_key_id(key);
        p.top_logprob[r * p.k + at] = (lp_key_value(key) - sh.row.m) * p.inv_temperature - sh.row.s;
      };
      auto keep = [&](int at, uint64_t key) {  // of this CTA's part
        if constexpr (kCluster)
          sh.top[at] = key;
        else
          put(at, key);
      };
      __syncthreads();  // sh.bound, sh.row
      const uint32_t bound = sh.bound;
      const float least = lp_least(bound);
      const bool deep = lp_order(second) >= bound;
      lp_candidates<false>(sh, order >= bound && deep, &sh.deep[turn]);
      lp_candidates<true>(sh, order >= bound && !deep, &sh.shallow[turn]);
      if (order >= bound && !deep) sh.step[tid] = best_step;
      __syncthreads();
      auto list = [&](float x, int64_t id) {
        if (lp_order(x) < bound) return;
        const int at = atomicAdd(&sh.listed[turn], 1);
        if (at < kLpList) sh.list[at] = lp_key(x, id);  // in any order: the keys are ranked
      };
#pragma unroll 1
      for (int i = tid; i < sh.shallow[turn] * kLpVecs; i += kLpThreads) {
        const int c = sh.cand[kLpThreads - 1 - i / kLpVecs];
        const int64_t v0 = seg.first + static_cast<int64_t>(sh.step[c]) * (kLpThreads * kLpVecs) + c;
        lp_scan_vector(row, p.V, seg, v0 + i % kLpVecs * kLpThreads, least, list);
      }
      lp_scan(sh, row, p.V, seg, sh.deep[turn], least, list);
      __syncthreads();
      const int n = sh.listed[turn];
      if (n <= kLpList)
        lp_rank_list(sh, n, p.k, tid, kLpThreads, keep);
      else
        lp_select_many<T>(sh, row, p.V, seg, p.k, order, turn, keep);
      if constexpr (kCluster) {
        __syncwarp();
        cluster_sync();  // every CTA's keys are written
        if (rank == 0 && warp == 0) {
          uint64_t key[kLpMaxCluster];
          uint32_t first[kLpMaxCluster];
#pragma unroll
          for (int i = 0; i < kLpMaxCluster; ++i) {
            key[i] = i < cluster && lane < p.k ? ld_cluster_u64(&sh.top[lane], i) : 0;
            first[i] = static_cast<uint32_t>(key[i] >> 32);
          }
          const uint32_t least = lp_bound(first, p.k, 8);
          int count = 0;
#pragma unroll
          for (int i = 0; i < kLpMaxCluster; ++i) {
            const bool in = first[i] >= least && key[i] != 0;
            const uint32_t any = __ballot_sync(0xffffffffu, in);
            if (in) sh.list[count + __popc(any & ((1u << lane) - 1u))] = key[i];
            count += __popc(any);
          }
          __syncwarp();
          lp_rank_list(sh, count, p.k, lane, 32, put);
        }
      }
    }
    if constexpr (kCluster) {
      __syncwarp();
      cluster_sync();  // the other CTAs' shared memory is read no more
    }
  }
  cp_async_wait<0>();
}

// dx = p (A - B log p), and c g more at the target, with t = log2 p:
// t = (x - m) c log2 e - log s log2 e.
template <typename T>
__global__ void __launch_bounds__(kLpThreads) token_logprobs_bwd_kernel(TokenLogprobsBwd p) {
  constexpr int P = kLpPer<T>;
  const int64_t r = blockIdx.x / p.chunks;
  const int64_t v0 = (blockIdx.x % p.chunks) * (kLpThreads * kLpVecs) + threadIdx.x;
  const T* row = static_cast<const T*>(p.logits) + r * p.ld;
  T* out = static_cast<T*>(p.dlogits) + r * p.ldd;
  uint4 u[kLpVecs];
#pragma unroll
  for (int i = 0; i < kLpVecs; ++i) u[i] = lp_load(row, p.V, v0 + i * kLpThreads);
  const float c = p.inv_temperature;
  const float m = p.row_max[r], log_sum = p.log_sum[r];
  const int64_t target = p.targets != nullptr ? p.targets[r] : -1;
  float g = p.g_logprob != nullptr && target >= 0 ? p.g_logprob[r] : 0.0f;
  if (target >= p.V) g = __uint_as_float(0x7FC00000u);
  const float gh = p.g_entropy != nullptr ? p.g_entropy[r] : 0.0f;
  const F2 A = splat2(-c * (g + (p.g_entropy != nullptr ? gh * p.entropy[r] : 0.0f))), B = splat2(-c * gh * kLn2);
  const F2 minus = splat2(-m), c2 = splat2(c * kLog2e), shift = splat2(-log_sum * kLog2e);
  const bool empty = m == kNegInf;
  const float empty_row = target >= p.V ? g : 0.0f;  // NaN, as everywhere for such a target
#pragma unroll
  for (int i = 0; i < kLpVecs; ++i) {
    const int64_t vec = v0 + i * kLpThreads, first = vec * P;
    if (first >= p.V) return;
    float x[P];
    lp_values<T>(u[i], x);
#pragma unroll
    for (int j = 0; j < P; j += 2) {
      F2 t = fma2(add2(F2{x[j], x[j + 1]}, minus), c2, shift);
      t = F2{max_nan(t.x, -1000.0f), max_nan(t.y, -1000.0f)};  // p = 0 there, and 0 log 0 = 0
      const F2 d = mul2(F2{ex2(t.x), ex2(t.y)}, fma2(B, t, A));
      x[j] = d.x, x[j + 1] = d.y;
    }
    if (target >= first && target < first + P) {
#pragma unroll
      for (int j = 0; j < P; ++j)
        if (first + j == target) x[j] += c * g;
    }
    if (empty) {  // every logit is -inf
#pragma unroll
      for (int j = 0; j < P; ++j) x[j] = empty_row;
    }
    if (first + P <= p.V) {
      if constexpr (sizeof(T) == 2)
        *reinterpret_cast<uint4*>(out + first) =
            make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
      else
        *reinterpret_cast<float4*>(out + first) = make_float4(x[0], x[1], x[2], x[3]);
    } else {
#pragma unroll
      for (int j = 0; j < P; ++j) {
        if (first + j >= p.V) continue;
        if constexpr (sizeof(T) == 2)
          out[first + j] = static_cast<uint16_t>(pack_bf16x2(x[j], 0.0f) & 0xFFFFu);
        else
          out[first + j] = x[j];
      }
    }
  }
}

namespace {

template <typename T, bool kTop, bool kCluster>
cudaError_t launch_fwd(const TokenLogprobsFwd& p, int cluster, cudaStream_t stream) {
  constexpr int smem = kLpRing + static_cast<int>(sizeof(LpShared));
  const auto kernel = token_logprobs_fwd_kernel<T, kTop, kCluster>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  static DeviceOnce configured;
  e = configured.run(dev, [&] { return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem); });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t config{};
  const int64_t rows = kCluster ? p.M : std::min<int64_t>(p.M, 148 * kLpPerSm);
  config.gridDim = dim3(static_cast<unsigned>(rows * cluster));
  config.blockDim = dim3(kLpThreads);
  config.dynamicSmemBytes = smem;
  config.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {static_cast<unsigned>(cluster), 1, 1};
  config.attrs = attr;
  config.numAttrs = kCluster ? 1 : 0;
  return cudaLaunchKernelEx(&config, kernel, p, cluster);
}

template <typename T>
cudaError_t launch_fwd_type(const TokenLogprobsFwd& p, cudaStream_t stream) {
  // CTAs per row: a power of two that keeps the machine's CTA slots filled
  // without a second wave, and gives each CTA a full step at least.
  const int64_t step = kLpThreads * kLpVecs * kLpPer<T>;
  int cluster = 1;
  while (cluster < kLpMaxCluster && p.M * cluster * 2 <= 148 * kLpPerSm && p.V >= step * cluster * 2) cluster *= 2;
  if (p.k > 0)
    return cluster > 1 ? launch_fwd<T, true, true>(p, cluster, stream) : launch_fwd<T, true, false>(p, 1, stream);
  return cluster > 1 ? launch_fwd<T, false, true>(p, cluster, stream) : launch_fwd<T, false, false>(p, 1, stream);
}

}  // namespace

cudaError_t launch_token_logprobs_fwd(const TokenLogprobsFwd& p, int fp32, cudaStream_t stream) {
  return fp32 ? launch_fwd_type<float>(p, stream) : launch_fwd_type<uint16_t>(p, stream);
}

cudaError_t launch_token_logprobs_bwd(TokenLogprobsBwd p, int fp32, cudaStream_t stream) {
  const int64_t per = kLpThreads * kLpVecs * (fp32 ? kLpPer<float> : kLpPer<uint16_t>);
  p.chunks = (p.V + per - 1) / per;
  const unsigned grid = static_cast<unsigned>(p.M * p.chunks);
  if (fp32)
    token_logprobs_bwd_kernel<float><<<grid, kLpThreads, 0, stream>>>(p);
  else
    token_logprobs_bwd_kernel<uint16_t><<<grid, kLpThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace qnf4
