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
// HBM-bound: 2 or 4 bytes per logit against about 8 instructions.  The k
// largest come from the same pass: a thread's running maximum is one
// candidate key (value, lowest id first); the k-th largest of the keys is a
// bound that at least k logits reach, and only the threads whose key reaches
// it are looked through once more (their logits are in L2).
//
// The gradient  dx_j = c (g (1[j = t] - p_j) - g_H p_j (log p_j + H)) is
// elementwise from the saved m, log s and H: one read, one write.
#include "common.cuh"
#include "kernels.cuh"

namespace qnf4 {

namespace {

constexpr int kLpThreads = 256;
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kLpVecs = 4;       // 16-byte vectors per thread and step
constexpr int kLpGroup = 4;      // threads whose keys are joined before the bound is chosen
constexpr int kLpList = 256;     // logits at or above the bound that are ranked directly
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

// (value, id) as one key: larger values first, the lower id first among
// equals (-0 = 0), NaN above everything.  0 is below every key.
__device__ __forceinline__ uint64_t lp_key(float v, int64_t id) {
  const uint32_t u = __float_as_uint(v + 0.0f);
  const uint32_t order = v != v ? 0xFFFFFFFFu : (u >> 31) ? ~u : (u | 0x80000000u);
  return (static_cast<uint64_t>(order) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(id));
}

__device__ __forceinline__ float lp_key_value(uint64_t key) {
  const uint32_t order = static_cast<uint32_t>(key >> 32);
  if (order == 0xFFFFFFFFu) return __uint_as_float(0x7FC00000u);
  return __uint_as_float((order >> 31) ? (order & 0x7FFFFFFFu) : ~order);
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
  __device__ __forceinline__ void join(LpSums o, float c2) {
    const float to = max_nan(m, o.m);
    move(to, c2);
    o.move(to, c2);
    s += o.s;
    q += o.q;
  }
};

struct LpShared {
  LpSums warp[kLpWarps];
  LpSums row;
  uint64_t thread_key[kLpThreads];
  uint64_t group_key[kLpThreads / kLpGroup];
  uint64_t list[kLpList];
  uint64_t bound;
  uint64_t best[kLpWarps];
  int cand[kLpThreads];
  int cands, listed;
};

}  // namespace

template <typename T>
__global__ void __launch_bounds__(kLpThreads) token_logprobs_fwd_kernel(TokenLogprobsFwd p) {
  constexpr int P = kLpPer<T>;
  __shared__ LpShared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t r = blockIdx.x;
  const T* row = static_cast<const T*>(p.logits) + r * p.ld;
  const int64_t vecs = (p.V + P - 1) / P;
  const float c2 = p.inv_temperature * kLog2e;

  LpSums a{kNegInf, 0.0f, 0.0f};
  float base = 0.0f;       // the maximum that t is relative to (0 while it is -inf)
  int64_t best_step = -1;  // first vector of the step that holds the thread's maximum first
  for (int64_t v0 = tid; v0 < vecs; v0 += kLpThreads * kLpVecs) {
    uint4 u[kLpVecs];
#pragma unroll
    for (int i = 0; i < kLpVecs; ++i) u[i] = lp_load(row, p.V, v0 + i * kLpThreads);
    float x[kLpVecs][P];
    float mx = kNegInf;
#pragma unroll
    for (int i = 0; i < kLpVecs; ++i) {
      lp_values<T>(u[i], x[i]);
#pragma unroll
      for (int j = 0; j < P; ++j) mx = max_nan(mx, x[i][j]);
    }
    if (best_step < 0 || (!(mx <= a.m) && a.m == a.m)) {
      best_step = v0;
      a.move(mx, c2);
      base = mx == kNegInf ? 0.0f : mx;
    }
#pragma unroll
    for (int i = 0; i < kLpVecs; ++i)
#pragma unroll
      for (int j = 0; j < P; ++j) {
        // Masked logits give t = -inf: a finite bound keeps e t = 0 there.
        const float t = max_nan((x[i][j] - base) * c2, -1000.0f);
        const float e = ex2(t);
        a.s += e;
        a.q = fmaf(e, t, a.q);
      }
  }

  LpSums w = a;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    LpSums o{__shfl_xor_sync(0xffffffffu, w.m, d), __shfl_xor_sync(0xffffffffu, w.s, d),
             __shfl_xor_sync(0xffffffffu, w.q, d)};
    w.join(o, c2);
  }
  if (lane == 0) sh.warp[warp] = w;
  if (tid == 0) sh.cands = sh.listed = 0;
  __syncthreads();
  if (tid == 0) {
    LpSums all = sh.warp[0];
    for (int i = 1; i < kLpWarps; ++i) all.join(sh.warp[i], c2);
    const bool empty = all.m == kNegInf;  // every logit is -inf
    const float log_sum = empty ? 0.0f : logf(all.s);
    if (p.entropy != nullptr) p.entropy[r] = empty ? 0.0f : log_sum - all.q / all.s * kLn2;
    if (p.row_max != nullptr) p.row_max[r] = all.m;
    if (p.log_sum != nullptr) p.log_sum[r] = log_sum;
    if (p.logprob != nullptr) {
      const int64_t t = p.targets[r];
      float v = 0.0f;
      if (t >= p.V) {
        v = __uint_as_float(0x7FC00000u);
      } else if (t >= 0) {
        float x;
        if constexpr (sizeof(T) == 2)
          x = bf16_bits_to_float(row[t]);
        else
          x = row[t];
        v = (x - (empty ? 0.0f : all.m)) * p.inv_temperature - log_sum;
      }
      p.logprob[r] = v;
    }
    sh.row = LpSums{empty ? 0.0f : all.m, log_sum, 0.0f};
  }
  if (p.k == 0) return;

  // The thread's key: its maximum and the first id that has it.
  uint64_t key = 0;
  if (best_step >= 0) {
    for (int i = kLpVecs - 1; i >= 0; --i) {
      float x[P];
      const int64_t vec = best_step + i * kLpThreads;
      lp_values<T>(lp_load(row, p.V, vec), x);
#pragma unroll
      for (int j = P - 1; j >= 0; --j)
        if (vec * P + j < p.V && (x[j] == a.m || x[j] != x[j])) key = lp_key(x[j], vec * P + j);
    }
  }
  sh.thread_key[tid] = key;
  uint64_t gk = key;
#pragma unroll
  for (int d = 1; d < kLpGroup; d *= 2) {
    const uint64_t o = __shfl_xor_sync(0xffffffffu, gk, d);
    gk = o > gk ? o : gk;
  }
  if (tid % kLpGroup == 0) sh.group_key[tid / kLpGroup] = gk;
  __syncthreads();
  // The k-th largest group key (keys differ: each holds its own id; empty groups' zeros rank last).
  if (tid < kLpThreads / kLpGroup) {
    const uint64_t mine = sh.group_key[tid];
    int above = 0;
#pragma unroll 8
    for (int i = 0; i < kLpThreads / kLpGroup; ++i) above += sh.group_key[i] > mine || (sh.group_key[i] == mine && i < tid);
    if (above == p.k - 1) sh.bound = mine;
  }
  __syncthreads();
  const uint64_t bound = sh.bound > 0 ? sh.bound : 1;
  if (key >= bound) sh.cand[atomicAdd(&sh.cands, 1)] = tid;
  __syncthreads();
  // Every logit of the candidate threads that reaches the bound.
  const int64_t per = (vecs + kLpThreads - 1) / kLpThreads;
  const int64_t items = static_cast<int64_t>(sh.cands) * per;
  for (int64_t i = tid; i < items; i += kLpThreads) {
    const int64_t vec = sh.cand[i / per] + (i % per) * kLpThreads;
    float x[P];
    lp_values<T>(lp_load(row, p.V, vec), x);
#pragma unroll
    for (int j = 0; j < P; ++j) {
      const uint64_t k = lp_key(x[j], vec * P + j);
      if (vec * P + j < p.V && k >= bound) {
        const int at = atomicAdd(&sh.listed, 1);
        if (at < kLpList) sh.list[at] = k;
      }
    }
  }
  __syncthreads();
  int32_t* ids = p.top_ids + r * p.k;
  float* lps = p.top_logprob + r * p.k;
  auto put = [&](int rank, uint64_t k) {
    ids[rank] = lp_key_id(k);
    lps[rank] = (lp_key_value(k) - sh.row.m) * p.inv_temperature - sh.row.s;
  };
  const int n = sh.listed;
  if (n <= kLpList) {
    if (tid < n) {
      const uint64_t mine = sh.list[tid];
      int above = 0;
      for (int i = 0; i < n; ++i) above += sh.list[i] > mine;
      if (above < p.k) put(above, mine);
    }
    return;
  }
  // Too many to rank (the largest logits sit in few threads): take the
  // largest key below the last one, k times.
  uint64_t last = ~uint64_t{0};
  for (int rank = 0; rank < p.k; ++rank) {
    uint64_t best = 0;
    for (int64_t i = tid; i < items; i += kLpThreads) {
      const int64_t vec = sh.cand[i / per] + (i % per) * kLpThreads;
      float x[P];
      lp_values<T>(lp_load(row, p.V, vec), x);
#pragma unroll
      for (int j = 0; j < P; ++j) {
        const uint64_t k = lp_key(x[j], vec * P + j);
        if (vec * P + j < p.V && k < last && k > best) best = k;
      }
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      const uint64_t o = __shfl_xor_sync(0xffffffffu, best, d);
      best = o > best ? o : best;
    }
    if (lane == 0) sh.best[warp] = best;
    __syncthreads();
    last = sh.best[0];
    for (int i = 1; i < kLpWarps; ++i) last = sh.best[i] > last ? sh.best[i] : last;
    if (tid == 0) put(rank, last);
    __syncthreads();
  }
}

template <typename T>
__global__ void __launch_bounds__(kLpThreads) token_logprobs_bwd_kernel(TokenLogprobsBwd p) {
  constexpr int P = kLpPer<T>;
  const int64_t r = blockIdx.x / p.chunks;
  const int64_t v0 = (blockIdx.x % p.chunks) * (kLpThreads * kLpVecs) + threadIdx.x;
  const T* row = static_cast<const T*>(p.logits) + r * p.ld;
  T* out = static_cast<T*>(p.dlogits) + r * p.ldd;
  const float c = p.inv_temperature;
  const float m = p.row_max[r], log_sum = p.log_sum[r];
  const int64_t t = p.targets != nullptr ? p.targets[r] : -1;
  const bool empty = m == kNegInf;
  float g = p.g_logprob != nullptr && t >= 0 ? p.g_logprob[r] : 0.0f;
  if (t >= p.V) g = __uint_as_float(0x7FC00000u);
  const float gh = p.g_entropy != nullptr ? p.g_entropy[r] : 0.0f;
  // dx = p (A - B log p), and c g more at the target.
  const float A = -c * (g + (p.g_entropy != nullptr ? gh * p.entropy[r] : 0.0f)), B = c * gh;
#pragma unroll
  for (int i = 0; i < kLpVecs; ++i) {
    const int64_t vec = v0 + i * kLpThreads, first = vec * P;
    if (first >= p.V) return;
    float x[P];
    lp_values<T>(lp_load(row, p.V, vec), x);
#pragma unroll
    for (int j = 0; j < P; ++j) {
      const float lp = max_nan((x[j] - m) * c - log_sum, -1000.0f);  // p = 0 there, and 0 log 0 = 0
      float d = ex2(lp * kLog2e) * (A - B * lp);
      if (first + j == t) d += c * g;
      x[j] = empty ? 0.0f : d;
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

cudaError_t launch_token_logprobs_fwd(const TokenLogprobsFwd& p, int fp32, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>(p.M);
  if (fp32)
    token_logprobs_fwd_kernel<float><<<grid, kLpThreads, 0, stream>>>(p);
  else
    token_logprobs_fwd_kernel<uint16_t><<<grid, kLpThreads, 0, stream>>>(p);
  return cudaGetLastError();
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
