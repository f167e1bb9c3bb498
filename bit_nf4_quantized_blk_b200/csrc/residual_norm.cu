// The pass between two blocks of a network (sm_100a): the norm after a block,
// its gate and residual scale, the residual sum and the norm before the next
// block, and its backward.
//
// Per row of D values, with rstd(v) = 1 / sqrt(mean(v^2) + eps):
//   p = y rstd(y) w_post           (p = y without w_post)
//   v = h + scale gate p           (gate = 1 without one; v = h without y)
//   h_out = round(v),  x = v rstd(v) w_pre,  optionally x's 8-bit checkpoint
// Backward, for upstream gradients dh_out of h_out and dx of x, with
// n = h_out rstd(v), m = y rstd(y):
//   g = dh_out + rstd(v) (dx w_pre - n mean(dx w_pre n)),   dh = g
//   dw_pre = sum_rows dx n,   dgate = sum_rows scale g p
//   dp = scale g gate,        dw_post = sum_rows dp m
//   dy = rstd(y) (dp w_post - m mean(dp w_post m))          (dy = dp without w_post)
//
// Every operand is touched once, so the bound is HBM: a row lives in the
// registers of its threads between the two reductions, and nothing is read
// twice.  A thread holds NC groups of 8 consecutive values, TPR groups apart
// (16-byte accesses, lanes side by side; 8 lanes hold one 64-value checkpoint
// block).  Rows of up to 512 values (256 of an fp32 stream) take one warp
// (reductions by shuffles alone), longer ones a CTA.  All arithmetic is fp32.
// CTAs stay for many rows: while a row is computed, the next one's operands
// travel to shared memory (cp.async), so the two reductions' waits do not stop
// the loads.  Measured, bf16, 8192 x 4096: forward with a checkpoint 56 to 59 us
// (303 MB, 5.1 to 5.4 TB/s; the barriers' waits are the largest stall), backward
// with every gradient 70 to 72 us (403 MB, 5.6 TB/s); an fp32 stream of 999 x
// 2048: backward 16.4 us, of which 36 MB would take 5.6.
//
// The backward's column sums stay in registers over all rows of a CTA; each
// CTA writes one partial row and residual_norm_finish_kernel adds those in a
// fixed order (no atomics).
#include <algorithm>
#include <type_traits>

#include "act8.cuh"
#include "kernels.cuh"

namespace qnf4 {

namespace {

constexpr int kWarpRowCtas = 8;  // rows (warps) of a CTA when a warp takes a row

template <int TPR>
constexpr int kNormThreads = TPR == 32 ? 32 * kWarpRowCtas : TPR;

// Threads that share an SM: what the registers allow (64 and 128 per thread).
constexpr int kFwdResident = 1024, kBwdResident = 512;

// Whether the backward keeps its channel factors in shared memory: read from
// L1 for every row their latency was a third of its stalls.  The longest rows
// leave no room.
template <int TPR>
constexpr bool kStash = TPR <= 512;

template <int TPR, int kResident>
constexpr int kMinCtas = kNormThreads<TPR> >= kResident ? 1 : kResident / kNormThreads<TPR>;

// Sum over the TPR threads of a row, the same in each of them.  `slots`: one
// float per warp, a different array for consecutive calls of a row.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* slots) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  if constexpr (TPR > 32) {
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) slots[warp] = v;
    __syncthreads();
    v = 0.0f;
    if constexpr (TPR == 64) {
      const float2 s = *reinterpret_cast<const float2*>(slots);
      v = s.x + s.y;
    } else {
      float u[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int w = 0; w < TPR / 32; w += 4) {
        const float4 s = *reinterpret_cast<const float4*>(slots + w);
        u[0] += s.x, u[1] += s.y, u[2] += s.z, u[3] += s.w;
      }
      v = (u[0] + u[1]) + (u[2] + u[3]);
    }
  }
  return v;
}

// Eight consecutive values are four pairs throughout.
__device__ __forceinline__ void unpack8(const uint4& u, F2 (&v)[4]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = F2{__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u)};
}

__device__ __forceinline__ uint4 pack8(const F2 (&v)[4]) {
  return make_uint4(pack_bf16x2(v[0].x, v[0].y), pack_bf16x2(v[1].x, v[1].y), pack_bf16x2(v[2].x, v[2].y),
                    pack_bf16x2(v[3].x, v[3].y));
}

// Eight values at element offset `at`.
__device__ __forceinline__ void load8(const float* p, int64_t at, F2 (&v)[4]) {
  const float4 a = *reinterpret_cast<const float4*>(p + at), b = *reinterpret_cast<const float4*>(p + at + 4);
  v[0] = F2{a.x, a.y}, v[1] = F2{a.z, a.w}, v[2] = F2{b.x, b.y}, v[3] = F2{b.z, b.w};
}
__device__ __forceinline__ void store8(uint16_t* p, int64_t at, const F2 (&v)[4]) {
  *reinterpret_cast<uint4*>(p + at) = pack8(v);
}
__device__ __forceinline__ void store8(float* p, int64_t at, const F2 (&v)[4]) {
  *reinterpret_cast<float4*>(p + at) = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
  *reinterpret_cast<float4*>(p + at + 4) = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
}

// A thread's share of one tensor's next row: copied to shared memory
// asynchronously, read back by the same thread (so it needs no barrier), into
// 16-byte slots kThreads apart (no bank conflicts).  Slots past the row's end
// are zero-filled.
template <typename T, int TPR, int NC>
struct RowSlot {
  static constexpr int kVecs = NC * static_cast<int>(sizeof(T)) / 2;  // 16-byte vectors
  static constexpr int kThreads = kNormThreads<TPR>;
  static constexpr int kBytes = kVecs * kThreads * 16;

  __device__ static __forceinline__ void fetch(uint8_t* slot, const T* row, int tid, int64_t D, bool live) {
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int at = (c * TPR + tid) * 8;
      const bool ok = live && at < D;
#pragma unroll
      for (int q = 0; q < kVecs / NC; ++q)
        cp_async_16(slot + ((c * (kVecs / NC) + q) * kThreads + threadIdx.x) * 16,
                    ok ? row + at + q * (16 / static_cast<int>(sizeof(T))) : row, ok);
    }
  }
  __device__ static __forceinline__ void write(uint8_t* slot, int c, const F2 (&v)[4]) {
    static_assert(sizeof(T) == 4, "fp32 slots");
    float4* s = reinterpret_cast<float4*>(slot) + c * (kVecs / NC) * kThreads + threadIdx.x;
    s[0] = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
    s[kThreads] = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
  }
  __device__ static __forceinline__ void read(const uint8_t* slot, int c, F2 (&v)[4]) {
    const uint4* s = reinterpret_cast<const uint4*>(slot) + c * (kVecs / NC) * kThreads + threadIdx.x;
    if constexpr (sizeof(T) == 2) {
      unpack8(*s, v);
    } else {
      const uint4 a = s[0], b = s[kThreads];
      v[0] = F2{__uint_as_float(a.x), __uint_as_float(a.y)}, v[1] = F2{__uint_as_float(a.z), __uint_as_float(a.w)};
      v[2] = F2{__uint_as_float(b.x), __uint_as_float(b.y)}, v[3] = F2{__uint_as_float(b.z), __uint_as_float(b.w)};
    }
  }
};

// w_pre (0 unless `has_pre`) and scale gate w_post of the eight channels at `at`.
template <typename Params>
__device__ __forceinline__ void read_factors(const Params& p, int at, bool has_pre, F2 (&pre)[4], F2 (&branch)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) pre[i] = splat2(0.0f), branch[i] = splat2(p.scale);
  if (at < p.D) {
    F2 f[4];
    if (p.w_post != nullptr) {
      load8(p.w_post, at, f);
#pragma unroll
      for (int i = 0; i < 4; ++i) branch[i] = mul2(branch[i], f[i]);
    }
    if (p.gate != nullptr) {
      load8(p.gate, at, f);
#pragma unroll
      for (int i = 0; i < 4; ++i) branch[i] = mul2(branch[i], f[i]);
    }
    if (has_pre) load8(p.w_pre, at, pre);
  }
}

}  // namespace

template <typename TRes, int TPR, int NC>
__global__ void __launch_bounds__(kNormThreads<TPR>, kMinCtas<TPR, kFwdResident>)
    residual_norm_fwd_kernel(ResidualNormFwd p) {
  using H = RowSlot<TRes, TPR, NC>;
  using Y = RowSlot<uint16_t, TPR, NC>;
  constexpr int kRows = kNormThreads<TPR> / TPR;
  extern __shared__ __align__(16) uint8_t slots_h[];
  uint8_t* slots_y = slots_h + H::kBytes;
  using W = RowSlot<float, TPR, NC>;
  uint8_t* factor_pre = slots_y + Y::kBytes;
  uint8_t* factor_branch = factor_pre + W::kBytes;
  __shared__ __align__(16) float sums[4][32];
  const int tid = threadIdx.x % TPR;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kRows;
  int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / TPR;
  const TRes* h = static_cast<const TRes*>(p.h);
  TRes* h_out = static_cast<TRes*>(p.h_out);
  const float inv_d = 1.0f / static_cast<float>(p.D);

  auto fetch = [&](int64_t next) {
    const bool live = next < p.M;
    const int64_t at = live ? next * p.D : 0;
    H::fetch(slots_h, h + at, tid, p.D, live);
    if (p.y != nullptr) Y::fetch(slots_y, p.y + at, tid, p.D, live);
    cp_async_commit();
  };
  fetch(row);
  // w_pre and the branch's factor scale gate w_post, each thread's own share, in
  // shared memory: read from L1 for every row they were half of the kernel's L1
  // traffic, and in registers they cost a quarter of the resident threads
  // (8192 x 4096 with a checkpoint: 60 us, so 56 to 59).
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    F2 pre[4], branch[4];
    read_factors(p, (c * TPR + tid) * 8, p.w_pre != nullptr, pre, branch);
    W::write(factor_pre, c, pre);
    W::write(factor_branch, c, branch);
  }
  int turn = 0;  // row_sum arrays alternate from row to row: a row's are written again two barriers later
  for (; row < p.M; row += stride, turn ^= 1) {
    const int64_t base = row * p.D;
    cp_async_wait<0>();
    F2 v[NC][4], y[NC][4];
    F2 ss = splat2(0.0f);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      H::read(slots_h, c, v[c]);
      if (p.y != nullptr) {
        Y::read(slots_y, c, y[c]);
#pragma unroll
        for (int i = 0; i < 4; ++i) ss = fma2(y[c][i], y[c][i], ss);
      }
    }
    fetch(row + stride);  // into the slots just read
    if (p.y != nullptr) {
      float rstd = 1.0f;
      if (p.w_post != nullptr) {
        rstd = rsqrtf(row_sum<TPR>(ss.x + ss.y, sums[2 * turn]) * inv_d + p.eps);
        if (p.rstd_post != nullptr && tid == 0) p.rstd_post[row] = rstd;
      }
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        F2 branch[4];
        W::read(factor_branch, c, branch);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[c][i] = fma2(mul2(y[c][i], splat2(rstd)), branch[i], v[c][i]);
      }
    }
    if (h_out != nullptr) {
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int at = (c * TPR + tid) * 8;
        if (at < p.D) store8(h_out, base + at, v[c]);
      }
    }
    if (p.x == nullptr) continue;
    ss = splat2(0.0f);
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) ss = fma2(v[c][i], v[c][i], ss);
    const float rstd = rsqrtf(row_sum<TPR>(ss.x + ss.y, sums[2 * turn + 1]) * inv_d + p.eps);
    if (p.rstd_pre != nullptr && tid == 0) p.rstd_pre[row] = rstd;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int at = (c * TPR + tid) * 8;
      uint4 x = make_uint4(0, 0, 0, 0);
      if (at < p.D) {
        F2 w_pre[4];
        W::read(factor_pre, c, w_pre);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[c][i] = mul2(mul2(v[c][i], splat2(rstd)), w_pre[i]);
        x = pack8(v[c]);
        *reinterpret_cast<uint4*>(p.x + base + at) = x;
      }
      if (p.codes != nullptr) {  // the checkpoint is of x as stored; 8 lanes hold a block
        uint32_t m = absmax_bf16x2(absmax_bf16x2(absmax_bf16x2(x.x & 0x7FFF7FFFu, x.y), x.z), x.w);
        m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 2));
        m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 4));
        m = max(m & 0xFFFFu, m >> 16);
        uint2 q;
        uint32_t step;
        if (p.format == kAct8Int8) {
          const Act8Encoder<kAct8Int8> enc(m);
          q = enc.encode8(x), step = enc.step;
        } else {
          const Act8Encoder<kAct8E4m3> enc(m);
          q = enc.encode8(x), step = enc.step;
        }
        if (at < p.D) {
          *reinterpret_cast<uint2*>(p.codes + base + at) = q;
          if ((tid & 7) == 0) p.step[(base + at) / kBlock] = static_cast<uint16_t>(step);
        }
      }
    }
  }
  cp_async_wait<0>();
}

template <typename TRes, int TPR, int NC>
__global__ void __launch_bounds__(kNormThreads<TPR>, kMinCtas<TPR, kBwdResident>)
    residual_norm_bwd_kernel(ResidualNormBwd p) {
  using H = RowSlot<TRes, TPR, NC>;
  using Y = RowSlot<uint16_t, TPR, NC>;
  constexpr int kRows = kNormThreads<TPR> / TPR;
  extern __shared__ __align__(16) uint8_t slots_dh[];
  uint8_t* slots_h = slots_dh + H::kBytes;
  uint8_t* slots_dx = slots_h + H::kBytes;
  uint8_t* slots_y = slots_dx + Y::kBytes;
  using W = RowSlot<float, TPR, NC>;
  uint8_t* factor_pre = slots_y + Y::kBytes;
  uint8_t* factor_branch = factor_pre + W::kBytes;
  __shared__ __align__(16) float sums[4][32];
  const int tid = threadIdx.x % TPR;
  pdl_launch_dependents();
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kRows;
  int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / TPR;
  const TRes* dh_out = static_cast<const TRes*>(p.dh_out);
  const TRes* h_out = static_cast<const TRes*>(p.h_out);
  TRes* dh = static_cast<TRes*>(p.dh);
  const float inv_d = 1.0f / static_cast<float>(p.D);
  const bool need_y = p.w_post != nullptr || p.dgate;  // else dy = scale gate g alone
  const bool branch = p.dy != nullptr || p.dgate || p.dw_post;

  // Two groups of copies per row, each refilled as soon as it is read.
  auto fetch = [&](int64_t next) {
    const bool live = next < p.M;
    const int64_t at = live ? next * p.D : 0;
    if (dh_out != nullptr) H::fetch(slots_dh, dh_out + at, tid, p.D, live);
    if (p.dx != nullptr) {
      H::fetch(slots_h, h_out + at, tid, p.D, live);
      Y::fetch(slots_dx, p.dx + at, tid, p.D, live);
    }
    cp_async_commit();
  };
  auto fetch_y = [&](int64_t next) {
    const bool live = next < p.M;
    if (need_y) Y::fetch(slots_y, p.y + (live ? next * p.D : 0), tid, p.D, live);
    cp_async_commit();
  };

  F2 s_pre[NC][4], s_branch[NC][4];  // column sums of dx n and of g m
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i) s_pre[c][i] = s_branch[c][i] = splat2(0.0f);

  // The row scalars of 32 rows at a time, one per lane.  Loaded row by row,
  // even a row ahead, their waits also held up the copies in flight (a fifth
  // of the kernel's time).
  const int lane = threadIdx.x & 31;
  float lane_pre = 0.0f, lane_post = 1.0f;
  auto fetch_rstd = [&](int64_t first) {
    const int64_t r = first + lane * stride;
    if (r >= p.M) return;
    if (p.dx != nullptr) lane_pre = p.rstd_pre[r];
    if (p.w_post != nullptr) lane_post = p.rstd_post[r];
  };
  fetch(row);
  fetch_y(row);
  // w_pre and the branch's factor scale gate w_post, each thread's own share.
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    F2 f[4], b[4];
    read_factors(p, (c * TPR + tid) * 8, p.dx != nullptr, f, b);
    if constexpr (kStash<TPR>) {
      W::write(factor_pre, c, f);
      W::write(factor_branch, c, b);
    }
  }
  int turn = 0;  // row_sum arrays alternate from row to row: a row's are written again two barriers later
  int nth = 0;   // of 32 rows
  for (; row < p.M; row += stride, turn ^= 1, nth = (nth + 1) & 31) {
    const int64_t base = row * p.D;
    if (nth == 0) fetch_rstd(row);
    F2 g[NC][4], dn[NC][4], n[NC][4], w[NC][4];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      F2 other[4];
      if constexpr (kStash<TPR>)
        W::read(factor_pre, c, w[c]);
      else
        read_factors(p, (c * TPR + tid) * 8, p.dx != nullptr, w[c], other);
    }
    cp_async_wait<1>();
#pragma unroll
    for (int c = 0; c < NC; ++c) {
#pragma unroll
      for (int i = 0; i < 4; ++i) g[c][i] = splat2(0.0f);
      if (dh_out != nullptr) H::read(slots_dh, c, g[c]);
      if (p.dx != nullptr) {
        H::read(slots_h, c, n[c]);
        Y::read(slots_dx, c, dn[c]);
      }
    }
    fetch(row + stride);
    const float rstd_pre = __shfl_sync(0xffffffffu, lane_pre, nth);
    const float rstd_post = __shfl_sync(0xffffffffu, lane_post, nth);
    if (p.dx != nullptr) {
      F2 dots = splat2(0.0f);
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          n[c][i] = mul2(n[c][i], splat2(rstd_pre));
          s_pre[c][i] = fma2(dn[c][i], n[c][i], s_pre[c][i]);
          dn[c][i] = mul2(dn[c][i], w[c][i]);
          dots = fma2(dn[c][i], n[c][i], dots);
        }
      const float dot = row_sum<TPR>(dots.x + dots.y, sums[2 * turn]) * inv_d;
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          g[c][i] = fma2(splat2(rstd_pre), fma2(n[c][i], splat2(-dot), dn[c][i]), g[c][i]);
    }
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      F2 other[4];
      if constexpr (kStash<TPR>)
        W::read(factor_branch, c, w[c]);
      else
        read_factors(p, (c * TPR + tid) * 8, p.dx != nullptr, other, w[c]);
    }
    if (dh != nullptr) {
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int at = (c * TPR + tid) * 8;
        if (at < p.D) store8(dh, base + at, g[c]);
      }
    }
    if (!branch) {
      cp_async_commit();  // keeps the two groups per row
      continue;
    }
    cp_async_wait<1>();
    F2 m[NC][4];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
#pragma unroll
      for (int i = 0; i < 4; ++i) m[c][i] = splat2(0.0f);
      if (need_y) Y::read(slots_y, c, m[c]);
    }
    fetch_y(row + stride);
    F2 dots = splat2(0.0f);
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        m[c][i] = mul2(m[c][i], splat2(rstd_post));
        s_branch[c][i] = fma2(g[c][i], m[c][i], s_branch[c][i]);
        g[c][i] = mul2(g[c][i], w[c][i]);
        dots = fma2(g[c][i], m[c][i], dots);
      }
    if (p.w_post != nullptr) {
      const float dot = row_sum<TPR>(dots.x + dots.y, sums[2 * turn + 1]) * inv_d;
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) g[c][i] = mul2(splat2(rstd_post), fma2(m[c][i], splat2(-dot), g[c][i]));
    }
    if (p.dy != nullptr) {
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int at = (c * TPR + tid) * 8;
        if (at < p.D) store8(p.dy, base + at, g[c]);
      }
    }
  }
  cp_async_wait<0>();

  // One partial row per CTA.  With a warp per row, the warps add theirs in turn.
  auto put = [&](const F2 (&s)[NC][4], int which) {
    float* dst = p.part + (static_cast<int64_t>(which) * gridDim.x + blockIdx.x) * p.D;
    for (int w = 0; w < kRows; ++w) {
      if (static_cast<int>(threadIdx.x) / TPR == w) {
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const int at = (c * TPR + tid) * 8;
          if (at >= p.D) continue;
          F2 o[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) o[i] = splat2(0.0f);
          if (w > 0) load8(dst, at, o);
#pragma unroll
          for (int i = 0; i < 4; ++i) o[i] = add2(o[i], s[c][i]);
          store8(dst, at, o);
        }
      }
      if (kRows > 1) __syncthreads();
    }
  };
  if (p.dw_pre) put(s_pre, 0);
  if (p.dgate || p.dw_post) put(s_branch, 1);
}

// Column sums from the `count` partial rows of quantity q = blockIdx.y: dw_pre
// is the first, and dgate and dw_post are both the second, T = sum g m, times
// what does not depend on the row (scale w_post and scale gate).  A CTA takes
// 32 columns; its 32 warps take every 32nd row, then add in a fixed tree.
__global__ void __launch_bounds__(1024) residual_norm_finish_kernel(ResidualNormBwd p, int count) {
  __shared__ float sums[32][33];
  pdl_wait_prior();
  if (blockIdx.y == 0 ? p.dw_pre == nullptr : p.dgate == nullptr && p.dw_post == nullptr) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t d0 = static_cast<int64_t>(blockIdx.x) * 32;
  const float* src = p.part + static_cast<int64_t>(blockIdx.y) * count * p.D + d0 + lane;
  float s = 0.0f;
#pragma unroll 8
  for (int i = warp; i < count; i += 32) s += src[i * p.D];
  sums[warp][lane] = s;
  __syncthreads();
  s = sums[lane][warp];  // warp w: column w
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
  if (lane != 0) return;
  const int64_t d = d0 + warp;
  if (blockIdx.y == 0) {
    p.dw_pre[d] = s;
    return;
  }
  if (p.dgate != nullptr) p.dgate[d] = s * p.scale * (p.w_post != nullptr ? p.w_post[d] : 1.0f);
  if (p.dw_post != nullptr) p.dw_post[d] = s * p.scale * (p.gate != nullptr ? p.gate[d] : 1.0f);
}

namespace {

// Threads per row (TPR) and 8-value groups per thread (NC), by the row's length.
// An fp32 stream has more bytes in flight per thread and runs better with one
// group up to 4096 values (8192 x 4096: forward 92 us with two, 81 with one,
// backward 139 and 137; 8192 x 2048: 51 and 45, 78 and 73; 4096 x 8192, where one
// takes 1024 threads: backward 147 and 206).  bf16 rows run better with two
// (8192 x 2048: backward 41 us, 45 with one).
struct NormShape {
  int tpr, nc;
};

constexpr NormShape norm_shape(int64_t D, bool fp32) {
  const int nc = D <= 256 || (fp32 && D <= 4096) ? 1 : 2;
  int tpr = 32;
  while (tpr * nc * 8 < D) tpr *= 2;
  return NormShape{tpr, nc};
}

template <typename TRes, typename F>
cudaError_t with_shape(int64_t D, F&& f) {
  using std::integral_constant;
  constexpr bool kFp32 = sizeof(TRes) == 4;
  constexpr int kMid = kFp32 ? 1 : 2;  // groups of the shapes in between
  const NormShape shape = norm_shape(D, kFp32);
  switch (shape.tpr) {
    case 32:
      if constexpr (!kFp32)
        if (shape.nc == 2) return f(integral_constant<int, 32>{}, integral_constant<int, 2>{});
      return f(integral_constant<int, 32>{}, integral_constant<int, 1>{});
    case 64: return f(integral_constant<int, 64>{}, integral_constant<int, kMid>{});
    case 128: return f(integral_constant<int, 128>{}, integral_constant<int, kMid>{});
    case 256: return f(integral_constant<int, 256>{}, integral_constant<int, kMid>{});
    case 512:
      if constexpr (kFp32)
        if (shape.nc == 1) return f(integral_constant<int, 512>{}, integral_constant<int, 1>{});
      return f(integral_constant<int, 512>{}, integral_constant<int, 2>{});
    default: return f(integral_constant<int, 1024>{}, integral_constant<int, 2>{});
  }
}

// CTAs of one wave on a 148-SM B200 with `threads` resident threads per SM,
// or as many as the rows need.
int64_t norm_ctas(int64_t M, int64_t D, bool fp32, int64_t resident) {
  const int64_t tpr = norm_shape(D, fp32).tpr, rows = tpr == 32 ? kWarpRowCtas : 1;
  const int64_t threads = tpr * rows, want = (M + rows - 1) / rows;
  const int64_t most = 148 * (threads >= resident ? 1 : resident / threads);
  return want < most ? want : most;
}

template <typename Kernel, typename Params>
cudaError_t launch_norm(Kernel kernel, DeviceOnce& configured, int ctas, int threads, int smem, const Params& p,
                        cudaStream_t stream) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = configured.run(dev, [&] { return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem); });
  if (e != cudaSuccess) return e;
  kernel<<<ctas, threads, smem, stream>>>(p);
  return cudaGetLastError();
}

template <typename TRes>
cudaError_t launch_fwd(const ResidualNormFwd& p, cudaStream_t stream) {
  return with_shape<TRes>(p.D, [&](auto tpr, auto nc) {
    constexpr int TPR = decltype(tpr)::value, NC = decltype(nc)::value;
    constexpr int smem =
        RowSlot<TRes, TPR, NC>::kBytes + RowSlot<uint16_t, TPR, NC>::kBytes + 2 * RowSlot<float, TPR, NC>::kBytes;
    static DeviceOnce configured;
    const int ctas = static_cast<int>(norm_ctas(p.M, p.D, sizeof(TRes) == 4, kFwdResident));
    return launch_norm(residual_norm_fwd_kernel<TRes, TPR, NC>, configured, ctas, kNormThreads<TPR>, smem, p, stream);
  });
}

template <typename TRes>
cudaError_t launch_bwd(const ResidualNormBwd& p, cudaStream_t stream) {
  return with_shape<TRes>(p.D, [&](auto tpr, auto nc) {
    constexpr int TPR = decltype(tpr)::value, NC = decltype(nc)::value;
    constexpr int smem = 2 * (RowSlot<TRes, TPR, NC>::kBytes + RowSlot<uint16_t, TPR, NC>::kBytes) +
                         (kStash<TPR> ? 2 * RowSlot<float, TPR, NC>::kBytes : 0);
    static DeviceOnce configured;
    const int ctas = residual_norm_bwd_ctas(p.M, p.D, sizeof(TRes) == 4);
    return launch_norm(residual_norm_bwd_kernel<TRes, TPR, NC>, configured, ctas, kNormThreads<TPR>, smem, p, stream);
  });
}

}  // namespace

int residual_norm_bwd_ctas(int64_t M, int64_t D, bool res_fp32) {
  // Every CTA leaves a partial row of the column sums: with few rows, the same
  // number of CTAs on each SM and three or more rows for each keep those below
  // the operands themselves.  GPU time of bf16 rows: 999 x 2048 (128 threads each)
  // 296 CTAs 11.3 us, 148 13.3, 444 12.3, all 592 12.9; 999 x 1024 (64 threads)
  // 296 9.8, 148 12.5, all 12.6; 3000 x 2048 888, so all 592, 19.2, 148 27.1.
  // Where few CTAs fit an SM anyway it makes no difference (fp32 rows, 999 x 2048,
  // 256 threads: 148 14.0, 296 14.2).
  return static_cast<int>(
      std::min<int64_t>(norm_ctas(M, D, res_fp32, kBwdResident), 148 * std::max<int64_t>(1, M / (148 * 3))));
}

cudaError_t launch_residual_norm_fwd(const ResidualNormFwd& p, int res_fp32, cudaStream_t stream) {
  return res_fp32 ? launch_fwd<float>(p, stream) : launch_fwd<uint16_t>(p, stream);
}

cudaError_t launch_residual_norm_bwd(const ResidualNormBwd& p, int res_fp32, cudaStream_t stream) {
  const cudaError_t e = res_fp32 ? launch_bwd<float>(p, stream) : launch_bwd<uint16_t>(p, stream);
  if (e != cudaSuccess || (!p.dw_pre && !p.dgate && !p.dw_post)) return e;
  return launch_dependent(residual_norm_finish_kernel, dim3(static_cast<unsigned>(p.D / 32), 2), 1024, 0, stream, p,
                          residual_norm_bwd_ctas(p.M, p.D, res_fp32 != 0));
}

}  // namespace qnf4
