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
// block).  Rows of up to 1024 values take one warp (reductions by shuffles
// alone), longer ones a CTA.  All arithmetic is fp32.
//
// The backward's column sums stay in registers over all rows of a CTA; each
// CTA writes one partial row and residual_norm_finish_kernel adds those in a
// fixed order (no atomics).
#include <type_traits>

#include "act8.cuh"
#include "kernels.cuh"

namespace qnf4 {

namespace {

constexpr int kWarpRowCtas = 8;  // rows (warps) of a CTA when a warp takes a row

template <int TPR>
constexpr int kNormThreads = TPR == 32 ? 32 * kWarpRowCtas : TPR;

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
#pragma unroll
    for (int w = 0; w < TPR / 32; ++w) v += slots[w];
  }
  return v;
}

__device__ __forceinline__ void unpack8(const uint4& u, float (&v)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}

// Eight values at element offset `at`; plain loads, as some inputs may be
// written by the same call (in place).
__device__ __forceinline__ void load8(const uint16_t* p, int64_t at, float (&v)[8]) {
  unpack8(*reinterpret_cast<const uint4*>(p + at), v);
}
__device__ __forceinline__ void load8(const float* p, int64_t at, float (&v)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p + at), b = *reinterpret_cast<const float4*>(p + at + 4);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void store8(uint16_t* p, int64_t at, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p + at) = pack8(v);
}
__device__ __forceinline__ void store8(float* p, int64_t at, const float (&v)[8]) {
  *reinterpret_cast<float4*>(p + at) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(p + at + 4) = make_float4(v[4], v[5], v[6], v[7]);
}

}  // namespace

template <typename TRes, int TPR, int NC>
__global__ void __launch_bounds__(kNormThreads<TPR>) residual_norm_fwd_kernel(ResidualNormFwd p) {
  __shared__ float slots[2][32];
  const int tid = threadIdx.x % TPR;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kNormThreads<TPR> / TPR) + threadIdx.x / TPR;
  if (row >= p.M) return;  // a whole warp (TPR = 32) or nothing
  const TRes* h = static_cast<const TRes*>(p.h);
  TRes* h_out = static_cast<TRes*>(p.h_out);
  const int64_t base = row * p.D;
  const float inv_d = 1.0f / static_cast<float>(p.D);

  float v[NC][8];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int at = (c * TPR + tid) * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[c][i] = 0.0f;
    if (at < p.D) load8(h, base + at, v[c]);
  }
  if (p.y != nullptr) {
    float y[NC][8];
    float ss = 0.0f;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int at = (c * TPR + tid) * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) y[c][i] = 0.0f;
      if (at < p.D) load8(p.y, base + at, y[c]);
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(y[c][i], y[c][i], ss);
    }
    float rstd = 1.0f;
    if (p.w_post != nullptr) {
      ss = row_sum<TPR>(ss, slots[0]);
      rstd = 1.0f / sqrtf(ss * inv_d + p.eps);
      if (p.rstd_post != nullptr && tid == 0) p.rstd_post[row] = rstd;
    }
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int at = (c * TPR + tid) * 8;
      if (at >= p.D) continue;
      float w[8], g[8];
      if (p.w_post != nullptr) {
        load8(p.w_post, at, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[c][i] = y[c][i] * rstd * w[i];
      }
      if (p.gate != nullptr) {
        load8(p.gate, at, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[c][i] *= g[i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] = fmaf(p.scale, y[c][i], v[c][i]);
    }
  }
  if (h_out != nullptr) {
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int at = (c * TPR + tid) * 8;
      if (at < p.D) store8(h_out, base + at, v[c]);
    }
  }
  if (p.x == nullptr) return;
  float ss = 0.0f;
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(v[c][i], v[c][i], ss);
  ss = row_sum<TPR>(ss, slots[1]);
  const float rstd = 1.0f / sqrtf(ss * inv_d + p.eps);
  if (p.rstd_pre != nullptr && tid == 0) p.rstd_pre[row] = rstd;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int at = (c * TPR + tid) * 8;
    uint4 x = make_uint4(0, 0, 0, 0);
    if (at < p.D) {
      float w[8];
      load8(p.w_pre, at, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = v[c][i] * rstd * w[i];
      x = pack8(w);
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

template <typename TRes, int TPR, int NC>
__global__ void __launch_bounds__(kNormThreads<TPR>) residual_norm_bwd_kernel(ResidualNormBwd p) {
  constexpr int kRows = kNormThreads<TPR> / TPR;
  __shared__ float slots[4][32];
  const int tid = threadIdx.x % TPR;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kRows;
  const TRes* dh_out = static_cast<const TRes*>(p.dh_out);
  const TRes* h_out = static_cast<const TRes*>(p.h_out);
  TRes* dh = static_cast<TRes*>(p.dh);
  const float inv_d = 1.0f / static_cast<float>(p.D);
  const bool need_y = p.w_post != nullptr || p.dgate;

  float s_pre[NC][8], s_gate[NC][8], s_post[NC][8];
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) s_pre[c][i] = s_gate[c][i] = s_post[c][i] = 0.0f;

  int turn = 0;  // row_sum arrays alternate from row to row: a row's are written again two barriers later
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / TPR; row < p.M;
       row += stride, turn ^= 1) {
    const int64_t base = row * p.D;
    float g[NC][8];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int at = (c * TPR + tid) * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) g[c][i] = 0.0f;
      if (dh_out != nullptr && at < p.D) load8(dh_out, base + at, g[c]);
    }
    if (p.dx != nullptr) {
      const float rstd = p.rstd_pre[row];
      float dn[NC][8], n[NC][8];
      float dot = 0.0f;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int at = (c * TPR + tid) * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i) dn[c][i] = n[c][i] = 0.0f;
        if (at >= p.D) continue;
        float w[8];
        load8(p.dx, base + at, dn[c]);
        load8(h_out, base + at, n[c]);
        load8(p.w_pre, at, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          n[c][i] *= rstd;
          s_pre[c][i] = fmaf(dn[c][i], n[c][i], s_pre[c][i]);
          dn[c][i] *= w[i];
          dot = fmaf(dn[c][i], n[c][i], dot);
        }
      }
      dot = row_sum<TPR>(dot, slots[2 * turn]) * inv_d;
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) g[c][i] = fmaf(rstd, dn[c][i] - n[c][i] * dot, g[c][i]);
    }
    if (dh != nullptr) {
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int at = (c * TPR + tid) * 8;
        if (at < p.D) store8(dh, base + at, g[c]);
      }
    }
    if (p.dy == nullptr && !p.dgate && !p.dw_post) continue;
    float m[NC][8];
    const float rstd = p.w_post != nullptr ? p.rstd_post[row] : 1.0f;
    float dot = 0.0f;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int at = (c * TPR + tid) * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) m[c][i] = 0.0f;
      if (at >= p.D) continue;
      float w[8], gt[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = gt[i] = 1.0f;
      if (need_y) load8(p.y, base + at, m[c]);
      if (p.w_post != nullptr) load8(p.w_post, at, w);
      if (p.gate != nullptr) load8(p.gate, at, gt);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        m[c][i] *= rstd;
        float dp = p.scale * g[c][i];
        s_gate[c][i] = fmaf(dp, m[c][i] * w[i], s_gate[c][i]);
        dp *= gt[i];
        s_post[c][i] = fmaf(dp, m[c][i], s_post[c][i]);
        g[c][i] = dp * w[i];
        dot = fmaf(g[c][i], m[c][i], dot);
      }
    }
    if (p.w_post != nullptr) {
      dot = row_sum<TPR>(dot, slots[2 * turn + 1]) * inv_d;
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) g[c][i] = rstd * (g[c][i] - m[c][i] * dot);
    }
    if (p.dy != nullptr) {
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int at = (c * TPR + tid) * 8;
        if (at < p.D) store8(p.dy, base + at, g[c]);
      }
    }
  }

  // One partial row per CTA.  With a warp per row, the warps add theirs in turn.
  auto put = [&](const float (&s)[NC][8], int which) {
    float* dst = p.part + (static_cast<int64_t>(which) * gridDim.x + blockIdx.x) * p.D;
    for (int w = 0; w < kRows; ++w) {
      if (static_cast<int>(threadIdx.x) / TPR == w) {
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const int at = (c * TPR + tid) * 8;
          if (at >= p.D) continue;
          float o[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = 0.0f;
          if (w > 0) load8(dst, at, o);
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] += s[c][i];
          store8(dst, at, o);
        }
      }
      if (kRows > 1) __syncthreads();
    }
  };
  if (p.dw_pre) put(s_pre, 0);
  if (p.dgate) put(s_gate, 1);
  if (p.dw_post) put(s_post, 2);
}

// dst_q[d] = sum of the `count` partial rows of gradient q = blockIdx.y.  A CTA
// takes 32 columns; its 8 warps take every eighth row, then add in order.
__global__ void __launch_bounds__(256) residual_norm_finish_kernel(const float* __restrict__ part, int count, int64_t D,
                                                                   float* dw_pre, float* dgate, float* dw_post) {
  __shared__ float sums[8][32];
  float* dst = blockIdx.y == 0 ? dw_pre : blockIdx.y == 1 ? dgate : dw_post;
  if (dst == nullptr) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t d = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  const float* src = part + static_cast<int64_t>(blockIdx.y) * count * D + d;
  float s = 0.0f;
  for (int i = warp; i < count; i += 8) s += src[i * D];
  sums[warp][lane] = s;
  __syncthreads();
  if (warp == 0) {
    s = 0.0f;
#pragma unroll
    for (int w = 0; w < 8; ++w) s += sums[w][lane];
    dst[d] = s;
  }
}

namespace {

// Threads per row and 8-value groups per thread, by the row's length.
template <typename F>
cudaError_t with_shape(int64_t D, F&& f) {
  if (D <= 256) return f(std::integral_constant<int, 32>{}, std::integral_constant<int, 1>{});
  if (D <= 512) return f(std::integral_constant<int, 32>{}, std::integral_constant<int, 2>{});
  if (D <= 1024) return f(std::integral_constant<int, 32>{}, std::integral_constant<int, 4>{});
  if (D <= 2048) return f(std::integral_constant<int, 128>{}, std::integral_constant<int, 2>{});
  if (D <= 4096) return f(std::integral_constant<int, 256>{}, std::integral_constant<int, 2>{});
  if (D <= 8192) return f(std::integral_constant<int, 512>{}, std::integral_constant<int, 2>{});
  return f(std::integral_constant<int, 1024>{}, std::integral_constant<int, 2>{});
}

int64_t rows_per_cta(int64_t D) { return D <= 1024 ? kWarpRowCtas : 1; }

}  // namespace

int residual_norm_bwd_ctas(int64_t M, int64_t D) {
  const int64_t want = (M + rows_per_cta(D) - 1) / rows_per_cta(D);
  // Resident CTAs of a 148-SM B200: 512 threads or one CTA per SM.
  const int64_t threads = D <= 1024 ? 256 : D <= 2048 ? 128 : D <= 4096 ? 256 : D <= 8192 ? 512 : 1024;
  const int64_t most = 148 * (threads >= 512 ? 1 : 512 / threads);
  return static_cast<int>(want < most ? want : most);
}

cudaError_t launch_residual_norm_fwd(const ResidualNormFwd& p, int res_fp32, cudaStream_t stream) {
  const int64_t rows = rows_per_cta(p.D);
  const unsigned grid = static_cast<unsigned>((p.M + rows - 1) / rows);
  return with_shape(p.D, [&](auto tpr, auto nc) {
    constexpr int TPR = decltype(tpr)::value, NC = decltype(nc)::value;
    if (res_fp32)
      residual_norm_fwd_kernel<float, TPR, NC><<<grid, kNormThreads<TPR>, 0, stream>>>(p);
    else
      residual_norm_fwd_kernel<uint16_t, TPR, NC><<<grid, kNormThreads<TPR>, 0, stream>>>(p);
    return cudaGetLastError();
  });
}

cudaError_t launch_residual_norm_bwd(const ResidualNormBwd& p, int res_fp32, cudaStream_t stream) {
  const int ctas = residual_norm_bwd_ctas(p.M, p.D);
  const cudaError_t e = with_shape(p.D, [&](auto tpr, auto nc) {
    constexpr int TPR = decltype(tpr)::value, NC = decltype(nc)::value;
    if (res_fp32)
      residual_norm_bwd_kernel<float, TPR, NC><<<ctas, kNormThreads<TPR>, 0, stream>>>(p);
    else
      residual_norm_bwd_kernel<uint16_t, TPR, NC><<<ctas, kNormThreads<TPR>, 0, stream>>>(p);
    return cudaGetLastError();
  });
  if (e != cudaSuccess || (!p.dw_pre && !p.dgate && !p.dw_post)) return e;
  residual_norm_finish_kernel<<<dim3(static_cast<unsigned>(p.D / 32), 3), 256, 0, stream>>>(p.part, ctas, p.D, p.dw_pre,
                                                                                           p.dgate, p.dw_post);
  return cudaGetLastError();
}

}  // namespace qnf4
