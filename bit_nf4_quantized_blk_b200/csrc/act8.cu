// 8-bit activation checkpoints (sm_100a): writing, reading back, and the two
// products of the LoRA backward that read the saved activation.
//
// "QLoRA: NF4 storage, gradients and local integration" (gradient paragraph
// after the teaching program): dA = s V^T X and, when U was not saved,
// U = X A^T are the only places where the backward of a QLoRA linear layer
// needs its input X.  Keeping X as one byte per value and a bf16 step per 64
// (act8.cuh) halves what the layer keeps between forward and backward, and
// these kernels read the codes as they are: X^ is never written out.
//
//  act8_quantize_kernel    8 values per lane and 8 lanes per block: the block
//                          maximum is three shuffles.  HBM-bound (3.03 bytes
//                          per value).
//  act8_dequantize_kernel  the reverse.
//  act8_colsum_kernel      part[z][j][k] = sum over the tokens m of split z of
//                          V[m][j] X^[m][k], then act8_colsum_reduce_kernel
//                          adds the splits in a fixed order (dA).
//  act8_skinny_kernel      part[z][m][j] = sum over the columns of split z of
//                          X^[m][k] A[j][k] (U).
// Deterministic: every sum runs in a fixed order; no atomics.
#include "act8.cuh"
#include "kernels.cuh"

namespace qnf4 {

namespace {

constexpr int kQThreads = 256;
constexpr int kQChunks = 4;  // 16-byte units per thread, 32 lanes apart

}  // namespace

template <int kFormat>
__global__ void __launch_bounds__(kQThreads) act8_quantize_kernel(const uint4* __restrict__ X, int64_t units,
                                                                  uint2* __restrict__ codes,
                                                                  uint16_t* __restrict__ step) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t u0 = (static_cast<int64_t>(blockIdx.x) * (kQThreads / 32) + warp) * (32 * kQChunks) + lane;
  uint4 v[kQChunks];
#pragma unroll
  for (int i = 0; i < kQChunks; ++i)
    v[i] = u0 + 32 * i < units ? ld_stream_u4(X + u0 + 32 * i) : make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int i = 0; i < kQChunks; ++i) {
    uint32_t m = absmax_bf16x2(absmax_bf16x2(absmax_bf16x2(v[i].x & 0x7FFF7FFFu, v[i].y), v[i].z), v[i].w);
    m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 2));
    m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 4));
    const Act8Encoder<kFormat> enc(max(m & 0xFFFFu, m >> 16));
    const int64_t u = u0 + 32 * i;
    if (u < units) {  // a block is 8 units: in or out as a whole
      codes[u] = enc.encode8(v[i]);
      if ((u & 7) == 0) step[u >> 3] = static_cast<uint16_t>(enc.step);
    }
  }
}

template <int kFormat>
__global__ void __launch_bounds__(kQThreads) act8_dequantize_kernel(const uint2* __restrict__ codes,
                                                                    const uint16_t* __restrict__ step, int64_t units,
                                                                    uint4* __restrict__ X) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t u0 = (static_cast<int64_t>(blockIdx.x) * (kQThreads / 32) + warp) * (32 * kQChunks) + lane;
  uint2 c[kQChunks];
  uint32_t s[kQChunks];
#pragma unroll
  for (int i = 0; i < kQChunks; ++i) {
    const int64_t u = u0 + 32 * i;
    c[i] = u < units ? __ldg(codes + u) : make_uint2(0, 0);
    s[i] = u < units ? __ldg(step + (u >> 3)) : 0u;
  }
#pragma unroll
  for (int i = 0; i < kQChunks; ++i) {
    const uint32_t s2 = s[i] | (s[i] << 16);
    const uint4 v = make_uint4(act8_decode2<kFormat, 0>(c[i].x, s2), act8_decode2<kFormat, 2>(c[i].x, s2),
                               act8_decode2<kFormat, 0>(c[i].y, s2), act8_decode2<kFormat, 2>(c[i].y, s2));
    if (u0 + 32 * i < units) st_stream_u4(X + u0 + 32 * i, v);
  }
}

namespace {

unsigned quant_grid(int64_t units) {
  constexpr int64_t per_cta = kQThreads * kQChunks;
  return static_cast<unsigned>((units + per_cta - 1) / per_cta);
}

}  // namespace

cudaError_t launch_act8_quantize(const uint16_t* X, int64_t n, int format, uint8_t* codes, uint16_t* step,
                                 cudaStream_t stream) {
  const int64_t units = n / 8;
  const auto* x = reinterpret_cast<const uint4*>(X);
  auto* c = reinterpret_cast<uint2*>(codes);
  if (format == kAct8Int8)
    act8_quantize_kernel<kAct8Int8><<<quant_grid(units), kQThreads, 0, stream>>>(x, units, c, step);
  else
    act8_quantize_kernel<kAct8E4m3><<<quant_grid(units), kQThreads, 0, stream>>>(x, units, c, step);
  return cudaGetLastError();
}

cudaError_t launch_act8_dequantize(const Act8View& a, uint16_t* X, cudaStream_t stream) {
  const int64_t units = a.rows * a.cols / 8;
  const auto* c = reinterpret_cast<const uint2*>(a.codes);
  auto* x = reinterpret_cast<uint4*>(X);
  if (a.format == kAct8Int8)
    act8_dequantize_kernel<kAct8Int8><<<quant_grid(units), kQThreads, 0, stream>>>(c, a.step, units, x);
  else
    act8_dequantize_kernel<kAct8E4m3><<<quant_grid(units), kQThreads, 0, stream>>>(c, a.step, units, x);
  return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// colsum: part[z][j][k] = sum_{m in split z} (hi[m][j] + lo[m][j]) X^[m][k]
// ---------------------------------------------------------------------------
// m16n8k16 MMAs with D = [16 j][8 columns], the token axis as K: A = V^T from
// the [m][64] hi / lo split by transposed 8x8 loads, B = X^ decoded in
// registers.  A lane's B registers are pairs of tokens (2t, 2t + 1 and 2t + 8,
// 2t + 9) of one column; which column a slot stands for is free, so lane
// (g, t) takes kCB consecutive code bytes of each of its four token rows, at
// byte g kCB of the warp's 8 kCB columns, and MMA i takes its i-th byte: the
// code loads are wide and nothing is exchanged between lanes.
//
// A CTA is 4 column groups x kWT token groups of warps; each warp runs its own
// ring of cp.async copies (codes: read back by the thread that copied them;
// V: by the warp), so no CTA barrier sits in the loop.  At the end the token
// groups' sums are added in shared memory and stored as one partial.
namespace {

constexpr int kCsWC = 4;      // column groups of a CTA
constexpr int kCsStages = 4;  // ring depth

template <int kRT>
struct ColsumShape {
  static constexpr int kCB = kRT == 1 ? 16 : 8;     // code bytes per lane and row
  static constexpr int kWT = kRT <= 2 ? 4 : 2;      // token groups of a CTA
  static constexpr int kCols = 8 * kCB;             // columns of a warp
  static constexpr int kWarps = kCsWC * kWT;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kCodeBytes = 16 * kCols;     // one step: 16 tokens
  static constexpr int kVBytes = 16 * kRT * 16 * 2;  // of one half of the split
  static constexpr int kStageBytes = kCodeBytes + 2 * kVBytes;
  static constexpr int kRingBytes = kWarps * kCsStages * kStageBytes;
  static constexpr int kRedPitch = kCols + 4;       // floats
  static constexpr int kRedBytes = kWarps * kRT * 16 * kRedPitch * 4;
  static constexpr int kSmem = kRingBytes > kRedBytes ? kRingBytes : kRedBytes;
  static constexpr int kCtaCols = kCsWC * kCols;
  static constexpr int kCtaTokens = kWT * 16;       // tokens of a CTA per step
};

template <int kBytes>
__device__ __forceinline__ void cp_async_n(void* dst, const void* src, bool valid) {
  const int n = valid ? kBytes : 0;
  if constexpr (kBytes == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(n) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(n), "n"(kBytes)
                 : "memory");
}

int colsum_splits_rt(int64_t M, int64_t K, int cta_cols, int cta_tokens) {
  const int64_t cols = (K + cta_cols - 1) / cta_cols, steps = (M + cta_tokens - 1) / cta_tokens;
  int64_t s = 148 / cols;  // one wave of one CTA per SM
  if (s > steps) s = steps;
  return static_cast<int>(s < 1 ? 1 : s);
}

template <int kRT>
int colsum_splits_of(int64_t M, int64_t K) {
  return colsum_splits_rt(M, K, ColsumShape<kRT>::kCtaCols, ColsumShape<kRT>::kCtaTokens);
}

}  // namespace

template <int kFormat, int kRT>
__global__ void __launch_bounds__(ColsumShape<kRT>::kThreads, 1)
    act8_colsum_kernel(const uint8_t* __restrict__ codes, const uint16_t* __restrict__ step,
                       const uint16_t* __restrict__ vhi, const uint16_t* __restrict__ vlo, int64_t M, int64_t K,
                       int splits, float* __restrict__ part) {
  using S = ColsumShape<kRT>;
  extern __shared__ __align__(16) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int wc = warp % kCsWC, wt = warp / kCsWC;
  const int64_t c0 = static_cast<int64_t>(blockIdx.x) * S::kCtaCols + wc * S::kCols;
  const int z = blockIdx.y;
  const int64_t total = (M + S::kCtaTokens - 1) / S::kCtaTokens;
  const int64_t first = total * z / splits;
  const int n = static_cast<int>(total * (z + 1) / splits - first);
  const int64_t m0 = (first * S::kWT + wt) * 16;  // the warp's first token; kCtaTokens further per step
  const int64_t kblocks = K / kBlock;
  uint8_t* ring = smem + warp * (kCsStages * S::kStageBytes);

  const int64_t col = c0 + g * S::kCB;  // this lane's columns: in or out of K as a whole (K % 64 == 0)
  const bool col_ok = col < K;
  // One step per lane: lane l holds that of token l / 2 of the step and of
  // the warp's block l % 2 (kCols = 128: two blocks; 64: one).
  constexpr int kBlocksPerWarp = S::kCols / kBlock;
  const int64_t blk = c0 / kBlock + (lane & (kBlocksPerWarp - 1));
  const int step_token = lane / kBlocksPerWarp;

  auto issue = [&](int i) {
    if (i < n) {
      uint8_t* st = ring + (i % kCsStages) * S::kStageBytes;
      const int64_t m = m0 + static_cast<int64_t>(i) * S::kCtaTokens;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int64_t row = m + 2 * t + (q & 1) + (q >> 1) * 8;
        const bool ok = col_ok && row < M;
        cp_async_n<S::kCB>(st + (q * 32 + lane) * S::kCB, codes + (ok ? row * K + col : 0), ok);
      }
#pragma unroll
      for (int q = 0; q < 2 * kRT; ++q) {
        const int chunk = q * 32 + lane;            // of 64 kRT: hi, then lo; 2 kRT chunks per token
        const int half = chunk / (32 * kRT), rest = chunk % (32 * kRT);
        const int64_t row = m + rest / (2 * kRT);
        const uint16_t* src = half ? vlo : vhi;
        cp_async_n<16>(st + S::kCodeBytes + chunk * 16, src + (row < M ? row * kRankPad + (rest % (2 * kRT)) * 8 : 0),
                       row < M);
      }
    }
    cp_async_commit();
  };
  auto load_step = [&](int i) -> uint32_t {
    const int64_t row = m0 + static_cast<int64_t>(i) * S::kCtaTokens + step_token;
    const bool ok = i < n && step_token < 16 && row < M && blk < kblocks;
    return ok ? step[row * kblocks + blk] : 0u;
  };

  float acc[kRT][S::kCB][4];
#pragma unroll
  for (int a = 0; a < kRT; ++a)
#pragma unroll
    for (int b = 0; b < S::kCB; ++b)
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[a][b][c] = 0.0f;

#pragma unroll
  for (int i = 0; i < kCsStages - 1; ++i) issue(i);
  uint32_t next_step = load_step(0);

  const int mat = lane >> 3, rr = lane & 7;
  for (int i = 0; i < n; ++i) {
    const uint32_t my_step = next_step;
    next_step = load_step(i + 1);
    cp_async_wait<kCsStages - 2>();
    __syncwarp();
    issue(i + kCsStages - 1);  // into the stage read in the previous iteration
    const uint8_t* st = ring + (i % kCsStages) * S::kStageBytes;
    // Packed steps of the token pairs (2t, 2t + 1) and (2t + 8, 2t + 9), block of column g kCB.
    const int b = g * S::kCB / kBlock;
    uint32_t s2[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int tok = 2 * t + 8 * h;
      const uint32_t lo = __shfl_sync(0xffffffffu, my_step, tok * kBlocksPerWarp + b);
      const uint32_t hi = __shfl_sync(0xffffffffu, my_step, (tok + 1) * kBlocksPerWarp + b);
      s2[h] = lo | (hi << 16);
    }
    uint32_t ah[kRT][4], al[kRT][4];
#pragma unroll
    for (int a = 0; a < kRT; ++a) {
      // Stored rows are tokens (2 kRT chunks of 8 j each): matrices (tokens 0-7, j lo), (0-7, hi), (8-15, lo), (8-15, hi).
      const uint32_t addr = smem_u32(st + S::kCodeBytes) + (((mat >> 1) * 8 + rr) * (2 * kRT) + a * 2 + (mat & 1)) * 16;
      ldmatrix_x4_trans(ah[a], addr);
      ldmatrix_x4_trans(al[a], addr + S::kVBytes);
    }
#pragma unroll
    for (int w = 0; w < S::kCB / 4; ++w) {
      uint32_t c[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        c[q] = *reinterpret_cast<const uint32_t*>(st + (q * 32 + lane) * S::kCB + 4 * w);
      // Byte pairs (row 2t, row 2t + 1) of the word's four columns.
      const uint32_t p[2][2] = {{__byte_perm(c[0], c[1], 0x5140), __byte_perm(c[0], c[1], 0x7362)},
                                {__byte_perm(c[2], c[3], 0x5140), __byte_perm(c[2], c[3], 0x7362)}};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint32_t bf[2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
          bf[h] = e % 2 == 0 ? act8_decode2<kFormat, 0>(p[h][e / 2], s2[h]) : act8_decode2<kFormat, 2>(p[h][e / 2], s2[h]);
#pragma unroll
        for (int a = 0; a < kRT; ++a) {
          mma_16816(acc[a][4 * w + e], ah[a], bf);
          mma_16816(acc[a][4 * w + e], al[a], bf);
        }
      }
    }
  }
  cp_async_wait<0>();
  __syncthreads();  // every ring is free: its space takes the warps' sums

  float* red = reinterpret_cast<float*>(smem);
  float* mine = red + warp * (kRT * 16 * S::kRedPitch);
#pragma unroll
  for (int a = 0; a < kRT; ++a)
#pragma unroll
    for (int b = 0; b < S::kCB; ++b)
#pragma unroll
      for (int c = 0; c < 4; ++c)
        mine[(a * 16 + g + (c >> 1) * 8) * S::kRedPitch + (2 * t + (c & 1)) * S::kCB + b] = acc[a][b][c];
  __syncthreads();
  constexpr int kOut = kRT * 16 * S::kCtaCols;
  for (int o = threadIdx.x; o < kOut; o += S::kThreads) {
    const int j = o / S::kCtaCols, c = o % S::kCtaCols;
    const float* src = red + (c / S::kCols) * (kRT * 16 * S::kRedPitch) + j * S::kRedPitch + c % S::kCols;
    float s = 0.0f;
#pragma unroll
    for (int q = 0; q < S::kWT; ++q) s += src[q * (kCsWC * kRT * 16 * S::kRedPitch)];
    const int64_t k = static_cast<int64_t>(blockIdx.x) * S::kCtaCols + c;
    if (k < K) part[(static_cast<int64_t>(z) * (kRT * 16) + j) * K + k] = s;
  }
}

// dst[j][k] = scale sum_z part[z][j][k]; part rows are r16 = 16 ceil(r / 16) per split.
__global__ void act8_colsum_reduce_kernel(const float4* __restrict__ part, int64_t k4, int r, int r16, int splits,
                                          float scale, float* __restrict__ dst) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;  // over r * K / 4
  if (i >= k4 * r) return;
  float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int z = 0; z < splits; ++z) {
    const float4 p = part[static_cast<int64_t>(z) * r16 * k4 + i];
    s.x += p.x;
    s.y += p.y;
    s.z += p.z;
    s.w += p.w;
  }
  float* o = dst + 4 * i;  // dst is only 4-byte aligned
  o[0] = scale * s.x;
  o[1] = scale * s.y;
  o[2] = scale * s.z;
  o[3] = scale * s.w;
}

size_t act8_colsum_partial_bytes(int64_t M, int64_t K) {
  const int64_t rows[4] = {16 * int64_t{colsum_splits_of<1>(M, K)}, 32 * int64_t{colsum_splits_of<2>(M, K)},
                           48 * int64_t{colsum_splits_of<3>(M, K)}, 64 * int64_t{colsum_splits_of<4>(M, K)}};
  int64_t most = 0;
  for (const int64_t v : rows) most = v > most ? v : most;
  return static_cast<size_t>(most) * static_cast<size_t>(K) * sizeof(float);
}

namespace {

template <int kFormat, int kRT>
cudaError_t launch_colsum_rt(const Act8View& x, const uint16_t* hi, const uint16_t* lo, float* part, int* splits,
                             cudaStream_t stream) {
  using S = ColsumShape<kRT>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  static DeviceOnce configured;
  e = configured.run(dev, [] {
    return cudaFuncSetAttribute(act8_colsum_kernel<kFormat, kRT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                S::kSmem);
  });
  if (e != cudaSuccess) return e;
  *splits = colsum_splits_of<kRT>(x.rows, x.cols);
  const dim3 grid(static_cast<unsigned>((x.cols + S::kCtaCols - 1) / S::kCtaCols), static_cast<unsigned>(*splits));
  act8_colsum_kernel<kFormat, kRT><<<grid, S::kThreads, S::kSmem, stream>>>(x.codes, x.step, hi, lo, x.rows, x.cols,
                                                                           *splits, part);
  return cudaGetLastError();
}

template <int kFormat>
cudaError_t launch_colsum_format(const Act8View& x, const uint16_t* hi, const uint16_t* lo, int rt, float* part,
                                 int* splits, cudaStream_t stream) {
  switch (rt) {
    case 1: return launch_colsum_rt<kFormat, 1>(x, hi, lo, part, splits, stream);
    case 2: return launch_colsum_rt<kFormat, 2>(x, hi, lo, part, splits, stream);
    case 3: return launch_colsum_rt<kFormat, 3>(x, hi, lo, part, splits, stream);
    default: return launch_colsum_rt<kFormat, 4>(x, hi, lo, part, splits, stream);
  }
}

}  // namespace

cudaError_t launch_act8_colsum(const Act8View& x, const uint16_t* hi, const uint16_t* lo, int r, float scale,
                               float* part, float* dst, cudaStream_t stream) {
  const int rt = (r + 15) / 16;
  int splits = 0;
  const cudaError_t e = x.format == kAct8Int8 ? launch_colsum_format<kAct8Int8>(x, hi, lo, rt, part, &splits, stream)
                                              : launch_colsum_format<kAct8E4m3>(x, hi, lo, rt, part, &splits, stream);
  if (e != cudaSuccess) return e;
  const int64_t k4 = x.cols / 4, items = k4 * r;
  act8_colsum_reduce_kernel<<<static_cast<unsigned>((items + 127) / 128), 128, 0, stream>>>(
      reinterpret_cast<const float4*>(part), k4, r, 16 * rt, splits, scale, dst);
  return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// skinny: part[z][m][j] = sum_{k in split z} X^[m][k] A[j][k]
// ---------------------------------------------------------------------------
// m16n8k16 MMAs with D = [16 tokens][8 j], K = the columns.  Within a 64-column
// block lane (g, t) holds the 16 columns 16t .. 16t + 15 of its rows, and MMA
// step s takes columns 16t + 4s .. + 3 as the lane's four K slots in both
// operands (a permutation of the block's columns): 16 code bytes per row and
// two 16-byte loads per row of A.  A warp covers 32 tokens, so A (from L1) is
// read once per two token tiles.
namespace {

constexpr int kSkWarps = 4;
constexpr int kSkMT = 2;  // 16-token tiles per warp
constexpr int kSkTokens = kSkWarps * kSkMT * 16;

}  // namespace

template <int kFormat, int NT>
__global__ void __launch_bounds__(32 * kSkWarps) act8_skinny_kernel(const uint8_t* __restrict__ codes,
                                                                    const uint16_t* __restrict__ step,
                                                                    const uint16_t* __restrict__ A, int64_t M,
                                                                    int64_t K, int r, int splits,
                                                                    float* __restrict__ part) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int64_t m0 = static_cast<int64_t>(blockIdx.x) * kSkTokens + warp * (kSkMT * 16);
  if (m0 >= M) return;
  const int z = blockIdx.y;
  const int64_t kblocks = K / kBlock;
  const int64_t b0 = kblocks * z / splits, b1 = kblocks * (z + 1) / splits;

  float acc[kSkMT][NT][4];
#pragma unroll
  for (int a = 0; a < kSkMT; ++a)
#pragma unroll
    for (int b = 0; b < NT; ++b)
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[a][b][c] = 0.0f;

  for (int64_t kb = b0; kb < b1; ++kb) {
    uint4 c[kSkMT][2];
    uint32_t s[kSkMT][2];
#pragma unroll
    for (int a = 0; a < kSkMT; ++a)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t row = m0 + a * 16 + h * 8 + g;
        const bool ok = row < M;
        c[a][h] = ok ? ld_stream_u4(codes + row * K + kb * kBlock + t * 16) : make_uint4(0, 0, 0, 0);
        s[a][h] = ok ? __ldg(step + row * kblocks + kb) : 0u;
        s[a][h] |= s[a][h] << 16;
      }
#pragma unroll
    for (int w = 0; w < 4; ++w) {  // columns 16t + 4w .. + 3
      uint32_t af[kSkMT][4];
#pragma unroll
      for (int a = 0; a < kSkMT; ++a)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t word = w == 0 ? c[a][h].x : w == 1 ? c[a][h].y : w == 2 ? c[a][h].z : c[a][h].w;
          af[a][h] = act8_decode2<kFormat, 0>(word, s[a][h]);
          af[a][h + 2] = act8_decode2<kFormat, 2>(word, s[a][h]);
        }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int j = nt * 8 + g;
        uint2 v = make_uint2(0, 0);
        if (j < r) v = __ldg(reinterpret_cast<const uint2*>(A + j * K + kb * kBlock + t * 16 + w * 4));
        const uint32_t bf[2] = {v.x, v.y};
#pragma unroll
        for (int a = 0; a < kSkMT; ++a) mma_16816(acc[a][nt], af[a], bf);
      }
    }
  }
#pragma unroll
  for (int a = 0; a < kSkMT; ++a)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t row = m0 + a * 16 + h * 8 + g;
      if (row >= M) continue;
      float* dst = part + (static_cast<int64_t>(z) * M + row) * kRankPad;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        *reinterpret_cast<float2*>(dst + nt * 8 + 2 * t) = make_float2(acc[a][nt][2 * h], acc[a][nt][2 * h + 1]);
    }
}

namespace {

template <int kFormat>
void launch_skinny_format(const Act8View& x, const uint16_t* A, int r, int splits, float* part, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>((x.rows + kSkTokens - 1) / kSkTokens), static_cast<unsigned>(splits));
  const int threads = 32 * kSkWarps;
  switch ((r + 15) / 16) {
    case 1:
      act8_skinny_kernel<kFormat, 2><<<grid, threads, 0, stream>>>(x.codes, x.step, A, x.rows, x.cols, r, splits, part);
      break;
    case 2:
      act8_skinny_kernel<kFormat, 4><<<grid, threads, 0, stream>>>(x.codes, x.step, A, x.rows, x.cols, r, splits, part);
      break;
    case 3:
      act8_skinny_kernel<kFormat, 6><<<grid, threads, 0, stream>>>(x.codes, x.step, A, x.rows, x.cols, r, splits, part);
      break;
    default:
      act8_skinny_kernel<kFormat, 8><<<grid, threads, 0, stream>>>(x.codes, x.step, A, x.rows, x.cols, r, splits, part);
  }
}

}  // namespace

cudaError_t launch_act8_skinny(const Act8View& x, const uint16_t* A, int r, float* part, const SkinnyOut& out,
                               cudaStream_t stream) {
  const int splits = skinny_splits(x.rows, x.cols);
  if (x.format == kAct8Int8)
    launch_skinny_format<kAct8Int8>(x, A, r, splits, part, stream);
  else
    launch_skinny_format<kAct8E4m3>(x, A, r, splits, part, stream);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_skinny_finalize(part, x.rows, r, splits, out, stream);
}

}  // namespace qnf4
