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
// colsum: part[z][j][k] = sum_{m in split z} V[m][j] X^[m][k], V = hi + lo + lo2
// ---------------------------------------------------------------------------
// m16n8k16 MMAs with D = [16 j][8 columns], the token axis as K: A = V^T from
// the [m][64] parts of V by transposed 8x8 loads, B = X^ decoded in registers.
// A lane's B registers are pairs of tokens (2t, 2t + 1 and 2t + 8, 2t + 9) of
// one column; which column a slot stands for is free, so lane (g, t) takes kCB
// consecutive columns of each of its four token rows, at column g kCB of the
// warp's 8 kCB, and MMA i takes its i-th: the loads are wide and nothing is
// exchanged between lanes.  The same kernel takes plain bf16 rows (dB, from dY
// and U), which only skip the decode.
//
// A CTA is 4 column groups x kWT token groups of warps; each warp runs its own
// ring of cp.async copies (X: read back by the thread that copied it; V: by
// the warp), so no CTA barrier sits in the loop.  At the end the token groups'
// sums are added in shared memory and stored as one partial.
namespace {

constexpr int kCsWC = 4;      // column groups of a CTA
constexpr int kCsStages = 3;  // ring depth
constexpr int kCsParts = 3;   // bf16 parts of V

template <int kFormat, int kRT>
struct ColsumShape {
  static constexpr bool kDense = kFormat == kAct8Dense;
  static constexpr int kCB = kRT == 1 && !kDense ? 16 : 8;    // columns per lane and row
  static constexpr int kWT = kRT == 1 || (kRT == 2 && !kDense) ? 4 : 2;  // token groups of a CTA
  static constexpr int kCols = 8 * kCB;                       // columns of a warp
  static constexpr int kWarps = kCsWC * kWT;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kLaneBytes = kCB * (kDense ? 2 : 1);   // of one row
  static constexpr int kXBytes = 4 * 32 * kLaneBytes;         // one step: 16 tokens
  static constexpr int kVBytes = 16 * kRT * 16 * 2;           // of one part
  static constexpr int kStageBytes = kXBytes + kCsParts * kVBytes;
  static constexpr int kRingBytes = kWarps * kCsStages * kStageBytes;
  static constexpr int kRedPitch = kCols + 4;                 // floats
  static constexpr int kRedBytes = kWarps * kRT * 16 * kRedPitch * 4;
  static constexpr int kSmem = kRingBytes > kRedBytes ? kRingBytes : kRedBytes;
  static constexpr int kCtaCols = kCsWC * kCols;
  static constexpr int kCtaTokens = kWT * 16;                 // tokens of a CTA per step
  static_assert(kSmem <= 227 * 1024, "one CTA's shared memory");

  // Splits of the tokens: one wave of one CTA per SM on a 148-SM B200.
  static int splits(int64_t M, int64_t C) {
    const int64_t cols = (C + kCtaCols - 1) / kCtaCols, steps = (M + kCtaTokens - 1) / kCtaTokens;
    int64_t s = 148 / cols;
    if (s > steps) s = steps;
    return static_cast<int>(s < 1 ? 1 : s);
  }
};

// Place of 16-byte chunk `c` of token row `row` in a V tile of 2 kRT chunks per
// row: permuted so that the eight rows of a transposed 8x8 load fall into
// different banks (unpermuted, rows of 128 bytes meet in the same four, and
// those loads bounded the kernel).  Rows of 96 bytes meet two by two as they are.
template <int kRT>
__device__ __forceinline__ int v_chunk(int row, int c) {
  const int key = kRT == 4 ? row & 7 : kRT == 2 ? (row >> 1) & 3 : kRT == 1 ? (row >> 2) & 1 : 0;
  return row * (2 * kRT) + (c ^ key);
}

template <int kBytes>
__device__ __forceinline__ void cp_async_n(void* dst, const void* src, bool valid) {
  const int n = valid ? kBytes : 0;
  if constexpr (kBytes == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(n) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(n), "n"(kBytes)
                 : "memory");
}

}  // namespace

template <int kFormat, int kRT>
__global__ void __launch_bounds__(ColsumShape<kFormat, kRT>::kThreads, 1)
    act8_colsum_kernel(Act8View x, const uint16_t* __restrict__ vhi, const uint16_t* __restrict__ vlo,
                       const uint16_t* __restrict__ vlo2, int splits, float* __restrict__ part) {
  using S = ColsumShape<kFormat, kRT>;
  extern __shared__ __align__(16) uint8_t smem[];
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int wc = warp % kCsWC, wt = warp / kCsWC;
  const int64_t M = x.rows, C = x.cols;
  const int64_t c0 = static_cast<int64_t>(blockIdx.x) * S::kCtaCols + wc * S::kCols;
  const int z = blockIdx.y;
  const int64_t total = (M + S::kCtaTokens - 1) / S::kCtaTokens;
  const int64_t first = total * z / splits;
  const int n = static_cast<int>(total * (z + 1) / splits - first);
  const int64_t m0 = (first * S::kWT + wt) * 16;  // the warp's first token; kCtaTokens further per step
  uint8_t* ring = smem + warp * (kCsStages * S::kStageBytes);

  const int64_t col = c0 + g * S::kCB;  // this lane's columns: in or out of C as a whole
  const bool col_ok = col < C;
  const int64_t row_bytes = C * (S::kDense ? 2 : 1), col_bytes = col * (S::kDense ? 2 : 1);
  // One step per lane: lane l holds that of token l / blocks of the step and
  // of the warp's block l % blocks (kCols = 128: two blocks; 64: one).
  constexpr int kBlocks = S::kCols / kBlock;
  const int64_t kblocks = C / kBlock, blk = c0 / kBlock + (lane & (kBlocks - 1));
  const int step_token = lane / kBlocks;

  auto issue = [&](int i) {
    if (i < n) {
      uint8_t* st = ring + (i % kCsStages) * S::kStageBytes;
      const int64_t m = m0 + static_cast<int64_t>(i) * S::kCtaTokens;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int64_t row = m + 2 * t + (q & 1) + (q >> 1) * 8;
        const bool ok = col_ok && row < M;
        cp_async_n<S::kLaneBytes>(st + (q * 32 + lane) * S::kLaneBytes, x.codes + (ok ? row * row_bytes + col_bytes : 0),
                                  ok);
      }
#pragma unroll
      for (int q = 0; q < kCsParts * kRT; ++q) {
        const int chunk = q * 32 + lane;  // of 32 kRT for each part: 2 kRT chunks of 8 j per token
        const int which = chunk / (32 * kRT), rest = chunk % (32 * kRT);
        const int tok = rest / (2 * kRT), c = rest % (2 * kRT);
        const int64_t row = m + tok;
        const uint16_t* src = which == 0 ? vhi : which == 1 ? vlo : vlo2;
        cp_async_n<16>(st + S::kXBytes + which * S::kVBytes + v_chunk<kRT>(tok, c) * 16,
                       src + (row < M ? row * kRankPad + c * 8 : 0), row < M);
      }
    }
    cp_async_commit();
  };
  auto load_step = [&](int i) -> uint32_t {
    if constexpr (S::kDense) return 0u;
    const int64_t row = m0 + static_cast<int64_t>(i) * S::kCtaTokens + step_token;
    const bool ok = i < n && step_token < 16 && row < M && blk < kblocks;
    return ok ? x.step[row * kblocks + blk] : 0u;
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
    uint32_t s2[2] = {0u, 0u};
    if constexpr (!S::kDense) {
      const int b = g * S::kCB / kBlock;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int tok = 2 * t + 8 * h;
        const uint32_t lo = __shfl_sync(0xffffffffu, my_step, tok * kBlocks + b);
        const uint32_t hi = __shfl_sync(0xffffffffu, my_step, (tok + 1) * kBlocks + b);
        s2[h] = lo | (hi << 16);
      }
    }
    // The lane's columns of its four rows (wide reads: by words they would conflict).
    uint32_t xr[4][S::kLaneBytes / 4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint8_t* src = st + (q * 32 + lane) * S::kLaneBytes;
      if constexpr (S::kLaneBytes == 16) {
        const uint4 v = *reinterpret_cast<const uint4*>(src);
        xr[q][0] = v.x, xr[q][1] = v.y, xr[q][2] = v.z, xr[q][3] = v.w;
      } else {
        const uint2 v = *reinterpret_cast<const uint2*>(src);
        xr[q][0] = v.x, xr[q][1] = v.y;
      }
    }
    // Four columns at a time: their B registers, then the parts of V one after
    // the other, so that an accumulator is used again 4 kRT MMAs later.
#pragma unroll
    for (int w = 0; w < S::kCB / 4; ++w) {
      uint32_t bf[4][2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if constexpr (S::kDense) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            bf[2 * e][h] = __byte_perm(xr[2 * h][2 * w + e], xr[2 * h + 1][2 * w + e], 0x5410);
            bf[2 * e + 1][h] = __byte_perm(xr[2 * h][2 * w + e], xr[2 * h + 1][2 * w + e], 0x7632);
          }
        } else {
          // Byte pairs (row 2t, row 2t + 1) of the word's four columns.
          const uint32_t p0 = __byte_perm(xr[2 * h][w], xr[2 * h + 1][w], 0x5140);
          const uint32_t p1 = __byte_perm(xr[2 * h][w], xr[2 * h + 1][w], 0x7362);
          bf[0][h] = act8_decode2<kFormat, 0>(p0, s2[h]);
          bf[1][h] = act8_decode2<kFormat, 2>(p0, s2[h]);
          bf[2][h] = act8_decode2<kFormat, 0>(p1, s2[h]);
          bf[3][h] = act8_decode2<kFormat, 2>(p1, s2[h]);
        }
      }
#pragma unroll
      for (int v = 0; v < kCsParts; ++v)
#pragma unroll
        for (int a = 0; a < kRT; ++a) {
          // Stored rows are tokens: matrices (tokens 0-7, j lo), (0-7, j hi), (8-15, j lo), (8-15, j hi).
          uint32_t af[4];
          ldmatrix_x4_trans(af, smem_u32(st + S::kXBytes + v * S::kVBytes) +
                                    v_chunk<kRT>((mat >> 1) * 8 + rr, a * 2 + (mat & 1)) * 16);
#pragma unroll
          for (int e = 0; e < 4; ++e) mma_16816(acc[a][4 * w + e], af, bf[e]);
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
    for (int c = 0; c < 4; ++c) {
      float* dst = mine + (a * 16 + g + (c >> 1) * 8) * S::kRedPitch + (2 * t + (c & 1)) * S::kCB;
#pragma unroll
      for (int b = 0; b < S::kCB; b += 4)
        *reinterpret_cast<float4*>(dst + b) =
            make_float4(acc[a][b][c], acc[a][b + 1][c], acc[a][b + 2][c], acc[a][b + 3][c]);
    }
  __syncthreads();
  constexpr int kOut = kRT * 16 * S::kCtaCols / 4;  // in fours
  for (int o = threadIdx.x; o < kOut; o += S::kThreads) {
    const int j = o / (S::kCtaCols / 4), c = o % (S::kCtaCols / 4) * 4;
    const float* src = red + (c / S::kCols) * (kRT * 16 * S::kRedPitch) + j * S::kRedPitch + c % S::kCols;
    float4 s = *reinterpret_cast<const float4*>(src);
#pragma unroll
    for (int q = 1; q < S::kWT; ++q) {
      const float4 o4 = *reinterpret_cast<const float4*>(src + q * (kCsWC * kRT * 16 * S::kRedPitch));
      s.x += o4.x, s.y += o4.y, s.z += o4.z, s.w += o4.w;
    }
    const int64_t k = static_cast<int64_t>(blockIdx.x) * S::kCtaCols + c;
    if (k < C) *reinterpret_cast<float4*>(part + (static_cast<int64_t>(z) * (kRT * 16) + j) * C + k) = s;
  }
}

// dst(j, k) = scale sum_z part[z][j][k]; part has r16 = 16 ceil(r / 16) rows
// per split.  A CTA takes 32 columns of 16 j: four columns of one j per
// thread.  [cols][r] outputs leave through shared memory, 16 j side by side.
constexpr int kCrCols = 32;

__global__ void __launch_bounds__(128) act8_colsum_reduce_kernel(const float* __restrict__ part, int64_t C, int r,
                                                                 int splits, float scale, float* __restrict__ dst,
                                                                 int dst_rc) {
  __shared__ float tile[kCrCols][17];
  pdl_wait_prior();
  const int64_t c0 = static_cast<int64_t>(blockIdx.x) * kCrCols;
  const int jj = threadIdx.x / (kCrCols / 4), cc = threadIdx.x % (kCrCols / 4) * 4, j = blockIdx.y * 16 + jj;
  const int64_t slice = static_cast<int64_t>(gridDim.y) * 16 * C;
  if (j < r && c0 + cc < C) {
    const float* src = part + j * C + c0 + cc;
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
    for (int z = 0; z < splits; ++z) {
      const float4 p = *reinterpret_cast<const float4*>(src + z * slice);
      s.x += p.x, s.y += p.y, s.z += p.z, s.w += p.w;
    }
    const float v[4] = {scale * s.x, scale * s.y, scale * s.z, scale * s.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (dst_rc)
        dst[j * C + c0 + cc + e] = v[e];
      else
        tile[cc + e][jj] = v[e];
    }
  }
  if (dst_rc) return;
  __syncthreads();
#pragma unroll
  for (int i = threadIdx.x; i < kCrCols * 16; i += 128) {
    const int c = i / 16, q = i % 16;
    if (c0 + c < C && blockIdx.y * 16 + q < r) dst[(c0 + c) * r + blockIdx.y * 16 + q] = tile[c][q];
  }
}

namespace {

template <int kFormat>
int64_t colsum_partial_rows(int64_t M, int64_t C) {
  const int64_t rows[4] = {16 * int64_t{ColsumShape<kFormat, 1>::splits(M, C)},
                           32 * int64_t{ColsumShape<kFormat, 2>::splits(M, C)},
                           48 * int64_t{ColsumShape<kFormat, 3>::splits(M, C)},
                           64 * int64_t{ColsumShape<kFormat, 4>::splits(M, C)}};
  int64_t most = 0;
  for (const int64_t v : rows) most = v > most ? v : most;
  return most;
}

template <int kFormat, int kRT>
cudaError_t launch_colsum_rt(const Act8View& x, const uint16_t* hi, const uint16_t* lo, const uint16_t* lo2,
                             float* part, int* splits, cudaStream_t stream) {
  using S = ColsumShape<kFormat, kRT>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  static DeviceOnce configured;
  e = configured.run(dev, [] {
    return cudaFuncSetAttribute(act8_colsum_kernel<kFormat, kRT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                S::kSmem);
  });
  if (e != cudaSuccess) return e;
  *splits = S::splits(x.rows, x.cols);
  const dim3 grid(static_cast<unsigned>((x.cols + S::kCtaCols - 1) / S::kCtaCols), static_cast<unsigned>(*splits));
  act8_colsum_kernel<kFormat, kRT><<<grid, S::kThreads, S::kSmem, stream>>>(x, hi, lo, lo2, *splits, part);
  return cudaGetLastError();
}

template <int kFormat>
cudaError_t launch_colsum_format(const Act8View& x, const uint16_t* hi, const uint16_t* lo, const uint16_t* lo2,
                                 int rt, float* part, int* splits, cudaStream_t stream) {
  switch (rt) {
    case 1: return launch_colsum_rt<kFormat, 1>(x, hi, lo, lo2, part, splits, stream);
    case 2: return launch_colsum_rt<kFormat, 2>(x, hi, lo, lo2, part, splits, stream);
    case 3: return launch_colsum_rt<kFormat, 3>(x, hi, lo, lo2, part, splits, stream);
    default: return launch_colsum_rt<kFormat, 4>(x, hi, lo, lo2, part, splits, stream);
  }
}

}  // namespace

size_t act8_colsum_partial_bytes(int64_t M, int64_t C) {
  const int64_t codes = colsum_partial_rows<kAct8Int8>(M, C), dense = colsum_partial_rows<kAct8Dense>(M, C);
  return static_cast<size_t>(codes > dense ? codes : dense) * static_cast<size_t>(C) * sizeof(float);
}

cudaError_t launch_act8_colsum(const Act8View& x, const uint16_t* hi, const uint16_t* lo, const uint16_t* lo2, int r,
                               float scale, float* part, float* dst, bool dst_rc, cudaStream_t stream) {
  const int rt = (r + 15) / 16;
  int splits = 0;
  const cudaError_t e =
      x.format == kAct8Dense  ? launch_colsum_format<kAct8Dense>(x, hi, lo, lo2, rt, part, &splits, stream)
      : x.format == kAct8Int8 ? launch_colsum_format<kAct8Int8>(x, hi, lo, lo2, rt, part, &splits, stream)
                              : launch_colsum_format<kAct8E4m3>(x, hi, lo, lo2, rt, part, &splits, stream);
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>((x.cols + kCrCols - 1) / kCrCols), static_cast<unsigned>(rt));
  return launch_dependent(act8_colsum_reduce_kernel, grid, 128, 0, stream, part, x.cols, r, splits, scale, dst,
                          dst_rc ? 1 : 0);
}

// ---------------------------------------------------------------------------
// skinny: part[z][m][j] = sum_{k in split z} X^[m][k] A[j][k]
// ---------------------------------------------------------------------------
// m16n8k16 MMAs with D = [16 tokens][8 j], K = the columns.  Which column a K
// slot stands for is free as long as both operands agree: in each half (32
// columns) of a 64-column block lane (g, t) takes columns 8t .. 8t + 7, of its
// token rows (8 code bytes) and of its rows of A (16 bytes), and MMA step s of
// the half takes columns 8t + 4s .. + 3 as the lane's four slots.  Every load
// is 8 or 16 bytes and feeds its registers as it is.
//
// A CTA is kSkWT groups of 32 tokens x kSkWK column shares.  The shares' blocks
// of A come through a ring in shared memory (read through L1, the rows of a
// block, 2 K bytes apart, evict each other where K is a power of two: five
// times slower at K = 8192), and the shares' sums are added in shared memory
// in a fixed order.  The codes and steps of a warp's next block are loaded
// before its current one is multiplied.
namespace {

constexpr int kSkWT = 4, kSkWK = 2;
constexpr int kSkWarps = kSkWT * kSkWK;
constexpr int kSkMT = 2;  // 16-token tiles of a warp
constexpr int kSkWarpTokens = kSkMT * 16, kSkTokens = kSkWT * kSkWarpTokens;
constexpr int kSkStages = 3;

template <int NT>
struct SkinnyShape {
  static constexpr int kTile = NT * 8 * 128;  // one block of A: [j][64 columns]
  static constexpr int kRing = kSkStages * kSkWK * kTile;
  static constexpr int kPitch = NT * 8 + 8;   // floats: rows g apart by 8 banks, so the lanes' pairs never meet
  static constexpr int kSums = kSkWK * kSkTokens * kPitch * static_cast<int>(sizeof(float));
  static constexpr int kSmem = kRing > kSums ? kRing : kSums;
};

// Byte offset of 16-byte chunk c of row j in a block of A: odd rows have their
// halves exchanged, so that two rows' 64 bytes make a conflict-free read.
__device__ __forceinline__ int sk_chunk(int j, int c) { return j * 128 + (c ^ ((j & 1) << 2)) * 16; }

int act8_skinny_splits(int64_t M, int64_t K) {
  const int64_t tiles = (M + kSkTokens - 1) / kSkTokens, blocks = K / kBlock;
  int64_t s = 148 / tiles;  // one wave of a CTA per SM
  if (s < 1) s = 1;
  const int64_t most = (blocks + kSkWK - 1) / kSkWK;  // a block per warp at least
  if (s > most) s = most;
  const int64_t room = skinny_splits(M, K);  // what the workspace's partials are sized for
  return static_cast<int>(s < room ? s : room);
}

template <int kFormat>
struct SkinnyX {  // one lane's part of a 64-column block of 32 tokens
  uint2 c[kSkMT][2][2];     // [tile][row g, g + 8][half]
  uint32_t s[kSkMT][2];     // packed steps

  __device__ __forceinline__ void load(const uint8_t* codes, const uint16_t* step, int64_t M, int64_t K, int64_t m0,
                                       int64_t kb, bool live) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int a = 0; a < kSkMT; ++a)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t row = m0 + a * 16 + h * 8 + g;
        const bool ok = live && row < M;
        const uint2* src = reinterpret_cast<const uint2*>(codes + (ok ? row * K + kb * kBlock + t * 8 : 0));
        c[a][h][0] = ok ? __ldg(src) : make_uint2(0, 0);
        c[a][h][1] = ok ? __ldg(src + 4) : make_uint2(0, 0);
        s[a][h] = ok ? __ldg(step + row * (K / kBlock) + kb) : 0u;
      }
  }
};

}  // namespace

template <int kFormat, int NT>
__global__ void __launch_bounds__(32 * kSkWarps) act8_skinny_kernel(const uint8_t* __restrict__ codes,
                                                                    const uint16_t* __restrict__ step,
                                                                    const uint16_t* __restrict__ A, int64_t M,
                                                                    int64_t K, int r, int splits,
                                                                    float* __restrict__ part) {
  using S = SkinnyShape<NT>;
  constexpr int kPitch = S::kPitch;
  extern __shared__ __align__(16) uint8_t ring[];
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3, wt = warp % kSkWT, wk = warp / kSkWT;
  const int64_t m0 = static_cast<int64_t>(blockIdx.x) * kSkTokens + wt * kSkWarpTokens;
  const int z = blockIdx.y;
  const int64_t kblocks = K / kBlock;
  const int64_t first = kblocks * z / splits, b1 = kblocks * (z + 1) / splits;
  const int steps = static_cast<int>((b1 - first + kSkWK - 1) / kSkWK);  // of kSkWK blocks

  auto issue = [&](int i) {
    if (i < steps) {
      uint8_t* st = ring + (i % kSkStages) * (kSkWK * S::kTile);
#pragma unroll
      for (int q = 0; q < kSkWK * S::kTile / 16 / (32 * kSkWarps); ++q) {
        const int chunk = q * (32 * kSkWarps) + threadIdx.x;
        const int share = chunk / (S::kTile / 16), rest = chunk % (S::kTile / 16), j = rest / 8, c = rest % 8;
        const int64_t kb = first + static_cast<int64_t>(i) * kSkWK + share;
        const bool ok = j < r && kb < b1;
        cp_async_16(st + share * S::kTile + sk_chunk(j, c), A + (ok ? j * K + kb * kBlock + c * 8 : 0), ok);
      }
    }
    cp_async_commit();
  };

  float acc[kSkMT][NT][4];
#pragma unroll
  for (int a = 0; a < kSkMT; ++a)
#pragma unroll
    for (int b = 0; b < NT; ++b)
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[a][b][c] = 0.0f;

#pragma unroll
  for (int i = 0; i < kSkStages - 1; ++i) issue(i);
  SkinnyX<kFormat> next;
  next.load(codes, step, M, K, m0, first + wk, first + wk < b1);
  for (int i = 0; i < steps; ++i) {
    const int64_t kb = first + static_cast<int64_t>(i) * kSkWK + wk;
    SkinnyX<kFormat> x = next;
    next.load(codes, step, M, K, m0, kb + kSkWK, kb + kSkWK < b1);
    cp_async_wait<kSkStages - 2>();
    __syncthreads();  // everyone's copies of this stage are there, and the one before is read
    issue(i + kSkStages - 1);
    const uint8_t* tile = ring + (i % kSkStages) * (kSkWK * S::kTile) + wk * S::kTile;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      uint4 av[NT];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        av[nt] = *reinterpret_cast<const uint4*>(tile + sk_chunk(nt * 8 + g, half * 4 + t));
#pragma unroll
      for (int w = 0; w < 2; ++w) {  // columns 8t + 4w .. + 3 of the half
        uint32_t af[kSkMT][4];
#pragma unroll
        for (int a = 0; a < kSkMT; ++a)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t word = w == 0 ? x.c[a][h][half].x : x.c[a][h][half].y;
            const uint32_t s2 = x.s[a][h] | (x.s[a][h] << 16);
            af[a][h] = act8_decode2<kFormat, 0>(word, s2);
            af[a][h + 2] = act8_decode2<kFormat, 2>(word, s2);
          }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const uint32_t bf[2] = {w == 0 ? av[nt].x : av[nt].z, w == 0 ? av[nt].y : av[nt].w};
#pragma unroll
          for (int a = 0; a < kSkMT; ++a) mma_16816(acc[a][nt], af[a], bf);
        }
      }
    }
  }
  cp_async_wait<0>();
  __syncthreads();  // the ring's space takes the sums
  float* sums = reinterpret_cast<float*>(ring);  // [kSkWK][kSkTokens][kPitch]
#pragma unroll
  for (int a = 0; a < kSkMT; ++a)
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        *reinterpret_cast<float2*>(sums + ((wk * kSkTokens) + wt * kSkWarpTokens + a * 16 + h * 8 + g) * kPitch + nt * 8 +
                                   2 * t) = make_float2(acc[a][nt][2 * h], acc[a][nt][2 * h + 1]);
  __syncthreads();
  constexpr int kOut = kSkTokens * NT * 2;  // in fours
  for (int i = threadIdx.x; i < kOut; i += 32 * kSkWarps) {
    const int m = i / (NT * 2), j = i % (NT * 2) * 4;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * kSkTokens + m;
    if (row >= M) break;
    float4 s = *reinterpret_cast<const float4*>(sums + m * kPitch + j);
#pragma unroll
    for (int w = 1; w < kSkWK; ++w) {
      const float4 o = *reinterpret_cast<const float4*>(sums + (w * kSkTokens + m) * kPitch + j);
      s.x += o.x, s.y += o.y, s.z += o.z, s.w += o.w;
    }
    *reinterpret_cast<float4*>(part + (static_cast<int64_t>(z) * M + row) * kRankPad + j) = s;
  }
}

namespace {

template <int kFormat, int NT>
cudaError_t launch_skinny_nt(const Act8View& x, const uint16_t* A, int r, int splits, float* part,
                             cudaStream_t stream) {
  constexpr int smem = SkinnyShape<NT>::kSmem;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  static DeviceOnce configured;
  e = configured.run(dev, [] {
    return cudaFuncSetAttribute(act8_skinny_kernel<kFormat, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  });
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>((x.rows + kSkTokens - 1) / kSkTokens), static_cast<unsigned>(splits));
  act8_skinny_kernel<kFormat, NT><<<grid, 32 * kSkWarps, smem, stream>>>(x.codes, x.step, A, x.rows, x.cols, r, splits,
                                                                        part);
  return cudaGetLastError();
}

template <int kFormat>
cudaError_t launch_skinny_format(const Act8View& x, const uint16_t* A, int r, int splits, float* part,
                                 cudaStream_t stream) {
  switch ((r + 15) / 16) {
    case 1: return launch_skinny_nt<kFormat, 2>(x, A, r, splits, part, stream);
    case 2: return launch_skinny_nt<kFormat, 4>(x, A, r, splits, part, stream);
    case 3: return launch_skinny_nt<kFormat, 6>(x, A, r, splits, part, stream);
    default: return launch_skinny_nt<kFormat, 8>(x, A, r, splits, part, stream);
  }
}

}  // namespace

cudaError_t launch_act8_skinny(const Act8View& x, const uint16_t* A, int r, float* part, const SkinnyOut& out,
                               cudaStream_t stream) {
  const int splits = act8_skinny_splits(x.rows, x.cols);
  const cudaError_t e = x.format == kAct8Int8 ? launch_skinny_format<kAct8Int8>(x, A, r, splits, part, stream)
                                              : launch_skinny_format<kAct8E4m3>(x, A, r, splits, part, stream);
  if (e != cudaSuccess) return e;
  return launch_skinny_finalize(part, x.rows, r, splits, out, stream);
}

}  // namespace qnf4
