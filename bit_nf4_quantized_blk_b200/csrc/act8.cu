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
// One tcgen05 product D[columns k][j] with the token axis as K.  Both operands
// are MN-major, so rows of tokens go to shared memory as they are: A is the
// X^ tile, B the three parts of V side by side (N = 192), so that A, whose
// reads bound the MMA at a small N, is read once for all three.  Their sums
// stay apart in tensor memory until the epilogue adds them.
//
// A CTA takes 256 columns (two M = 128 tiles) and a range of the tokens, 64 per
// step.  Warps 0-15 decode: each thread copies its 16 codes of two tokens to
// its own shared-memory slots four steps ahead (cp.async, read back by the same
// thread, so without a barrier), and writes them as bf16 in the 128-byte
// swizzle the descriptors name.  Warp 16 brings the parts of V by TMA (and X
// itself where it is plain bf16: dB, from dY and U), warp 17 issues the MMAs.
// At the end warps 0-15 read the accumulators: a lane is a column, so each j
// leaves as 128 contiguous bytes per warp.  Every barrier wait is bounded.
//
// The decoders' instructions bound it (about 1,500 cycles per step, the MMAs
// take 640), and some 6 us of launch, first loads and epilogue: 15.3 us at
// 1999 x 8192 and rank 64 (16.8 MB of codes), 7.7 us for dY at 1999 x 2048.
// Warp-level MMAs from registers, the same sums: 29.9 and 12 us.
namespace {

constexpr int kCsTok = 64;                          // tokens per step
constexpr int kCsCols = 256;                        // columns of a CTA
constexpr int kCsStages = 3;                        // operand tiles
constexpr int kCsSlots = 3;                         // code slots: steps in flight
constexpr int kCsParts = 3;                         // bf16 parts of V
constexpr int kCsBox = kCsTok * 128;                // [64 tokens][64 columns or j] bf16
constexpr int kCsXTile = kCsCols / 64 * kCsBox;
constexpr int kCsStage = kCsXTile + kCsParts * kCsBox;
constexpr int kCsDecoders = 512;                    // threads
constexpr int kCsWarps = kCsDecoders / 32;
constexpr int kCsThreads = kCsDecoders + 64;
constexpr int kCsPasses = kCsTok * kCsCols / 16 / kCsDecoders;  // 16 codes per thread and pass
constexpr int kCsSlot = kCsPasses * kCsDecoders * 16;
constexpr int kCsN = kCsParts * kRankPad;           // MMA N
constexpr uint32_t kCsTmemCols = 512;               // two tiles of kCsN, in a power of two
constexpr int kCsBarriers = 256;

template <int kFormat>
constexpr int kCsSmem = 1024 + kCsStages * kCsStage + kCsBarriers + (kFormat == kAct8Dense ? 0 : kCsSlots * kCsSlot);

struct CsBarriers {
  uint64_t x_full[kCsStages];  // decoded: one arrival per decoder warp
  uint64_t full[kCsStages];    // TMA
  uint64_t empty[kCsStages];
  uint64_t done, drain;
  uint32_t tmem;
  int abort_flag;
};

// Splits of the tokens: one wave of one CTA per SM on a 148-SM B200.
int cs_splits(int64_t M, int64_t C) {
  const int64_t cols = (C + kCsCols - 1) / kCsCols, steps = (M + kCsTok - 1) / kCsTok;
  int64_t s = 148 / cols;
  if (s > steps) s = steps;
  return static_cast<int>(s < 1 ? 1 : s);
}

__device__ __forceinline__ bool cs_warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* status) {
  bool ok = true;
  if ((threadIdx.x & 31) == 0) ok = mbar_wait(bar, parity, abort_flag, status);
  ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
  if (ok) (void)mbar_try_wait(bar, parity);
  return ok;
}

// tcgen05.wait::ld that hands the loaded registers on, so no use of them can
// be scheduled before the wait.
__device__ __forceinline__ void cs_wait_ld(uint32_t (&r)[kCsParts][16]) {
#pragma unroll
  for (int i = 0; i < kCsParts; ++i)
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[i][0]), "+r"(r[i][1]), "+r"(r[i][2]), "+r"(r[i][3]), "+r"(r[i][4]), "+r"(r[i][5]),
                   "+r"(r[i][6]), "+r"(r[i][7]), "+r"(r[i][8]), "+r"(r[i][9]), "+r"(r[i][10]), "+r"(r[i][11]),
                   "+r"(r[i][12]), "+r"(r[i][13]), "+r"(r[i][14]), "+r"(r[i][15])
                 :
                 : "memory");
}

}  // namespace

template <int kFormat>
__global__ void __launch_bounds__(kCsThreads, 1)
    act8_colsum_kernel(Act8View x, const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmHi,
                       const __grid_constant__ CUtensorMap tmLo, const __grid_constant__ CUtensorMap tmLo2, int r16,
                       int splits, float* __restrict__ part, int* status) {
  constexpr bool kDense = kFormat == kAct8Dense;
  extern __shared__ uint8_t smem_raw[];
  pdl_launch_dependents();
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  CsBarriers* bars = reinterpret_cast<CsBarriers*>(smem + kCsStages * kCsStage);
  uint8_t* slots = smem + kCsStages * kCsStage + kCsBarriers;
  volatile int* abort_flag = &bars->abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t M = x.rows, C = x.cols;
  const int64_t c0 = static_cast<int64_t>(blockIdx.x) * kCsCols;
  const int z = blockIdx.y;
  const int64_t total = (M + kCsTok - 1) / kCsTok, first = total * z / splits;
  const int n = static_cast<int>(total * (z + 1) / splits - first);  // steps, at least one

  if (tid == 0) {
    for (int s = 0; s < kCsStages; ++s) {
      mbar_init(&bars->x_full[s], kCsWarps);
      mbar_init(&bars->full[s], 1);
      mbar_init(&bars->empty[s], 1);
    }
    mbar_init(&bars->done, 1);
    mbar_init(&bars->drain, 1);
    bars->abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kCsWarps + 1) {
    tmem_alloc(&bars->tmem, kCsTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem;

  if (warp == kCsWarps) {
    if (lane == 0) {
      int issued = 0;
      for (int i = 0; i < n; ++i) {
        const int s = i % kCsStages, u = i / kCsStages;
        if (i >= kCsStages && !mbar_wait(&bars->empty[s], (u - 1) & 1, abort_flag, status)) break;
        uint8_t* st = smem + s * kCsStage;
        const int m = static_cast<int>((first + i) * kCsTok);
        mbar_arrive_expect_tx(&bars->full[s], kDense ? kCsStage : kCsParts * kCsBox);
        if constexpr (kDense)
          for (int g = 0; g < kCsCols / 64; ++g)
            tma_load_2d(st + g * kCsBox, &tmX, &bars->full[s], static_cast<int>(c0) + g * 64, m);
        tma_load_2d(st + kCsXTile, &tmHi, &bars->full[s], 0, m);
        tma_load_2d(st + kCsXTile + kCsBox, &tmLo, &bars->full[s], 0, m);
        tma_load_2d(st + kCsXTile + 2 * kCsBox, &tmLo2, &bars->full[s], 0, m);
        issued = i + 1;
      }
      // Every copy into shared memory has landed before the CTA can exit.
      for (int i = (issued > kCsStages ? issued - kCsStages : 0); i < issued; ++i)
        mbar_wait_teardown(&bars->full[i % kCsStages], (i / kCsStages) & 1, status);
    }
  } else if (warp == kCsWarps + 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_bf16_f32(128, kCsN, true) | (1u << 15);  // A and B MN-major
      // Groups of 64 columns (or of 64 j: one part) are a box apart, groups of
      // 8 tokens 1 KB; a K = 16 step is 16 tokens = 2 KB.
      const uint64_t a0 = smem_desc_mn128(smem_u32(smem), kCsBox, 1024);
      bool ok = true;
      for (int u = 0; ok && u * kCsStages < n; ++u)
#pragma unroll
        for (int s = 0; s < kCsStages; ++s) {
          const int i = u * kCsStages + s;
          if (!ok || i >= n) break;
          ok = mbar_wait(&bars->full[s], u & 1, abort_flag, status) &&
               (kDense || mbar_wait(&bars->x_full[s], u & 1, abort_flag, status));
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int kk = 0; kk < kCsTok / 16; ++kk)
              tc_mma_bf16_ss(tmem + static_cast<uint32_t>(h * 256), a0 + ((s * kCsStage + h * 2 * kCsBox + kk * 2048) >> 4),
                             a0 + ((s * kCsStage + kCsXTile + kk * 2048) >> 4), idesc, (i > 0 || kk > 0) ? 1u : 0u);
          tc_commit(&bars->empty[s]);
        }
      if (ok) tc_commit(&bars->done);
      tc_commit(&bars->drain);
      mbar_wait_teardown(&bars->drain, 0, status);
    }
  } else {
    bool ok = true;
    if constexpr (!kDense) {
      constexpr int kPassTok = kCsTok / kCsPasses;
      const int seg = tid % 16, tok0 = tid / 16;  // 16 columns of token tok0 + kPassTok pass
      const int64_t col = c0 + seg * 16;          // in or out of C as a whole
      // Rows left from this thread's first one; none if its columns are not there.
      const int64_t m0 = first * kCsTok + tok0;
      const int rows = col < C ? static_cast<int>(min(M - m0, static_cast<int64_t>(n) * kCsTok)) : 0;
      const uint8_t* const codes = x.codes + (rows > 0 ? m0 * C + col : 0);
      const uint16_t* const steps = x.step + (rows > 0 ? (m0 * C + col) / kBlock : 0);
      uint8_t* const slot = slots + tid * 16;
      auto fetch = [&](int i, int sl) {
        const uint8_t* src = codes + static_cast<int64_t>(i) * (kCsTok * C);
#pragma unroll
        for (int q = 0; q < kCsPasses; ++q) {
          const bool in = i * kCsTok + q * kPassTok < rows;
          cp_async_16(slot + sl * kCsSlot + q * (kCsDecoders * 16), in ? src + q * (kPassTok * C) : codes, in);
        }
        cp_async_commit();
      };
      auto load_steps = [&](int i, uint32_t (&s)[kCsPasses]) {
        const uint16_t* src = steps + static_cast<int64_t>(i) * (kCsTok * C / kBlock);
#pragma unroll
        for (int q = 0; q < kCsPasses; ++q)
          s[q] = i * kCsTok + q * kPassTok < rows ? __ldg(src + q * (kPassTok * C / kBlock)) : 0u;
      };
      // Odd groups of 64 columns take their second eight first, so that the
      // groups of a store meet no bank twice.
      const int group = seg / 4, odd = group & 1, chunk = (seg & 3) * 2, key = tok0 & 7;
      static_assert(kPassTok % 8 == 0, "one swizzle key for all passes");
      const int out0 = group * kCsBox + tok0 * 128 + (((chunk + odd) ^ key) << 4);
      const int out1 = group * kCsBox + tok0 * 128 + (((chunk + 1 - odd) ^ key) << 4);
      // Step i = kCsStages u + st, whose scales are in s; they are replaced by
      // those of step i + kCsStages in place (a copy from a set still loading
      // would wait for it).
      static_assert(kCsStages == kCsSlots, "one index for tiles and slots");
      auto decode = [&](int u, int st, uint32_t (&s)[kCsPasses]) {
        const int i = u * kCsStages + st;
        if (i >= n) return true;
        cp_async_wait<kCsSlots - 1>();
        uint2 c[kCsPasses][2];
#pragma unroll
        for (int q = 0; q < kCsPasses; ++q) {
          const uint8_t* src = slot + st * kCsSlot + q * (kCsDecoders * 16);
          c[q][0] = *reinterpret_cast<const uint2*>(src + odd * 8);
          c[q][1] = *reinterpret_cast<const uint2*>(src + 8 - odd * 8);
        }
        if (u > 0 && !cs_warp_wait(&bars->empty[st], (u - 1) & 1, abort_flag, status)) return false;
        uint8_t* dst = smem + st * kCsStage;
#pragma unroll
        for (int q = 0; q < kCsPasses; ++q) {
          const uint32_t s2 = s[q] | (s[q] << 16);
#pragma unroll
          for (int e = 0; e < 2; ++e)
            *reinterpret_cast<uint4*>(dst + (e == 0 ? out0 : out1) + q * (kPassTok * 128)) =
                make_uint4(act8_decode2<kFormat, 0>(c[q][e].x, s2), act8_decode2<kFormat, 2>(c[q][e].x, s2),
                           act8_decode2<kFormat, 0>(c[q][e].y, s2), act8_decode2<kFormat, 2>(c[q][e].y, s2));
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // before the MMA reads them
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->x_full[st]);
        fetch(i + kCsSlots, st);  // into the slot read above
        load_steps(i + kCsSlots, s);
        return true;
      };
      uint32_t scale[kCsSlots][kCsPasses];
#pragma unroll
      for (int i = 0; i < kCsSlots; ++i) {
        fetch(i, i);
        load_steps(i, scale[i]);
      }
      for (int u = 0; ok && u * kCsStages < n; ++u)
#pragma unroll
        for (int st = 0; st < kCsStages; ++st) ok = ok && decode(u, st, scale[st]);
      cp_async_wait<0>();
    }
    pdl_wait_prior();  // an overlapped launch ends after the kernel before it
    if (ok && cs_warp_wait(&bars->done, 0, abort_flag, status)) {
      tc_fence_after();
      const int quad = warp & 3, h = (warp >> 2) & 1;  // TMEM lanes 32 quad .. + 31 of column tile h
      const uint32_t acc = tmem + (static_cast<uint32_t>(quad * 32) << 16) + static_cast<uint32_t>(h * 256);
      const int64_t k = c0 + h * 128 + quad * 32 + lane;
      for (int j0 = warp / 8 * 16; j0 < r16; j0 += kCsWarps / 8 * 16) {
        uint32_t v[kCsParts][16];
#pragma unroll
        for (int i = 0; i < kCsParts; ++i) tmem_ld_32x32b_x16(acc + static_cast<uint32_t>(i * kRankPad + j0), v[i]);
        cs_wait_ld(v);
        if (k >= C) continue;
        float* dst = part + (static_cast<int64_t>(z) * r16 + j0) * C + k;
#pragma unroll
        for (int j = 0; j < 16; ++j)
          dst[j * C] = __uint_as_float(v[0][j]) + (__uint_as_float(v[1][j]) + __uint_as_float(v[2][j]));
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kCsWarps + 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kCsTmemCols);
  }
}

// dst(j, k) = scale sum_z part[z][j][k]; part has r16 = 16 ceil(r / 16) rows
// per split.  A CTA takes 32 columns of 16 j: four columns of one j per
// thread.  [cols][r] outputs leave through shared memory, 16 j side by side.
// The CTAs of a second job follow the first's.
constexpr int kCrCols = 32;

struct ColsumReduceJob {
  const float* part;
  int64_t C;
  int splits;
  float* dst;
  int dst_rc;
};

__global__ void __launch_bounds__(128)
    act8_colsum_reduce_kernel(const __grid_constant__ ColsumReduceJob job0, const __grid_constant__ ColsumReduceJob job1,
                              unsigned first, int r, float scale) {
  __shared__ float tile[kCrCols][17];
  pdl_wait_prior();
  const ColsumReduceJob& job = blockIdx.x < first ? job0 : job1;
  const float* __restrict__ part = job.part;
  float* __restrict__ dst = job.dst;
  const int64_t C = job.C;
  const int splits = job.splits, dst_rc = job.dst_rc;
  const int64_t c0 = static_cast<int64_t>(blockIdx.x < first ? blockIdx.x : blockIdx.x - first) * kCrCols;
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
cudaError_t launch_colsum_format(const Act8View& x, const CUtensorMap (&maps)[4], int r16, int splits, float* part,
                                 bool overlap, int* status, cudaStream_t stream) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  static DeviceOnce configured;
  e = configured.run(dev, [] {
    return cudaFuncSetAttribute(act8_colsum_kernel<kFormat>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kCsSmem<kFormat>);
  });
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>((x.cols + kCsCols - 1) / kCsCols), static_cast<unsigned>(splits));
  if (overlap)
    return launch_dependent(act8_colsum_kernel<kFormat>, grid, kCsThreads, kCsSmem<kFormat>, stream, x, maps[0], maps[1],
                            maps[2], maps[3], r16, splits, part, status);
  act8_colsum_kernel<kFormat><<<grid, kCsThreads, kCsSmem<kFormat>, stream>>>(x, maps[0], maps[1], maps[2], maps[3], r16,
                                                                             splits, part, status);
  return cudaGetLastError();
}

}  // namespace

size_t act8_colsum_partial_bytes(int64_t M, int64_t C) {
  return static_cast<size_t>(cs_splits(M, C)) * kRankPad * static_cast<size_t>(C) * sizeof(float);
}

cudaError_t launch_act8_colsums(const ColsumJob* jobs, int count, int r, float scale, int* status,
                                cudaStream_t stream) {
  const int rt = (r + 15) / 16;
  ColsumReduceJob reduce[2];
  unsigned blocks[2] = {0, 0};
  for (int i = 0; i < count; ++i) {
    const ColsumJob& job = jobs[i];
    const Act8View& x = job.x;
    const bool dense = x.format == kAct8Dense, overlap = i > 0;
    const uint16_t* parts[kCsParts] = {job.hi, job.lo, job.lo2};
    CUtensorMap maps[4];  // X (plain bf16 only; else any valid map) and the parts of V
    for (int q = 0; q < kCsParts; ++q)
      if (!encode_tensor_map_2d(&maps[1 + q], parts[q], x.rows, kRankPad, kCsTok, 64)) return cudaErrorInvalidValue;
    maps[0] = maps[1];
    if (dense && !encode_tensor_map_2d(&maps[0], x.codes, x.rows, x.cols, kCsTok, 64)) return cudaErrorInvalidValue;
    const int splits = cs_splits(x.rows, x.cols);
    const cudaError_t e =
        dense ? launch_colsum_format<kAct8Dense>(x, maps, 16 * rt, splits, job.part, overlap, status, stream)
        : x.format == kAct8Int8
            ? launch_colsum_format<kAct8Int8>(x, maps, 16 * rt, splits, job.part, overlap, status, stream)
            : launch_colsum_format<kAct8E4m3>(x, maps, 16 * rt, splits, job.part, overlap, status, stream);
    if (e != cudaSuccess) return e;
    reduce[i] = ColsumReduceJob{job.part, x.cols, splits, job.dst, job.dst_rc ? 1 : 0};
    blocks[i] = static_cast<unsigned>((x.cols + kCrCols - 1) / kCrCols);
  }
  const dim3 grid(blocks[0] + blocks[1], static_cast<unsigned>(rt));
  return launch_dependent(act8_colsum_reduce_kernel, grid, 128, 0, stream, reduce[0], reduce[count - 1], blocks[0], r,
                          scale);
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

cudaError_t launch_act8_skinny(const Act8View& x, const uint16_t* A, int r, float* part, int* splits,
                               cudaStream_t stream) {
  *splits = act8_skinny_splits(x.rows, x.cols);
  return x.format == kAct8Int8 ? launch_skinny_format<kAct8Int8>(x, A, r, *splits, part, stream)
                               : launch_skinny_format<kAct8E4m3>(x, A, r, *splits, part, stream);
}

}  // namespace qnf4
