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
//                          per value): 8192 x 14336 in 54 us, 6.6 TB/s.
//  act8_dequantize_kernel  the reverse: 51 us.
//  act8_colsum_kernel      part[z][j][k] = sum over the tokens m of split z of
//                          V[m][j] X^[m][k], then act8_colsum_reduce_kernel
//                          adds the splits in a fixed order (dA).
//  act8_rowsum_kernel      part[z][m][j] = sum over the columns of split z of
//                          X^[m][k] A[j][k] (U), or of dY[m][k] B[k][j] (V).
// Deterministic: every sum runs in a fixed order; no atomics.
#include <algorithm>

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
// Decoded tiles for the tensor cores
// ---------------------------------------------------------------------------
// Both products below are tcgen05 MMAs whose A operand is X^.  Warps 0-15
// decode: per step each thread takes two runs of 16 codes, which it copies to
// its own shared-memory slots three steps ahead (cp.async; read back by the
// same thread, so without a barrier), and writes them as bf16 in the 128-byte
// swizzle that the descriptors name.  Warp 16 brings the other operand by TMA
// (and X itself where it is plain bf16), warp 17 issues the MMAs.  At the end
// warps 0-15 read the accumulators.  Every barrier wait is bounded.
namespace {

constexpr int kTcDecoders = 512;  // threads
constexpr int kTcWarps = kTcDecoders / 32;
constexpr int kTcThreads = kTcDecoders + 64;
constexpr int kTcStages = 3;      // tiles, and code slots, in flight
constexpr int kTcPasses = 2;      // runs of 16 codes per thread and step
constexpr int kTcSlot = kTcPasses * kTcDecoders * 16;
constexpr int kTcBarriers = 256;

// The CTAs of one or two products: `tiles` independent ones, each with `splits`
// CTAs that share its `steps`.  `splits` enters as that product alone would have
// it: whole waves of a CTA per SM (148).
struct TcWork {
  int64_t tiles, steps;
  bool dense;
  int splits;
};

// Two products share one wave where that takes no longer than one after the
// other: nothing then waits for the first to end, and fewer splits leave fewer
// partials.  In units of half a microsecond a step of plain bf16 takes 1, one
// with decoding 2, and a second wave's start 4.  GPU time of the backward without
// dX, U recomputed, both pairs in turn and so: 1999 x 2048 x 8192, rank 64, 41.9
// and 33.6 us; 512 x 4096 x 4096, rank 64, 30.3 and 24.1; 2048 x 1024 x 4096, rank
// 32, 29.7 and 25.3.  A second wave's start of 0 units leaves the second of these
// at 30.2, one of 12 changes none by more than 1%.
void tc_share_wave(TcWork& a, TcWork& b) {
  auto time = [](const TcWork& w, int64_t splits) {
    return (w.tiles * splits + 147) / 148 * ((w.steps + splits - 1) / splits) * (w.dense ? 1 : 2);
  };
  int64_t best = time(a, a.splits) + time(b, b.splits) + 4;
  const TcWork a0 = a, b0 = b;
  for (int64_t s = 1; s <= a0.splits; ++s) {
    const int64_t left = (148 - a0.tiles * s) / b0.tiles, sb = left < b0.splits ? left : b0.splits;
    if (a0.tiles * s >= 148 || sb < 1) break;
    // 32 steps add 64 times in a row: 6 10^-7 of a sum that the tensor core truncates
    // (8192 x 4096 x 4096, rank 64: 77.0 us, dB off by 5.9e-7; with up to 64 steps 73.3
    // us and 1.5e-6, twice an fp32 product's 7.8e-7).
    if ((a0.steps + s - 1) / s > 32 || (b0.steps + sb - 1) / sb > 32) continue;
    const int64_t ta = time(a0, s), tb = time(b0, sb), t = ta > tb ? ta : tb;
    if (t <= best) best = t, a.splits = static_cast<int>(s), b.splits = static_cast<int>(sb);
  }
}

struct TcBarriers {
  uint64_t x_full[kTcStages];  // decoded: one arrival per decoder warp
  uint64_t full[kTcStages];    // TMA
  uint64_t empty[kTcStages];
  uint64_t done, drain;
  uint32_t tmem;
  int abort_flag;
};
static_assert(sizeof(TcBarriers) <= kTcBarriers, "room for the barriers");

template <int kFormat>
constexpr int tc_smem(int stage) {
  return 1024 + kTcStages * stage + kTcBarriers + (kFormat == kAct8Dense ? 0 : kTcStages * kTcSlot);
}

// The barriers and the accumulators' `columns` of tensor memory; by the CTA.
__device__ __forceinline__ uint32_t tc_setup(TcBarriers* bars, uint32_t columns) {
  if (threadIdx.x == 0) {
    for (int s = 0; s < kTcStages; ++s) {
      mbar_init(&bars->x_full[s], kTcWarps);
      mbar_init(&bars->full[s], 1);
      mbar_init(&bars->empty[s], 1);
    }
    mbar_init(&bars->done, 1);
    mbar_init(&bars->drain, 1);
    bars->abort_flag = 0;
    fence_mbar_init();
  }
  if (threadIdx.x >> 5 == kTcWarps + 1) {
    tmem_alloc(&bars->tmem, columns);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  return bars->tmem;
}

__device__ __forceinline__ void tc_teardown(uint32_t tmem, uint32_t columns) {
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x >> 5 == kTcWarps + 1) {
    tc_fence_after();
    tmem_dealloc(tmem, columns);
  }
}

__device__ __forceinline__ bool tc_warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* status) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  bool ok = true;
  if ((threadIdx.x & 31) == 0) ok = mbar_wait(bar, parity, abort_flag, status);
  ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
  if (ok) (void)mbar_try_wait(bar, parity);
  return ok;
}

// tcgen05.wait::ld that hands the loaded registers on, so no use of them can
// be scheduled before the wait.
__device__ __forceinline__ void tc_wait_ld(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}

// Warp 16's thread: `load(stage, bar, i)` issues the copies of step i, of
// `bytes` in all, for each of the n steps.
template <typename Load>
__device__ __forceinline__ void tc_produce(uint8_t* smem, int stage_bytes, TcBarriers* bars, int n, uint32_t bytes,
                                           int* status, Load&& load) {
  int issued = 0;
  for (int i = 0; i < n; ++i) {
    const int s = i % kTcStages, u = i / kTcStages;
    if (i >= kTcStages && !mbar_wait(&bars->empty[s], (u - 1) & 1, &bars->abort_flag, status)) break;
    mbar_arrive_expect_tx(&bars->full[s], bytes);
    load(smem + s * stage_bytes, &bars->full[s], i);
    issued = i + 1;
  }
  // Every copy into shared memory has landed before the CTA can exit.
  for (int i = (issued > kTcStages ? issued - kTcStages : 0); i < issued; ++i)
    mbar_wait_teardown(&bars->full[i % kTcStages], (i / kTcStages) & 1, status);
}

// Warp 17's thread: `mma(stage, i)` issues the MMAs of step i.
template <bool kDense, typename Mma>
__device__ __forceinline__ void tc_issue(TcBarriers* bars, int n, int* status, Mma&& mma) {
  bool ok = true;
  for (int u = 0; ok && u * kTcStages < n; ++u)
#pragma unroll
    for (int s = 0; s < kTcStages; ++s) {
      const int i = u * kTcStages + s;
      if (!ok || i >= n) break;
      ok = mbar_wait(&bars->full[s], u & 1, &bars->abort_flag, status) &&
           (kDense || mbar_wait(&bars->x_full[s], u & 1, &bars->abort_flag, status));
      if (!ok) break;
      tc_fence_after();
      mma(s, i);
      tc_commit(&bars->empty[s]);
    }
  if (ok) tc_commit(&bars->done);
  tc_commit(&bars->drain);
  mbar_wait_teardown(&bars->drain, 0, status);
}

// The decoders: n tiles of kRows rows x 16 kSegs columns, the first one's
// corner at (row0, col0) and `advance` elements from one to the next, as
// [box of 64 columns][row][64 bf16] at the start of each stage.  last(row, col):
// the first tile in which the run of 16 at (row, col) does not exist; zeros
// stand there.
template <int kFormat, int kSegs, int kRows, int kStage, typename Last>
__device__ __forceinline__ bool tc_decode(const Act8View& x, int64_t row0, int64_t col0, int64_t advance, int n,
                                          uint8_t* smem, uint8_t* slots, TcBarriers* bars, int* status, Last&& last) {
  constexpr int kPassRows = kTcDecoders / kSegs;
  static_assert(kPassRows * kTcPasses == kRows && kPassRows % 8 == 0, "whole passes, one swizzle key for all of them");
  const int seg = threadIdx.x % kSegs, tok = threadIdx.x / kSegs;
  const int64_t C = x.cols, at = (row0 + tok) * C + col0 + seg * 16;
  uint8_t* const slot = slots + threadIdx.x * 16;
  int end[kTcPasses];
#pragma unroll
  for (int q = 0; q < kTcPasses; ++q) end[q] = min(n, last(tok + q * kPassRows, seg * 16));
  // Tile by tile in turn: running pointers.
  const uint8_t* code = x.codes + at;
  const uint16_t* step = x.step + at / kBlock;
  const int64_t code_pass = kPassRows * C, step_pass = code_pass / kBlock, step_advance = advance / kBlock;
  auto fetch = [&](int i, int sl) {
#pragma unroll
    for (int q = 0; q < kTcPasses; ++q)
      cp_async_16(slot + sl * kTcSlot + q * (kTcDecoders * 16), i < end[q] ? code + q * code_pass : x.codes, i < end[q]);
    cp_async_commit();
    code += advance;
  };
  auto load_steps = [&](int i, uint32_t (&s)[kTcPasses]) {
#pragma unroll
    for (int q = 0; q < kTcPasses; ++q) s[q] = i < end[q] ? __ldg(step + q * step_pass) : 0u;
    step += step_advance;
  };
  // Odd boxes take their second eight columns first, so that the boxes of a
  // store meet no bank twice.
  const int box = seg / 4, odd = box & 1, chunk = (seg & 3) * 2, key = tok & 7;
  const int out0 = box * (kRows * 128) + tok * 128 + (((chunk + odd) ^ key) << 4);
  const int out1 = box * (kRows * 128) + tok * 128 + (((chunk + 1 - odd) ^ key) << 4);
  // Tile i = kTcStages u + st, whose scales are in s; they are replaced by
  // those of tile i + kTcStages in place (a copy from a set still loading would
  // wait for it).
  auto decode = [&](int u, int st, uint32_t (&s)[kTcPasses]) {
    const int i = u * kTcStages + st;
    if (i >= n) return true;
    cp_async_wait<kTcStages - 1>();
    uint2 c[kTcPasses][2];
#pragma unroll
    for (int q = 0; q < kTcPasses; ++q) {
      const uint8_t* src = slot + st * kTcSlot + q * (kTcDecoders * 16);
      c[q][0] = *reinterpret_cast<const uint2*>(src + odd * 8);
      c[q][1] = *reinterpret_cast<const uint2*>(src + 8 - odd * 8);
    }
    if (u > 0 && !tc_warp_wait(&bars->empty[st], (u - 1) & 1, &bars->abort_flag, status)) return false;
    uint8_t* dst = smem + st * kStage;
#pragma unroll
    for (int q = 0; q < kTcPasses; ++q) {
      const uint32_t s2 = s[q] | (s[q] << 16);
#pragma unroll
      for (int e = 0; e < 2; ++e)
        *reinterpret_cast<uint4*>(dst + (e == 0 ? out0 : out1) + q * (kPassRows * 128)) =
            make_uint4(act8_decode2<kFormat, 0>(c[q][e].x, s2), act8_decode2<kFormat, 2>(c[q][e].x, s2),
                       act8_decode2<kFormat, 0>(c[q][e].y, s2), act8_decode2<kFormat, 2>(c[q][e].y, s2));
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // before the MMA reads them
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&bars->x_full[st]);
    fetch(i + kTcStages, st);  // into the slot read above
    load_steps(i + kTcStages, s);
    return true;
  };
  uint32_t scale[kTcStages][kTcPasses];
#pragma unroll
  for (int i = 0; i < kTcStages; ++i) {
    fetch(i, i);
    load_steps(i, scale[i]);
  }
  bool ok = true;
  for (int u = 0; ok && u * kTcStages < n; ++u)
#pragma unroll
    for (int st = 0; st < kTcStages; ++st) ok = ok && decode(u, st, scale[st]);
  cp_async_wait<0>();
  return ok;
}

}  // namespace

// ---------------------------------------------------------------------------
// colsum: part[z][j][k] = sum_{m in split z} V[m][j] X^[m][k], V = hi + lo + lo2
// ---------------------------------------------------------------------------
// D[columns k][j] with the token axis as K.  Both operands are MN-major, so
// rows of tokens go to shared memory as they are: A is the X^ tile, B the three
// parts of V side by side (N = 192), so that A, whose reads bound the MMA at a
// small N, is read once for all three.  Their sums stay apart in tensor memory
// until the epilogue adds them, and those of V's first part are two, of every
// other 16 tokens each: the tensor core truncates, and one chain over 1,000
// tokens cost dB 1.2e-6 of its size.  A CTA takes 256 columns (two M = 128 tiles)
// and a range of the tokens, 64 per step; it takes dY and U for dB the same
// way.  In the epilogue a lane is a column, so each j leaves as 128 contiguous
// bytes per warp.
//
// Shared memory bounds it: a step's MMAs read 80 KB, its codes and decoded tile
// take another 100 KB (about 1,500 cycles a step; 900 for plain bf16), and some
// 6 us go to the first loads and the epilogue.  14.8 us at 1999 x 8192 and rank
// 64 (16.8 MB of codes), 7.4 us for dY at 1999 x 2048, each alone on the GPU.
// Warp-level MMAs from registers, the same sums: 29.9 and 12 us.
namespace {

constexpr int kCsTok = 64;                          // tokens per step
constexpr int kCsCols = 256;                        // columns of a CTA
constexpr int kCsParts = 3;                         // bf16 parts of V
constexpr int kCsBox = kCsTok * 128;                // [64 tokens][64 columns or j] bf16
constexpr int kCsXTile = kCsCols / 64 * kCsBox;
constexpr int kCsStage = kCsXTile + kCsParts * kCsBox;
constexpr int kCsN = kCsParts * kRankPad;           // MMA N
constexpr int kCsSums = 4;                          // accumulators: hi, lo, lo2, hi
constexpr uint32_t kCsTmemCols = 2 * kCsSums * kRankPad;
constexpr int64_t kCsSteps = 24;                    // most steps of a CTA, where there is room for the splits

TcWork cs_work(int64_t M, int64_t C, bool dense) {
  TcWork w{(C + kCsCols - 1) / kCsCols, (M + kCsTok - 1) / kCsTok, dense, 0};
  // Whole waves, as many as keep a CTA at 24 steps (48 additions in a row).  8192 x
  // 8192 x 8192, rank 64: 125 us and dA off by 8.0e-7; with up to 48 steps 115 us
  // and 1.3e-6, above an fp32 product's 1.1e-6; with 16 steps the same as with 24.
  int64_t waves = (w.tiles + 147) / 148;
  while (148 * waves / w.tiles < w.steps &&
         (w.steps + 148 * waves / w.tiles - 1) / (148 * waves / w.tiles) > kCsSteps)
    ++waves;
  w.splits = static_cast<int>(std::min<int64_t>(148 * waves / w.tiles, w.steps));
  return w;
}

}  // namespace

// kDirect: a product with a single split leaves its scaled result, [r][cols], in
// `out`, without partials and a reduction.
template <int kFormat, bool kDirect>
__global__ void __launch_bounds__(kTcThreads, 1)
    act8_colsum_kernel(Act8View x, const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmHi,
                       const __grid_constant__ CUtensorMap tmLo, const __grid_constant__ CUtensorMap tmLo2, int r16,
                       int r, int splits, float scale, float* __restrict__ out, bool after, int* status) {
  constexpr bool kDense = kFormat == kAct8Dense;
  extern __shared__ uint8_t smem_raw[];
  if (!after) pdl_launch_dependents();
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  TcBarriers* bars = reinterpret_cast<TcBarriers*>(smem + kTcStages * kCsStage);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t M = x.rows, C = x.cols;
  const int64_t c0 = static_cast<int64_t>(blockIdx.x) * kCsCols;
  const int z = blockIdx.y;
  const int64_t total = (M + kCsTok - 1) / kCsTok, first = total * z / splits;
  const int n = static_cast<int>(total * (z + 1) / splits - first);  // steps, at least one
  const uint32_t tmem = tc_setup(bars, kCsTmemCols);

  if (warp == kTcWarps) {
    if (lane == 0) {
      if (after) {  // V is the previous kernel's; what overlaps this one may read it too
        pdl_wait_prior();
        pdl_launch_dependents();
      }
      tc_produce(smem, kCsStage, bars, n, kDense ? kCsStage : kCsParts * kCsBox, status,
                 [&](uint8_t* st, uint64_t* bar, int i) {
                   const int m = static_cast<int>((first + i) * kCsTok);
                   if constexpr (kDense)
                     for (int g = 0; g < kCsCols / 64; ++g)
                       tma_load_2d(st + g * kCsBox, &tmX, bar, static_cast<int>(c0) + g * 64, m);
                   tma_load_2d(st + kCsXTile, &tmHi, bar, 0, m);
                   tma_load_2d(st + kCsXTile + kCsBox, &tmLo, bar, 0, m);
                   tma_load_2d(st + kCsXTile + 2 * kCsBox, &tmLo2, bar, 0, m);
                 });
    }
  } else if (warp == kTcWarps + 1) {
    constexpr uint32_t kMn = 1u << 15;  // A MN-major, as B
    constexpr uint32_t idesc = idesc_bf16_f32(128, kCsN, true) | kMn;
    constexpr uint32_t idesc_hi = idesc_bf16_f32(128, kRankPad, true) | kMn;
    constexpr uint32_t idesc_lo = idesc_bf16_f32(128, kCsN - kRankPad, true) | kMn;
    // Groups of 64 columns (or of 64 j: one part) are a box apart, groups of
    // 8 tokens 1 KB; a K = 16 step is 16 tokens = 2 KB.
    const uint64_t base = smem_desc_mn128(smem_u32(smem), kCsBox, 1024);
    if (lane == 0)
      tc_issue<kDense>(bars, n, status, [&](int s, int i) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int kk = 0; kk < kCsTok / 16; ++kk) {
            const uint32_t d = tmem + static_cast<uint32_t>(h * kCsSums * kRankPad);
            const uint64_t a = base + static_cast<uint64_t>((s * kCsStage + h * 2 * kCsBox + kk * 2048) >> 4);
            const uint64_t b = base + static_cast<uint64_t>((s * kCsStage + kCsXTile + kk * 2048) >> 4);
            if (kk % 2 == 0) {  // hi, lo, lo2
              tc_mma_bf16_ss(d, a, b, idesc, (i > 0 || kk > 0) ? 1u : 0u);
            } else {  // lo, lo2, and the other hi
              tc_mma_bf16_ss(d + kRankPad, a, b + (kCsBox >> 4), idesc_lo, 1u);
              tc_mma_bf16_ss(d + 3 * kRankPad, a, b, idesc_hi, (i > 0 || kk > 1) ? 1u : 0u);
            }
          }
      });
  } else {
    bool ok = true;
    if constexpr (!kDense) {
      const int rows = static_cast<int>(min(M - first * kCsTok, static_cast<int64_t>(n) * kCsTok));
      const int cols = static_cast<int>(min(C - c0, static_cast<int64_t>(kCsCols)));
      ok = tc_decode<kFormat, kCsCols / 16, kCsTok, kCsStage>(
          x, first * kCsTok, c0, kCsTok * C, n, smem, smem + kTcStages * kCsStage + kTcBarriers, bars, status,
          [&](int row, int col) { return col < cols ? (rows - row + kCsTok - 1) / kCsTok : 0; });
    }
    if (ok && tc_warp_wait(&bars->done, 0, &bars->abort_flag, status)) {
      tc_fence_after();
      const int quad = warp & 3, h = (warp >> 2) & 1;  // TMEM lanes 32 quad .. + 31 of column tile h
      const uint32_t acc = tmem + (static_cast<uint32_t>(quad * 32) << 16) + static_cast<uint32_t>(h * kCsSums * kRankPad);
      const int64_t k = c0 + h * 128 + quad * 32 + lane;
      for (int j0 = warp / 8 * 16; j0 < r16; j0 += kTcWarps / 8 * 16) {
        uint32_t v[kCsSums][16];
#pragma unroll
        for (int i = 0; i < kCsSums; ++i) tmem_ld_32x32b_x16(acc + static_cast<uint32_t>(i * kRankPad + j0), v[i]);
#pragma unroll
        for (int i = 0; i < kCsSums; ++i) tc_wait_ld(v[i]);
        if (k < C) {
          float* dst = out + (static_cast<int64_t>(z) * r16 + j0) * C + k;
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float sum = (__uint_as_float(v[0][j]) + __uint_as_float(v[3][j])) +
                              (__uint_as_float(v[1][j]) + __uint_as_float(v[2][j]));
            if constexpr (!kDirect)
              dst[j * C] = sum;
            else if (j0 + j < r)
              dst[j * C] = scale * sum;
          }
        }
        __syncwarp();  // the next load is the whole warp's
      }
    }
  }
  tc_teardown(tmem, kCsTmemCols);
  pdl_wait_prior();  // an overlapped launch ends after the kernel before it
}

// dst(j, k) = scale sum_z part[z][j][k]; part has r16 = 16 ceil(r / 16) rows
// per split.  A CTA takes 32 columns of 16 j, four columns of one j per thread;
// kGroups groups of threads take every kGroups-th split each and are joined in
// order.  A narrow matrix has few CTAs and up to 148 splits: more than 8 of them
// take four groups (backward of 5000 x 256 x 256, rank 40: 35 us with one group,
// 27 with four; GPU time of 8192 x 14336 x 4096 with 9 splits for dA, rank 16: 97.9
// and 95.4, rank 64, where dB's 6 splits have most of the work: 133.0 and 136.7; of
// 1999 x 2048 x 8192, rank 64, up to 4 splits: 33.6 and 34.0).
// [cols][r] outputs leave through shared memory, 16 j side by side.  The CTAs of a
// second job follow the first's.
constexpr int kCrCols = 32;

struct ColsumReduceJob {
  const float* part;
  int64_t C;
  int splits;
  float* dst;
  int dst_rc;
};

template <int kGroups>
__global__ void __launch_bounds__(128 * kGroups)
    act8_colsum_reduce_kernel(const __grid_constant__ ColsumReduceJob job0, const __grid_constant__ ColsumReduceJob job1,
                              unsigned first, int r, float scale) {
  __shared__ float tile[kCrCols][17];
  __shared__ float4 sums[kGroups][128];
  pdl_wait_prior();
  const ColsumReduceJob& job = blockIdx.x < first ? job0 : job1;
  const float* __restrict__ part = job.part;
  float* __restrict__ dst = job.dst;
  const int64_t C = job.C;
  const int splits = job.splits, dst_rc = job.dst_rc;
  const int64_t c0 = static_cast<int64_t>(blockIdx.x < first ? blockIdx.x : blockIdx.x - first) * kCrCols;
  const int group = threadIdx.x / 128, t = threadIdx.x % 128;
  const int jj = t / (kCrCols / 4), cc = t % (kCrCols / 4) * 4, j = blockIdx.y * 16 + jj;
  const int64_t slice = static_cast<int64_t>(gridDim.y) * 16 * C;
  const bool in = j < r && c0 + cc < C;
  float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (in) {
    const float* src = part + j * C + c0 + cc;
#pragma unroll 8
    for (int z = group; z < splits; z += kGroups) {
      const float4 p = *reinterpret_cast<const float4*>(src + z * slice);
      s.x += p.x, s.y += p.y, s.z += p.z, s.w += p.w;
    }
  }
  if constexpr (kGroups > 1) {
    sums[group][t] = s;
    __syncthreads();
  }
  if (group == 0 && in) {
#pragma unroll
    for (int g = 1; g < kGroups; ++g) {
      const float4 p = sums[g][t];
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
  for (int i = threadIdx.x; i < kCrCols * 16; i += 128 * kGroups) {
    const int c = i / 16, q = i % 16;
    if (c0 + c < C && blockIdx.y * 16 + q < r) dst[(c0 + c) * r + blockIdx.y * 16 + q] = tile[c][q];
  }
}

namespace {

template <int kFormat, bool kDirect>
cudaError_t launch_colsum_format(const Act8View& x, const CUtensorMap (&maps)[4], int r, int splits, float scale,
                                 float* out, bool after, int* status, cudaStream_t stream) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  static DeviceOnce configured;
  e = configured.run(dev, [] {
    return cudaFuncSetAttribute(act8_colsum_kernel<kFormat, kDirect>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                tc_smem<kFormat>(kCsStage));
  });
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>((x.cols + kCsCols - 1) / kCsCols), static_cast<unsigned>(splits));
  return launch_dependent(act8_colsum_kernel<kFormat, kDirect>, grid, kTcThreads, tc_smem<kFormat>(kCsStage), stream, x,
                          maps[0], maps[1], maps[2], maps[3], (r + 15) / 16 * 16, r, splits, scale, out, after, status);
}

}  // namespace

bool plan_act8_colsums(ColsumJob* jobs, int count, int r, float* pool, size_t room) {
  TcWork work[2];
  size_t split[2] = {0, 0};  // bytes of one
  for (int i = 0; i < count; ++i) {
    const Act8View& x = jobs[i].x;
    work[i] = cs_work(x.rows, x.cols, x.format == kAct8Dense);
    split[i] = static_cast<size_t>((r + 15) / 16 * 16) * static_cast<size_t>(x.cols) * sizeof(float);
  }
  // A single split in the result's own order needs no partials and, alone, no
  // reduction (17 x 1024 x 4096, rank 16: 10.8 us, so 10.3).  Beside another product,
  // whose reduction runs anyway, that costs 1 us and is done only where there is no
  // room (up to 16 tokens, ranks above 48: 16 x 512 x 512, rank 64, 15.6 us; with room
  // 14.8, one product after the other 18.4).  The other order, [cols][r], never: a row
  // per lane costs the epilogue 5 us at rank 64.
  bool want_direct = count == 1;
  auto direct = [&](int i) {
    return want_direct && jobs[i].dst_rc && jobs[i].x.format != kAct8Dense && work[i].splits == 1;
  };
  auto bytes = [&](int i) { return direct(i) ? 0 : static_cast<size_t>(work[i].splits) * split[i]; };
  if (count == 2) {
    tc_share_wave(work[0], work[1]);
    // Fewer splits where they take most room, while the chains stay short.
    auto spare = [&](int i) {
      const int fewer = work[i].splits - 1;
      return fewer > 0 && (work[i].steps + fewer - 1) / fewer <= kCsSteps;
    };
    want_direct = bytes(0) + bytes(1) > room;
    while (bytes(0) + bytes(1) > room) {
      int i = bytes(1) > bytes(0) ? 1 : 0;
      if (!spare(i)) i = 1 - i;
      if (!spare(i)) return false;
      --work[i].splits;
    }
  } else {
    const int64_t most = static_cast<int64_t>(room / split[0]);
    work[0].splits = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(work[0].splits, most)));
    if (bytes(0) > room) return false;
  }
  for (int i = 0; i < count; ++i) {
    jobs[i].splits = work[i].splits;
    jobs[i].part = direct(i) ? nullptr : pool;
    pool += bytes(i) / sizeof(float);
  }
  return true;
}

cudaError_t launch_act8_colsums(const ColsumJob* jobs, int count, int r, float scale, bool overlap_first, int* status,
                                cudaStream_t stream) {
  const int rt = (r + 15) / 16;
  ColsumReduceJob reduce[2];
  unsigned blocks[2] = {0, 0};
  int reductions = 0, most = 0;
  for (int i = 0; i < count; ++i) {
    const ColsumJob& job = jobs[i];
    const Act8View& x = job.x;
    const bool dense = x.format == kAct8Dense, after = i == 0 && !overlap_first;
    const uint16_t* parts[kCsParts] = {job.hi, job.lo, job.lo2};
    CUtensorMap maps[4];  // X (plain bf16 only; else any valid map) and the parts of V
    for (int q = 0; q < kCsParts; ++q)
      if (!encode_tensor_map_2d(&maps[1 + q], parts[q], x.rows, kRankPad, kCsTok, 64)) return cudaErrorInvalidValue;
    maps[0] = maps[1];
    if (dense && !encode_tensor_map_2d(&maps[0], x.codes, x.rows, x.cols, kCsTok, 64)) return cudaErrorInvalidValue;
    const int splits = job.splits;
    const bool direct = job.part == nullptr;  // of a checkpoint
    float* const out = direct ? job.dst : job.part;
    const auto launch = dense                       ? launch_colsum_format<kAct8Dense, false>
                        : x.format == kAct8Int8     ? direct ? launch_colsum_format<kAct8Int8, true>
                                                             : launch_colsum_format<kAct8Int8, false>
                        : direct                    ? launch_colsum_format<kAct8E4m3, true>
                                                    : launch_colsum_format<kAct8E4m3, false>;
    const cudaError_t e = launch(x, maps, r, splits, scale, out, after, status, stream);
    if (e != cudaSuccess) return e;
    if (direct) continue;
    reduce[reductions] = ColsumReduceJob{job.part, x.cols, splits, job.dst, job.dst_rc ? 1 : 0};
    blocks[reductions] = static_cast<unsigned>((x.cols + kCrCols - 1) / kCrCols);
    most = std::max(most, splits);
    ++reductions;
  }
  if (reductions == 0) return cudaSuccess;
  const dim3 grid(blocks[0] + blocks[1], static_cast<unsigned>(rt));
  const bool many = most > 8;
  return launch_dependent(many ? act8_colsum_reduce_kernel<4> : act8_colsum_reduce_kernel<1>, grid, many ? 512 : 128, 0,
                          stream, reduce[0], reduce[reductions - 1], blocks[0], r, scale);
}

// ---------------------------------------------------------------------------
// rowsum: part[z][m][j] = sum_{k in split z} X^[m][k] W(j, k)
// ---------------------------------------------------------------------------
// D[tokens][j] with the columns as K: A, the X^ tile, is K-major; B is K-major
// from W [r][K] (U = X^ A^T) or MN-major from W [K][r] (V = dY B, with dY plain
// bf16).  A CTA takes 128 tokens and a range of the columns, 128 per step.  One
// MMA of N = 64 per 16 columns: what W lacks of 64 j is zero-filled by TMA.
// Bounded as colsum is: 13.2 us at 1999 x 8192 (16.8 MB of codes), 7.6 us for V
// from dY 1999 x 2048, where warp-level MMAs took 20.4 and 16.2 us.
namespace {

constexpr int kRsTok = 128;                 // tokens of a CTA
constexpr int kRsCols = 128;                // columns per step
constexpr int kRsXBox = kRsTok * 128;       // [128 tokens][64 columns]
constexpr int kRsWBox = kRankPad * 128;     // [64 j][64 columns] or [64 columns][64 j]
constexpr int kRsXTile = kRsCols / 64 * kRsXBox;
constexpr int kRsStage = kRsXTile + kRsCols / 64 * kRsWBox;
constexpr int kRsSums = 8;                  // accumulators: the tensor core truncates, so its chains are kept short
constexpr uint32_t kRsTmemCols = kRsSums * kRankPad;
constexpr int64_t kRsSteps = 64;            // most steps of a CTA, where there is room for the splits

TcWork rs_work(int64_t M, int64_t K, bool dense) {
  TcWork w{(M + kRsTok - 1) / kRsTok, (K + kRsCols - 1) / kRsCols, dense, 0};
  // One wave, or as many CTAs as keep each at 64 steps (64 additions in a row: dA
  // of 24000 tokens and 14336 outputs, rank 64, is off by 1.2e-6, in one wave with
  // 112 steps by 2.2e-6; 314 and 331 us).
  w.splits = static_cast<int>(
      std::max<int64_t>((w.steps + kRsSteps - 1) / kRsSteps, std::min<int64_t>({148 / w.tiles, w.steps, 64})));
  return w;
}

}  // namespace

template <int kFormat>
__global__ void __launch_bounds__(kTcThreads, 1)
    act8_rowsum_kernel(Act8View x, const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                       int r16, int splits, float* __restrict__ part, int* status) {
  constexpr bool kDense = kFormat == kAct8Dense;
  extern __shared__ uint8_t smem_raw[];
  pdl_launch_dependents();
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  TcBarriers* bars = reinterpret_cast<TcBarriers*>(smem + kTcStages * kRsStage);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t M = x.rows, K = x.cols;
  const int64_t m0 = static_cast<int64_t>(blockIdx.x) * kRsTok;
  const int z = blockIdx.y;
  const int64_t total = (K + kRsCols - 1) / kRsCols, first = total * z / splits;
  const int n = static_cast<int>(total * (z + 1) / splits - first);  // steps, at least one
  const uint32_t tmem = tc_setup(bars, kRsTmemCols);

  if (warp == kTcWarps) {
    if (lane == 0)
      tc_produce(smem, kRsStage, bars, n, kDense ? kRsStage : kRsStage - kRsXTile, status,
                 [&](uint8_t* st, uint64_t* bar, int i) {
                   const int k = static_cast<int>((first + i) * kRsCols), m = static_cast<int>(m0);
                   for (int g = 0; g < kRsCols / 64; ++g) {
                     if constexpr (kDense) {  // V: W [K][r]
                       tma_load_2d(st + g * kRsXBox, &tmX, bar, k + g * 64, m);
                       tma_load_2d(st + kRsXTile + g * kRsWBox, &tmW, bar, 0, k + g * 64);
                     } else {  // U: W [r][K]
                       tma_load_2d(st + kRsXTile + g * kRsWBox, &tmW, bar, k + g * 64, 0);
                     }
                   }
                 });
  } else if (warp == kTcWarps + 1) {
    constexpr uint32_t idesc = idesc_bf16_f32(128, kRankPad, kDense);
    const uint32_t st = smem_u32(smem);
    // K = 16 columns: 32 bytes along a K-major row; 16 rows = 2 KB of an MN-major box.
    const uint64_t a = smem_desc_k128(st);
    const uint64_t b = kDense ? smem_desc_mn128(st + kRsXTile, kRsWBox, 1024) : smem_desc_k128(st + kRsXTile);
    if (lane == 0)
      tc_issue<kDense>(bars, n, status, [&](int s, int i) {
#pragma unroll
        for (int kk = 0; kk < kRsCols / 16; ++kk) {
          const int box = kk / 4, sub = kk % 4;
          static_assert(kRsSums == kRsCols / 16, "an accumulator per K step");
          tc_mma_bf16_ss(tmem + static_cast<uint32_t>(kk * kRankPad),
                         a + static_cast<uint64_t>((s * kRsStage + box * kRsXBox + sub * 32) >> 4),
                         b + static_cast<uint64_t>((s * kRsStage + box * kRsWBox + sub * (kDense ? 2048 : 32)) >> 4),
                         idesc, i > 0 ? 1u : 0u);
        }
      });
  } else {
    bool ok = true;
    if constexpr (!kDense) {
      const int rows = static_cast<int>(min(M - m0, static_cast<int64_t>(kRsTok)));
      const int cols = static_cast<int>(min(K - first * kRsCols, static_cast<int64_t>(n) * kRsCols));
      ok = tc_decode<kFormat, kRsCols / 16, kRsTok, kRsStage>(
          x, m0, first * kRsCols, kRsCols, n, smem, smem + kTcStages * kRsStage + kTcBarriers, bars, status,
          [&](int row, int col) { return row < rows ? (cols - col + kRsCols - 1) / kRsCols : 0; });
    }
    const int quad = warp & 3, j0 = warp / 4 * 16;  // TMEM lanes (tokens) 32 quad .. + 31, 16 j
    if (ok && tc_warp_wait(&bars->done, 0, &bars->abort_flag, status) && j0 < r16) {
      tc_fence_after();
      float v[16];
#pragma unroll
      for (int half = 0; half < kRsSums; half += 4) {
        uint32_t w[4][16];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          tmem_ld_32x32b_x16(
              tmem + (static_cast<uint32_t>(quad * 32) << 16) + static_cast<uint32_t>((half + i) * kRankPad + j0), w[i]);
#pragma unroll
        for (int i = 0; i < 4; ++i) tc_wait_ld(w[i]);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const float s = (__uint_as_float(w[0][j]) + __uint_as_float(w[1][j])) +
                          (__uint_as_float(w[2][j]) + __uint_as_float(w[3][j]));
          v[j] = half == 0 ? s : v[j] + s;
        }
      }
      const int64_t m = m0 + quad * 32 + lane;
      if (m < M) {
        float4* dst = reinterpret_cast<float4*>(part + (static_cast<int64_t>(z) * M + m) * kRankPad + j0);
#pragma unroll
        for (int q = 0; q < 4; ++q)
          dst[q] = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
      }
    }
  }
  tc_teardown(tmem, kRsTmemCols);
  pdl_wait_prior();  // an overlapped launch ends after the kernel before it
}

namespace {

template <int kFormat>
cudaError_t launch_rowsum_format(const Act8View& x, const CUtensorMap& tx, const CUtensorMap& tw, int r16, int splits,
                                 float* part, bool overlap, int* status, cudaStream_t stream) {
  constexpr int smem = tc_smem<kFormat>(kRsStage);
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  static DeviceOnce configured;
  e = configured.run(dev, [] {
    return cudaFuncSetAttribute(act8_rowsum_kernel<kFormat>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  });
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>((x.rows + kRsTok - 1) / kRsTok), static_cast<unsigned>(splits));
  if (overlap)
    return launch_dependent(act8_rowsum_kernel<kFormat>, grid, kTcThreads, smem, stream, x, tx, tw, r16, splits, part,
                            status);
  act8_rowsum_kernel<kFormat><<<grid, kTcThreads, smem, stream>>>(x, tx, tw, r16, splits, part, status);
  return cudaGetLastError();
}

}  // namespace

bool plan_act8_rowsums(RowsumJob* jobs, int count, float* pool, size_t room) {
  const int64_t M = jobs[0].x.rows;
  const size_t split = static_cast<size_t>(M) * kRankPad * sizeof(float);
  const int64_t most = static_cast<int64_t>(room / split);
  TcWork work[2];
  for (int i = 0; i < count; ++i) work[i] = rs_work(M, jobs[i].x.cols, jobs[i].x.format == kAct8Dense);
  if (count == 2) {
    tc_share_wave(work[0], work[1]);
    if (work[0].splits + work[1].splits > most) return false;
  } else {
    work[0].splits = static_cast<int>(std::min<int64_t>(work[0].splits, most));
    if (work[0].splits < 1) return false;
  }
  for (int i = 0; i < count; ++i) {
    jobs[i].splits = work[i].splits;
    jobs[i].part = pool;
    pool += static_cast<size_t>(work[i].splits) * split / sizeof(float);
  }
  return true;
}

cudaError_t launch_act8_rowsums(const RowsumJob* jobs, int count, int r, int* status, cudaStream_t stream) {
  const int r16 = (r + 15) / 16 * 16;
  for (int i = 0; i < count; ++i) {
    const RowsumJob& job = jobs[i];
    const Act8View& x = job.x;
    const bool dense = x.format == kAct8Dense, overlap = i > 0;
    CUtensorMap tx, tw;
    if (dense ? !encode_tensor_map_2d(&tw, job.W, x.cols, r, 64, kRankPad, true, job.ldw)
              : !encode_tensor_map_2d(&tw, job.W, r, x.cols, kRankPad, 64))
      return cudaErrorInvalidValue;
    tx = tw;
    if (dense && !encode_tensor_map_2d(&tx, x.codes, x.rows, x.cols, kRsTok, 64)) return cudaErrorInvalidValue;
    const cudaError_t e =
        dense ? launch_rowsum_format<kAct8Dense>(x, tx, tw, r16, job.splits, job.part, overlap, status, stream)
        : x.format == kAct8Int8
            ? launch_rowsum_format<kAct8Int8>(x, tx, tw, r16, job.splits, job.part, overlap, status, stream)
            : launch_rowsum_format<kAct8E4m3>(x, tx, tw, r16, job.splits, job.part, overlap, status, stream);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace qnf4
