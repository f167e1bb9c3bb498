// The 8-bit activation checkpoint: its rounding rules, shared by the kernels
// that write it (act8.cu, residual_norm.cu) and read it (act8.cu).
//
// A block is 64 consecutive values of a row.  With a its absolute maximum,
//   int8:  step = bf16(a / 127), q = round(x / step) in [-127, 127]
//   E4M3:  step = bf16(a / 256), q = E4M3(x / step), saturating
// and the block stands for x^ = bf16(q step).  Both roundings are to nearest
// even.  A bf16 step (not the exact a / 127) makes the decode one bf16 product
// of two bf16 numbers, q and step, rounded once: two values per instruction
// and no fp32 detour in the kernels that feed the tensor cores from it.
#pragma once

#include "common.cuh"

namespace qnf4 {

constexpr int kAct8Int8 = QLORA_ACT8_INT8;
constexpr int kAct8E4m3 = QLORA_ACT8_E4M3;
// The step of a block that holds a NaN or an infinity: all of it decodes to NaN.
constexpr uint32_t kAct8NanStep = 0x7FC0u;

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Largest magnitude of two packed bf16 and another such maximum, as bit
// patterns (magnitudes order like unsigned integers; NaN above infinity).
__device__ __forceinline__ uint32_t absmax_bf16x2(uint32_t m, uint32_t v) { return __vmaxu2(m, v & 0x7FFF7FFFu); }

// Encoder of one block: made from the bits of its absolute maximum.
template <int kFormat>
struct Act8Encoder {
  uint32_t step;  // bf16 bits
  float pre, d, inv, limit;

  __device__ __forceinline__ explicit Act8Encoder(uint32_t amax_bits) {
    if (amax_bits >= 0x7F80u) {
      step = kAct8NanStep;
      pre = d = inv = limit = 0.0f;
      return;
    }
    const float a = bf16_bits_to_float(amax_bits);
    step = pack_bf16x2(kFormat == kAct8Int8 ? __fdiv_rn(a, 127.0f) : a * 0x1p-8f, 0.0f) & 0xFFFFu;
    // 127 steps of more than 2^121 would pass the largest bf16 value.
    if (kFormat == kAct8Int8 && step > 0x7C00u) step = 0x7C00u;
    // Steps below 2^-60 are divided by with both sides scaled up, so that
    // neither the reciprocal nor the residual leaves the normal range.
    pre = step < 0x2180u ? 0x1p64f : 1.0f;
    d = bf16_bits_to_float(step) * pre;
    inv = step != 0 ? __frcp_rn(d) : 0.0f;
    // |x / step| passes 127.5 only where the step itself was cut or is subnormal.
    limit = (step >= 0x0080u && step < 0x7C00u) ? 0.0f : 127.0f;
  }

  // x / step, rounded once.  t = n inv is within two units in the last place;
  // the residual n - t d is exact in fp32 (x and step have 8 significant
  // bits), and one correction by it gives the nearest fp32 to the quotient
  // (Markstein's refinement), exactly the quotient where that is
  // representable, so ties are seen as ties.  Other quotients of two 8-bit
  // significands are at least 2^-17 (relative) away from a rounding border.
  __device__ __forceinline__ float quotient(float x) const {
    const float n = x * pre;
    const float t = n * inv;
    return fmaf(fmaf(-t, d, n), inv, t);
  }

  // Codes of four values, value 0 in the lowest byte.
  __device__ __forceinline__ uint32_t encode4(float x0, float x1, float x2, float x3) const {
    float q[4] = {quotient(x0), quotient(x1), quotient(x2), quotient(x3)};
    if constexpr (kFormat == kAct8Int8) {
      if (limit != 0.0f) {
#pragma unroll
        for (int i = 0; i < 4; ++i) q[i] = fminf(fmaxf(q[i], -limit), limit);
      }
      uint32_t b[4];
      // 1.5 2^23 + q rounds q to an integer (ties to even) in the low mantissa bits.
#pragma unroll
      for (int i = 0; i < 4; ++i) b[i] = __float_as_uint(q[i] + 12582912.0f);
      return __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
    } else {
      uint16_t lo, hi;
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(q[1]), "f"(q[0]));
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(q[3]), "f"(q[2]));
      return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
    }
  }

  // Codes of eight packed bf16 values.
  __device__ __forceinline__ uint2 encode8(const uint4& v) const {
    if (inv == 0.0f) return make_uint2(0u, 0u);
    auto lo = [](uint32_t w) { return __uint_as_float(w << 16); };
    auto hi = [](uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); };
    return make_uint2(encode4(lo(v.x), hi(v.x), lo(v.y), hi(v.y)), encode4(lo(v.z), hi(v.z), lo(v.w), hi(v.w)));
  }
};

// Two codes, in bytes kByte and kByte + 1 of `codes`, times the packed steps
// `steps` (low half: the first code's).
template <int kFormat, int kByte>
__device__ __forceinline__ uint32_t act8_decode2(uint32_t codes, uint32_t steps) {
  if constexpr (kFormat == kAct8Int8) {
    // 0x43 above a byte is bf16: 128 + (low 7 bits) with the byte's top bit
    // clear, and that bit is the exponent's lowest (128 -> 256).  So with t the
    // byte's low seven bits kept and c the rest, t - c = (128 + low7) - (128 or
    // 256) = the two's complement value, exact.
    const uint32_t x = __byte_perm(codes, 0x43434343u, kByte == 0 ? 0x4140 : 0x4342);
    return mul_bf16x2(sub_bf16x2(x & 0xFF7FFF7Fu, x & 0xFF80FF80u), steps);
  } else {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(kByte == 0 ? codes : codes >> 16)));
    float f0, f1;  // E4M3 values are exact in fp16, and their products with a bf16 step in fp32
    asm("{\n\t.reg .f16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
        : "=f"(f0), "=f"(f1)
        : "r"(h));
    return pack_bf16x2(f0 * bf16_bits_to_float(steps & 0xFFFFu), f1 * __uint_as_float(steps & 0xFFFF0000u));
  }
}

}  // namespace qnf4
