// The 8-bit activation checkpoint: its rounding rules, shared by the kernels
// that write it (act8.cu, residual_norm.cu) and read it (act8.cu).
//
// A block is 64 consecutive values of a row.  With a its absolute maximum,
//   int8:  step = bf16(a / 127), q = round(x / step) in [-127, 127]
//   E4M3:  step = bf16(a / 256), q = E4M3(x / step), saturating
// and the block stands for x^ = bf16(q step).  Both roundings are to nearest
// even.  A bf16 step (not the exact a / 127) makes the decode one product of two
// bf16 numbers, q and step, rounded once.  int8: a packed bf16 product, two
// values per instruction, with no fp32 detour in the kernels that feed the tensor
// cores from it.  E4M3: codes to fp16 two at a time, to fp32, the exact product
// there, and one rounding to a bf16 pair.
#pragma once

#include "common.cuh"
#include "f32x2.cuh"

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
  float d, inv;   // divisor and its approximate reciprocal
  float pre;      // factor of the values before the division
  bool plain;     // pre = 1, and no quotient leaves the int8 range

  __device__ __forceinline__ explicit Act8Encoder(uint32_t amax_bits) {
    const float a = bf16_bits_to_float(amax_bits);
    // a times fp32(1 / 127) rounds to the same bf16 as a / 127 for every bf16 a.
    step = pack_bf16x2(a * (kFormat == kAct8Int8 ? 1.0f / 127.0f : 0x1p-8f), 0.0f) & 0xFFFFu;
    // 127 steps of more than 2^121 would pass the largest bf16 value.
    if (kFormat == kAct8Int8 && step > 0x7C00u) step = 0x7C00u;
    if (amax_bits >= 0x7F80u) step = kAct8NanStep;
    // Steps below 2^-90 are divided by with both sides scaled up, so that
    // neither the reciprocal nor the residual leaves the normal range.
    plain = step >= 0x1280u && step < 0x7C00u;
    pre = plain ? 1.0f : step < 0x1280u ? 0x1p64f : 1.0f;
    d = bf16_bits_to_float(step) * pre;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(d));
  }

  // x / step for two values, each rounded once.  t = n inv is within a few
  // units in the last place; the residual n - t d is exact in fp32 (x and step
  // have 8 significant bits), and one correction by it gives the nearest fp32
  // to the quotient (Markstein's refinement), exactly the quotient where that
  // is representable, so ties are seen as ties.  Other quotients of two 8-bit
  // significands are at least 2^-17 (relative) away from a rounding border.
  __device__ __forceinline__ F2 quotient(F2 n) const {
    const F2 t = mul2(n, splat2(inv));
    return fma2(fma2(t, splat2(-d), n), splat2(inv), t);
  }

  // Codes of four values (two packed bf16 words), value 0 in the lowest byte.
  template <bool kPlain>
  __device__ __forceinline__ uint32_t encode4(uint32_t w0, uint32_t w1) const {
    F2 a{__uint_as_float(w0 << 16), __uint_as_float(w0 & 0xFFFF0000u)};
    F2 b{__uint_as_float(w1 << 16), __uint_as_float(w1 & 0xFFFF0000u)};
    if constexpr (!kPlain) a = mul2(a, splat2(pre)), b = mul2(b, splat2(pre));
    a = quotient(a), b = quotient(b);
    if constexpr (kFormat == kAct8Int8) {
      if constexpr (!kPlain) {
        a = F2{fminf(fmaxf(a.x, -127.0f), 127.0f), fminf(fmaxf(a.y, -127.0f), 127.0f)};
        b = F2{fminf(fmaxf(b.x, -127.0f), 127.0f), fminf(fmaxf(b.y, -127.0f), 127.0f)};
      }
      // 1.5 2^23 + q rounds q to an integer (ties to even) in the low mantissa bits.
      a = add2(a, splat2(12582912.0f)), b = add2(b, splat2(12582912.0f));
      return __byte_perm(__byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040),
                         __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040), 0x5410);
    } else {
      uint16_t lo, hi;
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(a.y), "f"(a.x));
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(b.y), "f"(b.x));
      return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
    }
  }

  // Codes of eight packed bf16 values.
  __device__ __forceinline__ uint2 encode8(const uint4& v) const {
    if (plain) return make_uint2(encode4<true>(v.x, v.y), encode4<true>(v.z, v.w));
    if (step == 0 || step == kAct8NanStep) return make_uint2(0u, 0u);
    return make_uint2(encode4<false>(v.x, v.y), encode4<false>(v.z, v.w));
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
