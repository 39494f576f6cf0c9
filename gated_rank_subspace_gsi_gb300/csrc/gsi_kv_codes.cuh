// gsi_kv_codes.cuh -- 8-bit codes and tail values as fp16 operands of the
// cache's attention, and the exponential of its softmax.
#pragma once

#include "gsi_kv.cuh"

namespace gsi {

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Exponents f of V's scales lie in [-80, 122], and sums are kept relative to the
// maximum m of s + f (logit and exponent).  Where scales of one row's blocks are far
// apart, 2^f weighs more than fp32 holds although the divisor, a sum of 2^s, does not:
// - to a larger maximum, sums are brought by two factors of 2^(d / 2), and a divisor
//   takes them one by one (weighted sums may vanish, they are too small to count);
// - a scale below 2^-kScaleSpan of the largest before it in the share is taken as
//   that, so that 2^(s + f - m) is in range wherever 2^s counts.  What the block's
//   values gain is below 2^-98 of the largest value.
constexpr int kScaleSpan = 100;
__device__ __forceinline__ float ex2_half(float d) { return ex2(0.5f * d); }
// V's scale (bits of a power of two) as it is used; top: the largest so far.
__device__ __forceinline__ int clip_scale(int bits, int& top) {
  top = max(top, bits);
  return max(bits, top - (kScaleSpan << 23));
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Four codes as fp16: bytes 0, 1 in lo, bytes 2, 3 in hi.
// int8: 0x64bb is 1024 + bb in fp16, so the code plus 128 is placed in the low
// byte and 1152 taken off, exactly.
template <int FMT>
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if (FMT == kInt8) {
    const uint32_t x = w ^ 0x80808080u;
    const uint32_t l = __byte_perm(x, 0x64646464u, 0x4140), h = __byte_perm(x, 0x64646464u, 0x4342);
    const uint32_t off = 0x64806480u;
    const __half2 a = __hsub2(*reinterpret_cast<const __half2*>(&l), *reinterpret_cast<const __half2*>(&off));
    const __half2 b = __hsub2(*reinterpret_cast<const __half2*>(&h), *reinterpret_cast<const __half2*>(&off));
    lo = *reinterpret_cast<const uint32_t*>(&a);
    hi = *reinterpret_cast<const uint32_t*>(&b);
  } else {
    asm("{\n\t.reg .b16 p, q;\n\tmov.b32 {p, q}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, p;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, q;\n\t}"
        : "=r"(lo), "=r"(hi) : "r"(w));
  }
}

// Two bf16 values times inv, as fp16.
__device__ __forceinline__ uint32_t bf16_f16(uint32_t w, float inv) {
  return pack_f16(__uint_as_float(w << 16) * inv, __uint_as_float(w & 0xFFFF0000u) * inv);
}

// Warp-level MMA, 16 x 8 x 16, fp16 operands.
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

}  // namespace gsi
