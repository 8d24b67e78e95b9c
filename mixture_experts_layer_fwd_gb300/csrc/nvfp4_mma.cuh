// Products of a few rows with a matrix in NVFP4 on the 16 x 8 x 16 matrix
// instruction: rows of the 4-bit matrix on M, the few rows on N, codes expanded
// straight into the operand registers.
//
// The order of the reduction index is free as long as both operands share it: a
// lane holds 8 consecutive values (one word of codes) of matrix rows g and g + 8
// and the same 8 of row g of the other operand (g = lane / 4), which are two
// instructions.  Codes times E4M3 scales have at most five significant bits
// between 2^-10 and 2688: exact in fp16.  Sums are fp32.
#pragma once

#include "kv4_attention.cuh"

namespace moe {

DEVINL void mma_16x8x16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// One word of codes of matrix rows g and g + 8, times their scales.
struct Expanded {
  uint32_t a[4], b[4];
};
DEVINL Expanded expand(uint32_t codes_g, uint32_t scale_g, uint32_t codes_g8, uint32_t scale_g8) {
  Expanded e;
  kv4::e2m1x8(codes_g, e.a);
  kv4::e2m1x8(codes_g8, e.b);
#pragma unroll
  for (int i = 0; i < 4; ++i) e.a[i] = kv4::hmul2(e.a[i], scale_g), e.b[i] = kv4::hmul2(e.b[i], scale_g8);
  return e;
}
// The first (H = 0) or second of a word's two instructions.  They add to the same sums, so
// others' come in between: the second waits some 20 cycles for the first.
template <int H>
DEVINL void mma_half(float (&c)[4], const Expanded& e, const uint4& x) {
  mma_16x8x16(c, e.a[2 * H], e.b[2 * H], e.a[2 * H + 1], e.b[2 * H + 1], H ? x.z : x.x, H ? x.w : x.y);
}

// Eight bf16 values times a power of two as fp16.
DEVINL uint4 bf16x8_to_f16x8(const uint4& v, float up) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    h[i] = kv4::pack_f16x2(__uint_as_float(w[i] << 16) * up, __uint_as_float(w[i] & 0xFFFF0000u) * up);
  return make_uint4(h[0], h[1], h[2], h[3]);
}
// Largest magnitude of eight bf16 values, as bits.
DEVINL uint32_t bf16x8_top(const uint4& v) {
  const uint32_t m = 0x7FFF7FFFu;
  const uint32_t t = __vmaxu2(__vmaxu2(v.x & m, v.y & m), __vmaxu2(v.z & m, v.w & m));
  return max(t & 0xFFFFu, t >> 16);
}
// Exponent e of the power of two that brings a row of that largest magnitude to 2^15 or
// more, below 2^16 (65280 at most, which fp16 has): exact in fp16 down to 2^-29 of it, off
// by 2^-40 of it at most below.  (Rows below 2^-105: exact, times 2^120.)
DEVINL int f16_exponent(uint32_t top) { return min(15 + 127 - static_cast<int>(top >> 7), 120); }
DEVINL float power_of_two(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }  // -126 <= e <= 127

}  // namespace moe
