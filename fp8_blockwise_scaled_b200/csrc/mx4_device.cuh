// 4-bit microscaled formats: code conversions and the tcgen05 forms that take
// block scales.
//
// Codes are E2M1 (+-0, 0.5, 1, 1.5, 2, 3, 4, 6), two to a byte, the element of
// the lower index in the low nibble.  A row's scales are one byte a block:
//   MXFP4  32 values, E8M0 (2^(byte - 127));
//   NVFP4  16 values, E4M3, below one fp32 scale for the tensor.
// Scales are stored in the order in which tensor memory takes them, as atoms of
// 512 bytes for 128 rows x 4 blocks: row r, block j at byte
// (r % 32) * 16 + (r / 32) * 4 + j, so that one tcgen05.cp (32 lanes x 16 bytes)
// puts an atom into four columns.
#pragma once

#include <stdint.h>

#include "device.cuh"
#include "kernels.h"
#include "qmath.cuh"

namespace fp8blk {

// Values of a block, and elements of a row that one atom covers.
template <bool kNv>
__host__ __device__ constexpr int mx4_block() { return kNv ? 16 : 32; }
template <bool kNv>
__host__ __device__ constexpr int mx4_atom_elems() { return 4 * mx4_block<kNv>(); }

// Eight values -> eight codes, x[0] in the lowest nibble (round to nearest
// even, values above 6 saturate).
__device__ __forceinline__ uint32_t cvt8_e2m1(const float (&x)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return r;
}

// Four values -> four codes, x0 in the lowest nibble.
__device__ __forceinline__ uint16_t cvt4_e2m1(float x0, float x1, float x2, float x3) {
  uint16_t r;
  asm("{\n\t.reg .b8 a, b;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "mov.b16 %0, {a, b};\n\t}"
      : "=h"(r)
      : "f"(x0), "f"(x1), "f"(x2), "f"(x3));
  return r;
}

// One value -> its E4M3 code (saturating), and an E4M3 code's value.
__device__ __forceinline__ uint32_t cvt_e4m3(float x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.0f), "f"(x));
  return r & 0xFFu;
}

__device__ __forceinline__ float e4m3_value(uint32_t code) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(code)));
  float f;
  asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %1;\n\tcvt.f32.f16 %0, l;\n\t}" : "=f"(f) : "r"(h));
  return f;
}

// An E8M0 byte's value, 2^(byte - 127) (byte 0: the subnormal 2^-127; 255: NaN).
__device__ __forceinline__ float e8m0_value(uint32_t byte) {
  return __uint_as_float(byte == 0 ? 0x00400000u : byte == 255 ? 0x7FC00000u : byte << 23);
}

// The scale byte of an NVFP4 block of maximum amax; g and rg = RN(1 / g): the tensor's
// scale.  amax / 6 and that by g are correctly rounded by Markstein's correction, as
// x / s in qmath.cuh: q0 = RN(a y) with y the correctly rounded reciprocal, then
// RN(q0 + RN(a - q0 b) y).  Below 128 whatever g holds (a scale has no sign, and the
// byte is an index into a table of 128).
__device__ __forceinline__ uint32_t nvfp4_scale(float amax, float g, float rg) {
  constexpr float kSixth = 0x1.555556p-3f;              // RN(1 / 6)
  const float a0 = amax * kSixth, a = fmaf(fmaf(-6.0f, a0, amax), kSixth, a0);
  const float t0 = a * rg, t = fmaf(fmaf(-g, t0, a), rg, t0);
  return cvt_e4m3(t) & 0x7Fu;
}

// What the values of an NVFP4 block with that scale byte are divided by.  nr: +0 for
// a divisor of zero, else negative (finish_codes), also for one that is no number.
__device__ __forceinline__ QScale nvfp4_divisor(uint32_t byte, float g) {
  QScale q;
  q.s = e4m3_value(byte) * g;
  q.nr = q.s > 0.0f ? -__frcp_rn(q.s) : (q.s == 0.0f ? 0.0f : -1.0f);
  return q;
}

// Codes of NVFP4 values: the negated quotient's signs flipped back, and zeros of no
// sign where the block's divisor is zero (there the quotient's sign follows x).  nr
// is negative but for that divisor, so its sign bit, spread over the word, is the
// mask (16384 x 8960 in both directions: 1.6% of the time; with a comparison and a
// select 5%).
template <bool kNv>
__device__ __forceinline__ uint32_t finish_codes(uint32_t codes, float nr) {
  if constexpr (!kNv) return codes;
  uint32_t keep;
  asm("prmt.b32 %0, %1, 0, 0xBBBB;" : "=r"(keep) : "r"(__float_as_uint(nr)));
  return (codes ^ 0x88888888u) & keep;
}

// Scale byte of a block of maximum amax, and what its values are divided by (NVFP4) or
// multiplied with (MXFP4: q.nr alone).
template <bool kNv>
__device__ __forceinline__ uint32_t block_scale(float amax, float g, float rg, QScale& q) {
  if constexpr (kNv) {
    const uint32_t byte = nvfp4_scale(amax, g, rg);
    q = nvfp4_divisor(byte, g);
    return byte;
  } else {
    // amax is the largest bit pattern of the block without signs, so a NaN or an
    // infinity in the block gives 253, which no finite amax does (finish_scales).
    const uint32_t byte = max(static_cast<int>(__float_as_uint(amax) >> 23) - 2, 0);
    q.s = 0.0f;
    q.nr = __uint_as_float((254u - byte) << 23);      // 1 / scale, exactly
    return byte;
  }
}

// Four scale bytes as they are stored: an MXFP4 block that holds a NaN or an infinity
// (byte 253) gets 255, the format's NaN.  Done on the staged bytes, four at a time,
// not where every thread of a block computes its scale (16384 x 8960, both
// directions: 4% more time).
template <bool kNv>
__device__ __forceinline__ uint32_t finish_scales(uint32_t bytes) {
  if constexpr (kNv) return bytes;
  return bytes | ((((bytes & 0x7F7F7F7Fu) + 0x03030303u) & bytes & 0x80808080u) >> 6);
}
template <bool kNv>
__device__ __forceinline__ uint4 finish_scales(uint4 v) {
  return make_uint4(finish_scales<kNv>(v.x), finish_scales<kNv>(v.y), finish_scales<kNv>(v.z), finish_scales<kNv>(v.w));
}

// A pair of values by their blocks' scales: -RN(x / d) (NVFP4, whose code signs
// are flipped afterwards) or x / scale (MXFP4, exact).
template <bool kNv>
__device__ __forceinline__ float2 scaled2(float2 x, float2 s, float2 nr) {
  if constexpr (kNv) return neg_quotient2(x, s, nr);
  else return __fmul2_rn(x, nr);
}

// Copies one scale atom (32 lanes x 16 bytes) from shared memory into four
// columns of tensor memory, the same in all four lane quarters.
__device__ __forceinline__ void tmem_cp_atom(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}
__device__ __forceinline__ void tmem_cp_atom_pair(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// Shared-memory descriptor of a scale atom: no swizzle, 8-row groups (16 bytes
// a row) 128 bytes apart.
__device__ __forceinline__ uint64_t smem_desc_atom(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(1) << 16;             // leading byte offset (one 16-byte column: unused)
  d |= static_cast<uint64_t>(128 >> 4) << 32;      // stride byte offset
  d |= static_cast<uint64_t>(1) << 46;             // descriptor version for sm_100
  return d;
}

// Instruction descriptor of the block-scaled 4-bit products: E2M1 A and B,
// fp32 D, both K-major, tile m x n; scales E4M3 (NVFP4) or E8M0 (MXFP4).
__host__ __device__ constexpr uint32_t idesc_mx4(int m, int n, bool nv) {
  return (1u << 7) | (1u << 10)                      // A, B format: E2M1
         | (static_cast<uint32_t>(n >> 3) << 17)     // N / 8
         | (nv ? 0u : 1u << 23)                      // scale format: E8M0 where set
         | (static_cast<uint32_t>(m >> 7) << 27);    // M / 128
}

// The bits of that descriptor that name the byte pair of a scale word which an
// instruction of 64 values with two scales (MXFP4) takes: 0 or 2.
__host__ __device__ constexpr uint32_t idesc_scale_id(uint32_t id) { return (id << 4) | (id << 29); }

// D[tmem] (+)= (A scaled by sfa) . (B scaled by sfb)^T over 64 values of K.
template <bool kNv>
__device__ __forceinline__ void umma_mx4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                         uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  if constexpr (kNv)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
            d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
            d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}

// The same across a pair of CTAs (M = 256).
template <bool kNv>
__device__ __forceinline__ void umma_mx4_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                              uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  if constexpr (kNv)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
            d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
            d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}

}  // namespace fp8blk
