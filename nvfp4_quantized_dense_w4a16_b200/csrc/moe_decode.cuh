// The weight tiles of stacked experts, and their decode to bf16.
//
// A tile is 64 weight rows; its K chunks of 64 elements follow one another,
// 2304 bytes each: 64 x 16 B codes of elements 0..31, 64 x 16 B of elements
// 32..63, 64 x 4 E4M3 scales.  Two readers want them in shared memory without
// bank conflicts: a thread per row (the rows of a warp are consecutive), and
// MMA fragments (the lanes of a quad hold the same row's four 32-element parts
// of two chunks, eight rows a warp).  So the 16-byte slots are permuted by the
// part they belong to, and the scales of rows 16w + g and 16w + 8 + g stand
// side by side.
//
// Inside a 32-bit word (eight E2M1 codes) the bits are arranged so that each
// pair of elements comes out of one or two shifts and a mask, as a bf16 pair
// whose value is E2M1 * 2^-126 (sign at bit 15, magnitude at bits 8..6: two
// exponent bits and the top mantissa bit, subnormal for 0 and 0.5).  The block
// scale is applied as the bf16 number s * 2^118, so an element is exactly
// E2M1 * s * 2^-8 (at most 6 significant bits), and sums are scaled by 2^8.
// Scales have no sign, so a byte holds five exponent bits and the mantissa's
// three: E4M3's subnormal scales are normal there, and a scale becomes a bf16
// number by one shift and one addition.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

namespace ffn {
namespace moe {

constexpr int kTileRows = 64;
constexpr int kChunkK = 64;
constexpr int kChunkBytes = 2304;
constexpr float kUnscale = 256.0f;

// Offsets in a chunk (c: its index along K): codes of row r's 32-element half h,
// and its four scales.
__host__ __device__ __forceinline__ int code_offset(int r, int h, int c) {
  return 1024 * h + 16 * (r ^ (2 * h + 4 * (c & 1)));
}
__host__ __device__ __forceinline__ int scale_offset(int r, int c) {
  return 2048 + 64 * ((r >> 4) ^ (c & 1)) + 8 * (r & 7) + 4 * ((r >> 3) & 1);
}

// Pair i (elements 2i, 2i + 1) of a word c is read from
//   i = 0: c & M,  1: (c << 4) & M,  2: rotr(c, 6) & M,
//   i = 3: ((c << 6) & MA) | (rotr(c, 2) & MB)
// with M the bits {6, 7, 8, 15} of both halves, MB bit 8 of both and MA the
// rest: the source bits of the four pairs are disjoint.
constexpr uint32_t kMask = 0x81C081C0u, kMaskA = 0x80C080C0u, kMaskB = 0x01000100u;

// Where bit p of pair i's mask comes from.
__host__ __device__ constexpr int source_bit(int i, int p) {
  return i == 0 ? p : i == 1 ? p - 4 : i == 2 ? (p + 6) & 31 : (p & 15) == 8 ? (p + 2) & 31 : p - 6;
}

// Eight codes in element order (element e in bits 4e..4e+3) -> the arranged word.
__host__ __device__ __forceinline__ uint32_t arrange_codes(uint32_t codes) {
  uint32_t out = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e)
#pragma unroll
    for (int b = 0; b < 4; ++b)
      out |= ((codes >> (4 * e + b)) & 1u) << source_bit(e >> 1, (b == 3 ? 15 : 6 + b) + 16 * (e & 1));
  return out;
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  __nv_bfloat162 r = __hmul2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
  return *reinterpret_cast<uint32_t*>(&r);
}

// E4M3 byte (its sign ignored) -> scale byte: exponent + 10 above the mantissa.
__host__ __device__ __forceinline__ uint32_t scale_byte(uint32_t e4m3) {
  const uint32_t e = (e4m3 >> 3) & 15u, m = e4m3 & 7u;
  if (e) return (e + 3) << 3 | m;
  return m >= 4 ? 3u << 3 | (m & 3u) << 1 : m >= 2 ? 2u << 3 | (m & 1u) << 2 : m << 3;
}

// Scale `byte` of a word -> the bf16 number s * 2^118 in both halves; select:
// 0x4040 + 0x0101 * byte.  (A zero byte gives 2^108; its block's codes are zero.)
__device__ __forceinline__ uint32_t scale_twice(uint32_t word, uint32_t select) {
  return __byte_perm(word, 0, select) * 16u + 0x75807580u;
}

// s2 holds the block's scale twice.
__device__ __forceinline__ void decode8(uint32_t c, uint32_t s2, uint32_t (&o)[4]) {
  o[0] = mul_bf16x2(c & kMask, s2);
  o[1] = mul_bf16x2((c * 16u) & kMask, s2);
  o[2] = mul_bf16x2(__funnelshift_r(c, c, 6) & kMask, s2);
  o[3] = mul_bf16x2(((c * 64u) & kMaskA) | (__funnelshift_r(c, c, 2) & kMaskB), s2);
}

}  // namespace moe
}  // namespace ffn
