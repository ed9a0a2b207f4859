// Device decode of the bf16-format weight tiles (as launch_tile_weight writes
// them with for_w4a16): one word of eight rearranged E2M1 codes -> four bf16
// pairs of element (2i, 2i + 1), each equal to E2M1 * scale * 2^-8 exactly.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

namespace ffn {
namespace moe {

constexpr int kTileRows = 128;     // weight rows of a tile
constexpr int kChunkK = 64;        // K elements of a tile's chunk
constexpr int kChunkBytes = 4608;  // 128 x 16 B low codes, 128 x 16 B high codes, 512 B scales
constexpr float kUnscale = 256.0f;

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  __nv_bfloat162 r = __hmul2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
  return *reinterpret_cast<uint32_t*>(&r);
}

// Two E4M3 scales -> the bf16 numbers s * 2^118 (low byte in the low half).
// The tiles hold them without a sign; the half-precision value is exact, and
// three bits to the right its exponent field is bf16's, re-biased.
__device__ __forceinline__ uint32_t scale_pair(uint32_t two) {
  uint32_t h;
  asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(h) : "r"(two));
  return ((h >> 3) & 0x1FFF1FFFu) + 0x73007300u;
}

// The code bits land at bf16 bits 15 (sign) and 8..6 (magnitude), which is the
// E2M1 value times 2^-126; s2 holds the block's scale twice.
__device__ __forceinline__ void decode8(uint32_t c, uint32_t s2, uint32_t (&o)[4]) {
  constexpr uint32_t kMask = 0x81C081C0u, kMaskA = 0x80C080C0u, kMaskB = 0x01000100u;
  o[0] = mul_bf16x2(c & kMask, s2);
  o[1] = mul_bf16x2((c * 16u) & kMask, s2);
  o[2] = mul_bf16x2(__funnelshift_r(c, c, 6) & kMask, s2);
  o[3] = mul_bf16x2(((c * 64u) & kMaskA) | (__funnelshift_r(c, c, 2) & kMaskB), s2);
}

}  // namespace moe
}  // namespace ffn
