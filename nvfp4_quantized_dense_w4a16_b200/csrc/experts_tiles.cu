// Builds the weight tiles of stacked experts (moe_decode.cuh) from canonical
// NVFP4 tensors.
#include "moe.h"
#include "moe_decode.cuh"
#include "profile.h"

namespace ffn {
namespace {

using namespace moe;

// One thread per row of a tile's chunk.  A block whose scale is zero gets zero
// codes; rows and K past the weight are zero.
__global__ void __launch_bounds__(256) tile_experts_kernel(const uint8_t* __restrict__ codes,
                                                           const uint8_t* __restrict__ scales, int64_t weights,
                                                           int64_t rows, int64_t k, int tiles, int kc,
                                                           uint8_t* __restrict__ out) {
  const int64_t idx = blockIdx.x * (int64_t)blockDim.x + threadIdx.x;
  const int r = (int)(idx % kTileRows);
  const int64_t chunk = idx / kTileRows;  // [weight][tile][c]
  if (chunk >= weights * tiles * kc) return;
  const int c = (int)(chunk % kc);
  const int64_t tile = chunk / kc, weight = tile / tiles, row = (tile % tiles) * kTileRows + r;
  uint32_t w[8] = {};
  uint32_t sc = 0;
  if (row < rows) {
    const uint8_t* crow = codes + (weight * rows + row) * (k / 2) + 32 * (int64_t)c;
    const uint8_t* srow = scales + (weight * rows + row) * (k / 16) + 4 * (int64_t)c;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (64 * (int64_t)c + 32 * h < k) {  // k is a multiple of 32
        const uint4 v = *reinterpret_cast<const uint4*>(crow + 16 * h);
        w[4 * h] = v.x, w[4 * h + 1] = v.y, w[4 * h + 2] = v.z, w[4 * h + 3] = v.w;
        sc |= scale_byte(srow[2 * h]) << (16 * h) | scale_byte(srow[2 * h + 1]) << (16 * h + 8);
      }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = ((sc >> (8 * (i >> 1))) & 0xFFu) == 0 ? 0u : arrange_codes(w[i]);
  uint8_t* base = out + chunk * kChunkBytes;
  *reinterpret_cast<uint4*>(base + code_offset(r, 0, c)) = make_uint4(w[0], w[1], w[2], w[3]);
  *reinterpret_cast<uint4*>(base + code_offset(r, 1, c)) = make_uint4(w[4], w[5], w[6], w[7]);
  *reinterpret_cast<uint32_t*>(base + scale_offset(r, c)) = sc;
}

}  // namespace

int experts_tiles(int64_t rows) { return (int)((rows + kTileRows - 1) / kTileRows); }

size_t experts_tile_bytes(int64_t rows, int64_t k) {
  return (size_t)experts_tiles(rows) * ((k + kChunkK - 1) / kChunkK) * kChunkBytes;
}

cudaError_t launch_tile_experts(const void* codes, const void* scales, int64_t weights, int64_t rows, int64_t k,
                                uint8_t* out, cudaStream_t s) {
  const int tiles = experts_tiles(rows), kc = (int)((k + kChunkK - 1) / kChunkK);
  const int64_t blocks = (weights * tiles * kc * kTileRows + 255) / 256;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  ProfScope prof(s, "tile_experts");
  tile_experts_kernel<<<(unsigned)blocks, 256, 0, s>>>(static_cast<const uint8_t*>(codes),
                                                       static_cast<const uint8_t*>(scales), weights, rows, k, tiles, kc,
                                                       out);
  return cudaGetLastError();
}

}  // namespace ffn
