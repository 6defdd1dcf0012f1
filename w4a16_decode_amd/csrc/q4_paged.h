// Device-side view of the paged INT4 KV cache, shared by the kernels that write and
// read it (layout: include/q4_attn.h).
#pragma once

#include "q4_device.h"
#include "q4_internal.h"

namespace q4 {

constexpr int kTokTile = 16;  // tokens per tile of codes (MFMA M for K, half of MFMA K for V)

// Dword of a tile (2D dwords) holding a lane's codes of 32-channel block m; lane =
// token + 16 * (channel / 8 % 4) for K, channel % 16 + 16 * (token / 4) for V.
template <int D>
__device__ __forceinline__ int tile_dword(int m, int lane) {
  constexpr int I = D / 32 < 4 ? D / 32 : 4;  // dwords a lane loads at once (8 or 16 bytes)
  return ((m / I) * kWave + lane) * I + m % I;
}

// Byte of a V dword for token t % 4: byte pairs (0, 2) and (1, 3) of a dword become
// half2 operands, so tokens 0, 1 sit in bytes 0, 2 and tokens 2, 3 in bytes 1, 3.
__device__ __forceinline__ int v_byte(int t4) { return ((t4 & 1) << 1) | (t4 >> 1); }

// Tile of a slot's page row for KV head h, in tiles from the start of the cache.
__device__ __forceinline__ int64_t slot_tile(uint32_t slot, int page_size, int heads, int h) {
  const uint32_t page = slot / (uint32_t)page_size;
  const uint32_t row = slot - page * (uint32_t)page_size;
  return ((int64_t)page * heads + h) * (page_size / kTokTile) + row / kTokTile;
}

}  // namespace q4
