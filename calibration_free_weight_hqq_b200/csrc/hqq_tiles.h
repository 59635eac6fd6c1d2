// hqq_tiles.h - sizes that the host and device sides of the products share.
#pragma once

namespace hqqk {

constexpr int kSms = 148;  // of a B200

// Bytes of a row of `codes` codes (64, 128 or 256) of a tile in shared memory. At 3 bits: the 16-byte
// pieces it may span, one more where they would be even (rows then start on different banks).
__host__ __device__ constexpr int tile_row_bytes(int nbits, int codes) {
  return nbits == 3 ? 16 * (((39 + codes - 1) / 40 + 1) | 1) : codes * nbits / 8;
}
// Bytes of a tile of 16 rows.
__host__ __device__ constexpr int tile_bytes(int nbits, int codes) {
  return 16 * tile_row_bytes(nbits, codes);
}

}  // namespace hqqk
