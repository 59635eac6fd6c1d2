// hqq_tiles.h - sizes that the host and device sides of the products share.
#pragma once

namespace hqqk {

constexpr int kSms = 148;  // of a B200

// Bytes that a lane's chunk of 32 codes takes in shared memory (3 bits: the five words it may span).
__host__ __device__ constexpr int chunk_bytes(int nbits) { return nbits == 3 ? 20 : 4 * nbits; }

}  // namespace hqqk
