// Order of the device status codes (host and device).
#pragma once

#include <cstdint>

#if defined(__CUDACC__)
#define NABLA_HD __host__ __device__ __forceinline__
#else
#define NABLA_HD inline
#endif

namespace nabla {

// Rank of a code, by which the largest of several is reported: no error, input errors (0x3xx),
// timeouts (0x1xx, ranked 0x4xx).  A wait that gave up may leave any row wrong, an input error
// concerns the rows of its sequences only, so it must not hide a timeout.
NABLA_HD uint32_t status_rank(uint32_t code) { return code >> 8 == 1u ? code + 0x300u : code; }
NABLA_HD bool is_timeout_rank(uint32_t rank) { return rank >> 8 == 4u; }
NABLA_HD uint32_t status_of_rank(uint32_t rank) { return is_timeout_rank(rank) ? rank - 0x300u : rank; }

}  // namespace nabla
