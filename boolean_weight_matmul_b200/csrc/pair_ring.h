// Barriers of the CTA-pair GEMM's ring of bits and scales (gemm_pair.cu), apart so
// that a host program can check them.
#pragma once

#ifdef __CUDACC__
#define MBOK_HD __host__ __device__ __forceinline__
#else
#define MBOK_HD inline
#endif

namespace mbok {

constexpr int kPairMaxSlots = 8;   // of any ring, and barriers of each kind
constexpr int kPairGroups = 4;     // groups of unpack warps: group i takes stages i, i + 4, ...

// Stage g's barrier, and the parity of its phase there.  A parity wait tells a
// phase from its neighbours only, so that whoever waits for stage g must know that
// the barrier's previous phase is complete.  A group knows this of its own stages
// (they were complete when it read them) and of no other's: copies land in any
// order.  So the barriers go by eight stages, a multiple of kPairGroups, and not by
// the ring's slots, of which there are 4 to 8: with 6, a group's wait for a stage
// passed at once if the copy six stages before, another group's, was late.
MBOK_HD int pair_bits_barrier(int g) { return int(unsigned(g) % unsigned(kPairMaxSlots)); }
MBOK_HD unsigned pair_bits_parity(int g) { return unsigned(g) / unsigned(kPairMaxSlots) & 1u; }

}  // namespace mbok
