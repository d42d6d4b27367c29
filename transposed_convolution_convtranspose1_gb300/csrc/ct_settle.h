// ct_settle.h -- what the barriers of a ring of copies are still owed when a
// kernel gives up (plain C++: tests compile it for the host).
//
// The SMs of a group (one, or a pair) each copy their piece of every operand into
// stage k % stages for use k of the ring.  The first SM's barrier of that stage
// counts all of them: its phase ends when the first SM's producer of each operand
// has arrived, which announces the pieces of all SMs, and those bytes have landed.
// Where producers stopped at different uses, the phase would never end, or it
// would say nothing of copies that are on their way.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define CT_SETTLE_FN __host__ __device__
#else
#define CT_SETTLE_FN
#endif

namespace ct {

// For one operand and use k: whether an arrival is missing, how many bytes it
// announces, and how many announced ones will never land.
struct Owed {
    bool arrive;
    uint32_t announce, absent;
};

// first, second: uses that the producers on the first and the second SM issued;
// bytes: of one SM's piece.
CT_SETTLE_FN constexpr Owed owed(uint32_t k, uint32_t first, uint32_t second, bool pair, uint32_t bytes) {
    const bool other = pair && second > k;
    return first > k ? Owed{false, 0, pair && !other ? bytes : 0} : Owed{true, other ? bytes : 0, 0};
}

// Uses from here on may be unfinished: a stage is filled again only after its use
// before has landed on all SMs.  n: the uses that the furthest producer issued.
CT_SETTLE_FN constexpr uint32_t unsettled_from(uint32_t n, uint32_t stages) { return n > stages ? n - stages : 0; }

}  // namespace ct
