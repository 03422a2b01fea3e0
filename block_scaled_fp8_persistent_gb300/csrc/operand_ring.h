// Where the stages of the products' operands lie in shared memory (grouped16.cu), as plain integers
// that the host compiles too.
//
// A stage is as large as its tile needs it: the weights' units, and of each half's rows as many as
// they fill, so that short tiles have more stages in flight (51 units: four stages of 512 rows, six of
// 256, nine of 32).  Producer and MMA thread place stages by the same rule: one behind the other, at
// the start where the end is too near.
#pragma once
#include <cstdint>

#ifdef __CUDACC__
#define BSFP8_BOTH __host__ __device__ __forceinline__
#else
#define BSFP8_BOTH inline
#endif

namespace bsfp8 {
namespace g16 {

constexpr uint32_t UNIT = 4096;      // 32 rows of 128 bytes: what a stage of the ring counts in
constexpr uint32_t RING = 51;        // units
constexpr uint32_t W_UNITS = 4;      // a CTA's 128 weight rows
constexpr uint32_t MAX_STAGES = 10;  // barriers: one more than the smallest stages that fit

// Units of a half's rows in a stage: 128, 64 or 32 rows, the box of one load (several small ones
// cost more than the rows they save: 64 groups of 160 rows 350 us with 3 of 32 rows, 313 with 128).
BSFP8_BOTH uint32_t half_units(int height) {
  return height > 128 ? 4 : height > 64 ? 2 : height > 0 ? 1 : 0;
}

struct RingPlace {
  uint32_t head = 0, slot = 0, phase = 0;
  // start of a stage of `units`; the barriers' slot and phase are those of the members
  BSFP8_BOTH uint32_t take(uint32_t units, uint32_t& skipped) {
    const bool wraps = head + units > RING;  // (also where nothing is skipped: head == RING)
    skipped = wraps ? RING - head : 0;
    const uint32_t at = wraps ? 0 : head;
    head = at + units;
    return at;
  }
  BSFP8_BOTH void next() {
    if (++slot == MAX_STAGES) { slot = 0; phase ^= 1; }
  }
};

// The producer's account of what is in the ring.  A stage counts with the units skipped before it,
// so that those are free when it is.
struct RingFill {
  static constexpr int kBits = 6;
  uint32_t oldest = 0, oldest_phase = 0;  // the barrier of the oldest stage
  uint32_t stages = 0, used = 0;          // stages, units (and skipped ones)
  uint64_t sizes = 0;                     // of the stages, the oldest's first
  BSFP8_BOTH bool fits(uint32_t units) const {
    return used + units <= RING && stages + 1 < MAX_STAGES;
  }
  BSFP8_BOTH void put(uint32_t units) {
    used += units;
    sizes |= (uint64_t)units << (kBits * stages);
    ++stages;
  }
  BSFP8_BOTH void drop_oldest() {
    if (++oldest == MAX_STAGES) { oldest = 0; oldest_phase ^= 1; }
    used -= (uint32_t)(sizes & ((1u << kBits) - 1));
    sizes >>= kBits;
    --stages;
  }
};

}  // namespace g16
}  // namespace bsfp8
