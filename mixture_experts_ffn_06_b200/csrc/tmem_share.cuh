// tmem_share.cuh -- shared memory that goes with TMEM columns.
//
// An SM has 512 columns, and tcgen05.alloc waits for them without a limit.  A block that
// waits there while blocks it depends on (its cluster's, or on other streams) wait for one
// another could wait for good, so blocks that hold TMEM take enough shared memory that
// those that fit on an SM together never ask for more than 512 columns: in proportion to
// their columns, at least kTmemSmemLeast each, and a block with all 512 leaves less than
// that.  (A whole SM's shared memory for 512 columns would keep the blocks without TMEM
// that run beside it out as well.)  What a block takes is its static and dynamic shared
// memory and 1 KB that the system reserves.
#pragma once
#include <cstddef>
#include <cstdint>

namespace moe {

constexpr size_t kSmSmem = 228 * 1024;         // shared memory of an SM
constexpr size_t kSmemReserved = 1024;         // of it, the system's for each block
constexpr size_t kTmemSmemLeast = 20 * 1024;   // of a block with TMEM

// Least static and dynamic shared memory of a block with so many columns.
constexpr size_t tmem_smem_least(uint32_t cols) {
  return (cols >= 512                      ? kSmSmem - kTmemSmemLeast + 16
          : kSmSmem / 512 * cols > kTmemSmemLeast ? kSmSmem / 512 * cols
                                                  : kTmemSmemLeast) -
         kSmemReserved;
}

}  // namespace moe
