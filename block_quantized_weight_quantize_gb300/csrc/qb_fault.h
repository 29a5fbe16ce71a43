// qb_fault.h -- the bits of the library's device fault word (a __device__ int in
// qb_api.cu, passed to kernels by address) and how q_device_status reports them.
// Plain C++, so that a host compiler takes it as well.
#pragma once

#include "qgemv.h"

namespace qb {

// Set when a kernel gives up a bounded wait.
constexpr int kFaultMbarTimeout = 1;
// ... and when a 4-bit cache or page kernel meets an index outside its cache.
constexpr int kFaultIndex = 2;

// The bit that a call reports and clears: one a call, the first first; 0: none.
inline int fault_reported(int word) { return word & -word; }
inline int fault_status(int bit) {
    return bit == 0 ? QB_OK : bit == kFaultIndex ? QB_E_INDEX : QB_E_DEVICE;
}

}  // namespace qb
