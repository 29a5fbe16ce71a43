// qb_kv_index.h -- index arithmetic of the paged caches that has to hold at the
// ends of its ranges.  Plain C++, so that a host compiler takes it as well.
#pragma once

#include <algorithm>
#include <cstdint>

#ifdef __CUDACC__
#define QB_HD __host__ __device__ __forceinline__
#else
#define QB_HD inline
#endif

namespace qb {

#ifndef __CUDACC__
using std::max;
#endif

// Slots that a request of `count` tokens may write, its first one being entry
// `first` of `nslots`.
QB_HD int64_t kv_slots_room(int64_t count, int64_t first, int64_t nslots) {
    const int64_t left = nslots > first ? nslots - first : 0;
    return count < left ? count : left;
}

// The first key that a token at place `pos` sees (negative: a token before the
// first key) with the last `window` ones in sight, 0: all.
QB_HD int kv_first_seen(int pos, int window) {
    return window == 0 ? 0 : max(pos, window - 1) - (window - 1);
}

// Parts of `size` keys that hold `len` (0 up to 2^31 - 1).
QB_HD int kv_parts(int len, int size) { return (int)(((uint32_t)len + (uint32_t)size - 1u) / (uint32_t)size); }

}  // namespace qb
