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
using std::min;
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

// The keys k0..k0+31 that lie in lo..hi (none where hi < lo), a bit each; k0, lo >= 0.
QB_HD uint32_t kv_range_word(int lo, int hi, int k0) {
    const int a = max(lo - k0, 0), b = min(hi - k0, 31);
    return a > b ? 0u : (0xFFFFFFFFu >> (31 - b)) & (0xFFFFFFFFu << a);
}

// Bits at..at+31 of `words` words, zeros outside them.
QB_HD uint32_t kv_bits_at(const uint32_t *mask, int words, int at) {
    const int w = at >> 5, sh = at & 31;
    const uint32_t lo = w >= 0 && w < words ? mask[w] : 0u, hi = w + 1 >= 0 && w + 1 < words ? mask[w + 1] : 0u;
    return sh ? lo >> sh | hi << (32 - sh) : lo;
}

QB_HD int kv_popc(uint32_t x) {
#ifdef __CUDA_ARCH__
    return __popc(x);
#else
    return __builtin_popcount(x);
#endif
}

// What a token sees beside the sinks: the keys lo..hi; of the drafts that its mask marks,
// which are the keys from the sequence's context on, those at dlo and after it.
struct KvSight {
    int lo, hi, dlo;
};
constexpr int kKvNoKey = 0x7FFFFFFF;

// A token of a tree of T drafts, the last keys of a sequence: draft i is key base + i (base
// negative: the first ones have no key).  Its keys in order are those before the drafts and
// its marked drafts; with window > 0 it sees the last `window` of them.
QB_HD KvSight kv_tree_sight(const uint32_t *mask, int words, int T, int base, int window) {
    const int nb = max(base, 0);
    KvSight s = {0, nb - 1, nb};
    if (window == 0) return s;
    const int skip = nb - base;  // drafts without a key
    const int last = min(T, 32 * words) - 1;
    int n = 0;
    for (int w = 0; w < words; ++w) n += kv_popc(mask[w] & kv_range_word(skip, last, 32 * w));
    int gone = kv_first_seen(nb - 1 + n, window);  // keys of the list that are out of the window
    s.lo = min(gone, nb);
    gone -= nb;
    for (int w = 0; w < words && gone >= 0; ++w) {  // the draft that is number `gone` of the marked ones
        uint32_t m = mask[w] & kv_range_word(skip, last, 32 * w);
        const int c = kv_popc(m);
        if (gone < c) {
            for (; gone > 0; --gone) m &= m - 1;
            s.dlo = base + 32 * w + kv_popc((m & (0u - m)) - 1u);
            return s;
        }
        gone -= c;
    }
    return s;
}

// The keys k0..k0+31 that a token sees, a bit each; k0 a multiple of 32.  mask: the drafts that it
// marks, NULL without a tree; base: the key of draft 0; sinks: keys that stay visible (0 without a window).
QB_HD uint32_t kv_seen_word(const KvSight &s, int sinks, const uint32_t *mask, int words, int base, int len, int k0) {
    uint32_t w = kv_range_word(s.lo, s.hi, k0) | kv_range_word(0, min(sinks - 1, s.hi), k0);
    const int nb = max(base, 0);
    if (mask && k0 >= nb - 31) {
        const uint32_t in = kv_range_word(s.dlo, len - 1, k0) | kv_range_word(nb, min(sinks, len) - 1, k0);
        if (in) w |= kv_bits_at(mask, words, k0 - base) & in;
    }
    return w;
}

// Parts of `size` keys that an item takes: numbers hole..end - 1, of which those below `jump` stand for
// the first keys (number - hole), the others for themselves.  first: the first key that a window leaves.
struct KvParts {
    int hole, jump;
};
QB_HD KvParts kv_sink_parts(int first, int sinks, int size) {
    KvParts p;
    p.jump = first / size;
    p.hole = p.jump - min(kv_parts(sinks, size), p.jump);
    return p;
}
QB_HD int kv_part(int u, int hole, int jump) { return u < jump ? u - hole : u; }

}  // namespace qb
