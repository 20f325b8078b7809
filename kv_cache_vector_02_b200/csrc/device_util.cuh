// Small device helpers shared by the libtq kernels.
#pragma once

#include <cstdint>

#include <cuda_fp16.h>

#include "tq_internal.h"

namespace tq {

// Device invariant checks of a TQ_DEBUG build: true when cond holds; otherwise the
// check sets TQ_DEVERR_INTERNAL in the error word and returns false, and the caller
// skips the access.  In a normal build it is `true` and costs nothing.
#ifdef TQ_DEBUG
#define TQ_DCHECK(cond, err) ((cond) ? true : (atomicOr((err), TQ_DEVERR_INTERNAL), false))
#else
#define TQ_DCHECK(cond, err) true
#endif

// Code j (0 <= j < 128) of one packed row of container width w (4, 2 or 1 bits).
__device__ __forceinline__ int extract_code(const uint8_t* row, int j, int w) {
    const int bit = j * w;
    return (row[bit >> 3] >> (bit & 7)) & ((1 << w) - 1);
}

// The last b in [0, B) with key(b) <= s, of a non-decreasing key (0 if there is none).  All
// 32 lanes probe at once.
template <typename Key>
__device__ __forceinline__ int find_last(int B, int s, int lane, Key key) {
    int lo = 0, n = B;  // the answer is in [lo, lo + n)
    while (n > 1) {
        const int step = (n + 31) / 32;
        const int b = lo + lane * step;
        const bool ok = lane * step < n && (lane == 0 || key(b) <= s);
        const int last = 31 - __clz(__ballot_sync(0xffffffffu, ok));
        lo += last * step;
        n = min(step, n - last * step);
    }
    return lo;
}

// Tiles of q queries, over ragged sequences cu[0 .. B]: sequence b's tiles have the slots from
// floor(cu[b] / q) + b on.  (Its ceil(n_b / q) tiles fit before the next one's: floor((c + n) / q)
// + 1 >= floor(c / q) + ceil(n / q).)  The sequence of slot s:
__device__ __forceinline__ int find_tile_seq(const int32_t* cu, int B, int q, int s, int lane) {
    // (unsigned: an entry far out of range finds some sequence, whose own entries are then checked)
    return find_last(B, s, lane, [=](int b) { return (int)((uint32_t)(cu[b] / q) + (uint32_t)b); });
}

// The last sequence that begins at or before row i.
__device__ __forceinline__ int find_row_seq(const int32_t* cu, int B, int i, int lane) {
    return find_last(B, i, lane, [=](int b) { return cu[b]; });
}

}  // namespace tq
