// What the kernels over the paged 8-bit cache share: its sizes, the batch of
// sequences, and how a wave finds its sequence.  Internal header: HIP device
// code only.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mnb_internal.h"

namespace mnb {

// The batch as the device reads it.  Its numbers come from device memory and
// are not trusted: every use below is clamped to the buffers.
struct CacheBatch {
    const int32_t* starts;    // [S + 1]
    const int32_t* lengths;   // [S]
    const int32_t* table;     // [S][max_pages]
    int32_t S, T;
    int32_t max_pages, page_bits;   // pages of 1 << page_bits tokens
    int32_t pages;
};

// One sequence: its rows t0 .. t0 + n - 1 of the packed tokens and its length
// with them; token i stands at position length - n + i.
struct Sequence {
    int32_t t0, n, length;
};

__device__ __forceinline__ int32_t clamp32(int32_t v, int32_t lo, int32_t hi)
{
    return v < lo ? lo : v > hi ? hi : v;
}

// A value that every lane of the wave holds alike, in scalar registers.
__device__ __forceinline__ int32_t uniform(int32_t v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int64_t uniform64(int64_t v)
{
    return (int64_t)((uint64_t)(uint32_t)uniform((int32_t)(v >> 32)) << 32 | (uint32_t)uniform((int32_t)v));
}

// A length beyond the page table's width keeps its value (positions count from
// it); what reads the table checks the width.
__device__ __forceinline__ Sequence sequence(const CacheBatch& b, int32_t s)
{
    Sequence q;
    q.t0 = clamp32(b.starts[s], 0, b.T);
    q.n = clamp32(b.starts[s + 1], q.t0, b.T) - q.t0;
    q.length = b.lengths[s] < 0 ? 0 : b.lengths[s];
    return q;
}

__device__ __forceinline__ Sequence uniform_sequence(const CacheBatch& b, int32_t s)
{
    const Sequence q = sequence(b, s);
    return Sequence{uniform(q.t0), uniform(q.n), uniform(q.length)};
}

// The largest s < count with f(s) <= v for a rising f with f(0) <= v, sixty-four
// candidates at a time (every lane gets the answer).  f is called with 0 <= s <
// count only, so any f gives some s in range.
template <class F>
__device__ __forceinline__ int32_t wave_search(int32_t count, int64_t v, F f)
{
    const int32_t lane = threadIdx.x & 63;
    int32_t lo = 0, n = count;
    while (n > 1) {
        const int32_t step = (n + 63) >> 6;
        const int32_t at = lo + lane * step;
        const bool below = lane * step < n && f(at) <= v;
        const uint64_t m = __builtin_amdgcn_ballot_w64(below);
        // Candidates below v come first; the last of them starts the range.
        const int32_t k = m ? 63 - __builtin_clzll(m) : 0;
        const int32_t left = n - k * step;
        lo += k * step;
        n = left < step ? left : step;
    }
    return __builtin_amdgcn_readfirstlane(lo);
}

// Sum over the lanes up to this one.
__device__ __forceinline__ int32_t wave_prefix32(int32_t v)
{
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);   // row_shr:1
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);   // row_shr:2
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);   // row_shr:4
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);   // row_shr:8
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);   // row_bcast:15 into rows 1 and 3
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);   // row_bcast:31 into rows 2 and 3
    return v;
}

// The sequences of a batch, lane s holding the s-th where there are up to 64 of
// them (read once, together).
struct Sequences {
    const CacheBatch& b;
    Sequence mine;
    __device__ __forceinline__ explicit Sequences(const CacheBatch& batch) : b(batch), mine{0, 0, 0}
    {
        const int32_t lane = threadIdx.x & 63;
        if (b.S <= 64) mine = sequence(b, lane < b.S ? lane : b.S - 1);
    }
    __device__ __forceinline__ Sequence at(int32_t s) const      // s alike in every lane
    {
        if (b.S > 64) return uniform_sequence(b, s);
        return Sequence{__builtin_amdgcn_readlane(mine.t0, s), __builtin_amdgcn_readlane(mine.n, s),
                        __builtin_amdgcn_readlane(mine.length, s)};
    }
};

// Sequence s = the largest with f(its first row, s) <= v, for a rising f.  Up to 64
// sequences are read at once, lane s the s-th.
struct Found {
    int32_t s;
    Sequence q;
};
template <class F>
__device__ __forceinline__ Found find_sequence(const CacheBatch& b, int64_t v, F f)
{
    if (b.S > 64) {
        const int32_t s = wave_search(b.S, v, [&](int32_t i) { return f(clamp32(b.starts[i], 0, b.T), i); });
        return Found{s, uniform_sequence(b, s)};
    }
    const Sequences all(b);
    const int32_t lane = threadIdx.x & 63;
    const uint64_t m = __builtin_amdgcn_ballot_w64(lane < b.S && f(all.mine.t0, lane) <= v);
    const int32_t s = m ? 63 - __builtin_clzll(m) : 0;
    return Found{s, all.at(s)};
}

}  // namespace mnb
