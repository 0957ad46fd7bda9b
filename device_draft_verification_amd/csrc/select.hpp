// Selection of a row's first entries in the order (larger z, lower v): keys that
// hold that order in one integer, and bars that at least `keep` of a workgroup's
// entries reach.
#pragma once

#include "rows.hpp"

namespace specv {

__device__ inline uint32_t ordered32(float z) {
    const uint32_t b = __float_as_uint(z);
    return b ^ (b & 0x80000000u ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ inline float unordered32(uint32_t o) {
    return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}

// Key of a candidate; 0 marks no candidate (a finite z never has it). Both zeros
// are one logit: -0 + 0 is +0.
__device__ inline uint64_t make_key(float z, int v) {
    return static_cast<uint64_t>(ordered32(z + 0.0f)) << 32 | ~static_cast<uint32_t>(v);
}
__device__ inline float key_logit(uint64_t k) { return unordered32(static_cast<uint32_t>(k >> 32)); }
__device__ inline int key_token(uint64_t k) { return static_cast<int>(~static_cast<uint32_t>(k)); }

// The wavefront's values sorted, largest first (bitonic).
__device__ inline int wave_sort(int v) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int k = 2; k <= 64; k <<= 1)
#pragma unroll
        for (int j = k >> 1; j > 0; j >>= 1) {
            const int o = __shfl_xor(v, j, 64);
            const bool keep_max = ((lane & j) == 0) == ((lane & k) == 0);
            v = (o > v) == keep_max ? o : v;
        }
    return v;
}

// The keep-th largest of the maxima of the workgroup's runs of G lanes (T / G of
// them, at most 64), the same in every thread: a value belongs to the keep
// largest when fewer than keep others are larger, and the smallest such value is
// asked for. Every wavefront counts for itself, so one barrier does. Values are
// BITS wide. lds: T / G values.
template <int T, int G, int BITS>
__device__ inline int kth_of_groups(int v, int keep, int* lds) {
    constexpr int N = T / G;
    static_assert(N <= 64 && 64 % N == 0, "one maximum per lane");
#pragma unroll
    for (int off = 1; off < G; off <<= 1)
        v = max(v, __shfl_xor(v, off, 64));
    if (threadIdx.x % G == 0)
        lds[threadIdx.x / G] = v;
    __syncthreads();
    v = lds[threadIdx.x % N];
    if constexpr (N == 64) {
        // One maximum per lane: the bits of the keep-th largest from the top, each
        // by a ballot (counting larger ones costs two vector instructions for each
        // of the 64). Of 32 bits the lowest 12 stay 0: that lowers the bar by less
        // than 2^-11 of its value, and it lets no fewer entries through.
        constexpr unsigned kZero = 1u << (BITS - 1);
        const unsigned o = static_cast<unsigned>(v) + kZero;
        unsigned t = 0;
#pragma unroll
        for (int bit = BITS - 1; bit >= (BITS == 32 ? 12 : 0); --bit) {
            const unsigned up = t | 1u << bit;
            t = __popcll(__ballot(o >= up)) >= keep ? up : t;
        }
        return static_cast<int>(t - kZero);
    }
    int larger = 0;
#pragma unroll
    for (int j = 0; j < N; ++j)
        larger += lds[j] > v;
    v = larger < keep ? v : 0x7FFFFFFF;
#pragma unroll
    for (int off = 1; off < N; off <<= 1)
        v = min(v, __shfl_xor(v, off, 64));
    return v;
}

// The keep-th largest of the threads' own values: every wavefront sorts its 64;
// a thread's place in the whole is its place in its own list plus the entries
// before it in the others (equal values are placed by wavefront). lds: T values
// and one more.
template <int T>
__device__ inline int kth_of_threads(int v, int keep, int* lds) {
    const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
    v = wave_sort(v);
    lds[wid * 64 + lane] = v;
    __syncthreads();
    int place = lane;
#pragma unroll
    for (int w = 0; w < T / 64; ++w) {
        if (w == wid)
            continue;
        const int* list = lds + w * 64;
        int lo = 0;  // entries of the list before v
#pragma unroll
        for (int step = 64; step > 0; step >>= 1) {
            const int at = lo + step - 1;
            if (at < 64 && (w < wid ? list[at] >= v : list[at] > v))
                lo += step;
        }
        place += lo;
    }
    if (place == keep - 1)
        lds[T] = v;
    __syncthreads();
    return lds[T];
}

// A bar that at least `keep` of the workgroup's entries reach (each thread
// giving the largest of its own, `busy` threads having any), and few more: of
// evenly spread data the keep-th largest of 16 maxima lets about 1.4 keep (keep
// = 8) to 3.4 keep (16) entries through, of 64 maxima 1.4 keep (32), of the
// threads' own 1.15 keep (64 of 256). The maxima cost a few lane exchanges and
// one barrier, the threads' own a sort.
template <int T, int BITS>
__device__ inline int bar_of(int v, int keep, int busy, int* lds) {
    if (keep <= 16 && busy >= T / 16 * keep)
        return kth_of_groups<T, T / 16, BITS>(v, keep, lds);
    if (keep <= 48 && busy >= T / 64 * keep)
        return kth_of_groups<T, T / 64, BITS>(v, keep, lds);
    return kth_of_threads<T>(v, keep, lds);
}

// Names the piece's registers, so that what was unpacked from them before is
// unpacked again instead of being kept (64 registers against 32).
template <int U>
__device__ __forceinline__ void repack(uint4 (&q)[U]) {
#pragma unroll
    for (int u = 0; u < U; ++u)
        asm volatile("" : "+v"(q[u].x), "+v"(q[u].y), "+v"(q[u].z), "+v"(q[u].w));
}

}  // namespace specv
