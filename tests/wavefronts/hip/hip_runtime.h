// What the kernels' sources need of the HIP runtime, on the host: a workgroup's lanes are
// fibres of one thread. Lanes of a wavefront meet at every exchange between them (ballots,
// lane moves, the first lane's value, a wavefront's barrier), and between two of these one
// runs as far as it can before the next begins. So do the wavefronts between the
// workgroup's barriers, in an order that the caller gives. What a kernel leaves unordered
// between its lanes or wavefronts comes out in one order or another. Memory accesses take
// effect at once.
#pragma once

#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>
#include <ucontext.h>

#include <algorithm>
#include <functional>
#include <type_traits>
#include <vector>

#define __device__
#define __host__
#define __global__
#define __shared__ static
#define __forceinline__ inline
#define __launch_bounds__(...)
#define __align__(n) __attribute__((aligned(n)))

struct dim3 {
    unsigned x, y, z;
    dim3(unsigned a = 1, unsigned b = 1, unsigned c = 1) : x(a), y(b), z(c) {}
};
struct uint2 { unsigned x, y; };
struct alignas(16) uint4 { unsigned x, y, z, w; };
struct alignas(16) int4 { int x, y, z, w; };
struct alignas(16) float4 { float x, y, z, w; };
struct alignas(16) ulonglong2 { unsigned long long x, y; };
inline uint4 make_uint4(unsigned x, unsigned y, unsigned z, unsigned w) { return {x, y, z, w}; }
inline uint2 make_uint2(unsigned x, unsigned y) { return {x, y}; }
inline float4 make_float4(float x, float y, float z, float w) { return {x, y, z, w}; }

typedef void* hipStream_t;
typedef void* hipEvent_t;
typedef int hipError_t;
inline hipError_t hipGetLastError() { return 0; }
inline hipError_t hipExtLaunchKernel(const void*, dim3, dim3, void**, size_t, hipStream_t, hipEvent_t, hipEvent_t, int) {
    return 0;
}

using std::max;
using std::min;

// ------------------------------------------------------------- a workgroup ---

namespace wavefronts {

struct Index { unsigned x, y, z; };

struct Group {
    static constexpr size_t kStack = 128 << 10;
    static constexpr int kMostExchanges = 1 << 18;  // of a lane: more than any run here that ends
    enum State { kRuns, kBarrier, kEnded };
    struct Lane {
        ucontext_t at;
        std::vector<char> stack;
        uint64_t given = 0;      // to an exchange
        int exchanges = 0;       // met so far
        bool barrier = false, ended = false;
    };
    std::vector<Lane> lanes;
    ucontext_t home;
    std::function<void()> body;
    int cur = -1;
    const char* fault = nullptr;

    void back() { swapcontext(&lanes[cur].at, &home); }
    void fail(const char* what) {
        if (!fault)
            fault = what;
        for (;;)
            back();
    }
};

inline Group*& group() {
    static Group* g = nullptr;
    return g;
}

}  // namespace wavefronts

inline wavefronts::Index threadIdx, blockIdx;
inline struct { unsigned x, y, z; } gridDim, blockDim;

namespace wavefronts {

inline void enter() {
    Group& g = *group();
    g.body();
    g.lanes[g.cur].ended = true;
    for (;;)
        g.back();
}

// Every lane of the wavefront gives a value; all of them are returned.
inline const std::vector<uint64_t>& exchange(uint64_t v) {
    static std::vector<uint64_t> seen[16];
    Group& g = *group();
    const int lane = g.cur, first = lane & ~63, wave = lane >> 6;
    g.lanes[lane].given = v;
    const int n = ++g.lanes[lane].exchanges;
    if (n > Group::kMostExchanges)
        g.fail("a wavefront does not come to an end");
    for (;;) {  // until all lanes have met this exchange
        bool all = true;
        for (int l = first; l < first + 64; ++l)
            all = all && g.lanes[l].exchanges >= n;
        if (all)
            break;
        g.back();
    }
    // The last one to arrive keeps what all gave, before any gives its next value.
    bool fresh = true;
    for (int l = first; l < first + 64; ++l)
        fresh = fresh && g.lanes[l].exchanges == n;
    if (fresh) {
        seen[wave].resize(64);
        for (int l = 0; l < 64; ++l)
            seen[wave][l] = g.lanes[first + l].given;
    }
    return seen[wave];
}

inline void barrier() {
    Group& g = *group();
    g.lanes[g.cur].barrier = true;
    while (g.lanes[g.cur].barrier)
        g.back();
}

// One workgroup of `threads` lanes; order[]: the wavefronts', each time they may run. Returns
// what went wrong, or null.
inline const char* run_group(int block, int threads, const int* order, const std::function<void()>& body) {
    Group g;
    group() = &g;
    g.body = body;
    g.lanes.resize(threads);
    blockIdx = {static_cast<unsigned>(block), 0, 0};
    blockDim = {static_cast<unsigned>(threads), 1, 1};
    for (auto& l : g.lanes) {
        l.stack.resize(Group::kStack);
        getcontext(&l.at);
        l.at.uc_stack.ss_sp = l.stack.data();
        l.at.uc_stack.ss_size = l.stack.size();
        l.at.uc_link = nullptr;
        makecontext(&l.at, enter, 0);
    }
    const int waves = threads / 64;
    auto state = [&](int w) {
        int at_barrier = 0, ended = 0;
        for (int l = 64 * w; l < 64 * w + 64; ++l) {
            at_barrier += g.lanes[l].barrier;
            ended += g.lanes[l].ended;
        }
        return ended == 64 ? Group::kEnded : at_barrier == 64 ? Group::kBarrier : Group::kRuns;
    };
    for (;;) {
        int at_barrier = 0, ended = 0;
        for (int i = 0; i < waves; ++i) {
            const int w = order[i];
            for (int idle = 0; state(w) == Group::kRuns; ++idle) {
                for (int l = 64 * w; l < 64 * w + 64; ++l)
                    if (!g.lanes[l].ended && !g.lanes[l].barrier) {
                        const int before = g.lanes[l].exchanges;
                        g.cur = l;
                        threadIdx = {static_cast<unsigned>(l), 0, 0};
                        swapcontext(&g.home, &g.lanes[l].at);
                        if (g.fault)
                            return g.fault;
                        if (g.lanes[l].exchanges != before || g.lanes[l].ended || g.lanes[l].barrier)
                            idle = 0;
                    }
                if (idle > 2)
                    return "lanes of a wavefront wait at different places";
            }
            at_barrier += state(w) == Group::kBarrier;
            ended += state(w) == Group::kEnded;
        }
        if (ended == waves)
            return nullptr;
        if (ended)
            return "wavefronts wait at a barrier that others do not come to";
        for (auto& l : g.lanes)
            l.barrier = false;
    }
}

}  // namespace wavefronts

// -------------------------------------------------------------- intrinsics ---

template <typename To, typename From>
inline To bits_as(From v) {
    static_assert(sizeof(To) == sizeof(From), "of one size");
    To r;
    memcpy(&r, &v, sizeof r);
    return r;
}
inline uint32_t __float_as_uint(float v) { return bits_as<uint32_t>(v); }
inline float __uint_as_float(uint32_t v) { return bits_as<float>(v); }
inline long long __double_as_longlong(double v) { return bits_as<long long>(v); }
inline double __longlong_as_double(long long v) { return bits_as<double>(v); }
inline int __popcll(unsigned long long v) { return __builtin_popcountll(v); }
inline int __ffsll(long long v) { return __builtin_ffsll(v); }
inline unsigned __umul24(unsigned a, unsigned b) { return (a & 0xFFFFFF) * (b & 0xFFFFFF); }

inline unsigned long long __ballot(int p) {
    const auto& v = wavefronts::exchange(p != 0);
    unsigned long long r = 0;
    for (int l = 0; l < 64; ++l)
        r |= static_cast<unsigned long long>(v[l]) << l;
    return r;
}
template <typename V>
inline V lane_value(V v, int from) {
    uint64_t b = 0;
    memcpy(&b, &v, sizeof v);
    const uint64_t x = wavefronts::exchange(b)[from];
    V r;
    memcpy(&r, &x, sizeof r);
    return r;
}
template <typename V>
inline V __shfl_xor(V v, int mask, int) { return lane_value(v, (threadIdx.x & 63) ^ mask); }
template <typename V>
inline V __shfl_up(V v, int n, int) {
    const int l = threadIdx.x & 63;
    return lane_value(v, l >= n ? l - n : l);
}
inline int __builtin_amdgcn_readfirstlane(int v) { return lane_value(v, 0); }
inline unsigned __builtin_amdgcn_mbcnt_lo(unsigned m, unsigned add) {
    const int l = threadIdx.x & 63;
    return add + __builtin_popcount(l >= 32 ? m : m & ((1u << l) - 1));
}
inline unsigned __builtin_amdgcn_mbcnt_hi(unsigned m, unsigned add) {
    const int l = threadIdx.x & 63;
    return add + (l < 32 ? 0 : __builtin_popcount(m & ((1u << (l - 32)) - 1)));
}
inline int __builtin_amdgcn_update_dpp(int, int v, int ctrl, int, int, bool) {
    const int l = threadIdx.x & 63;
    int from = l;
    if (ctrl < 0x100)  // quad_perm
        from = (l & ~3) | (ctrl >> (2 * (l & 3)) & 3);
    else if (ctrl == 0x140)  // row_mirror
        from = l ^ 15;
    else if (ctrl == 0x141)  // row_half_mirror
        from = l ^ 7;
    else
        wavefronts::group()->fail("a lane move that is not known here");
    return lane_value(v, from);
}
typedef uint32_t swapped __attribute__((ext_vector_type(2)));
inline swapped __builtin_amdgcn_permlane16_swap(uint32_t a, uint32_t b, bool, bool) {
    const int l = threadIdx.x & 63;
    const auto& v = wavefronts::exchange(static_cast<uint64_t>(b) << 32 | a);
    const uint64_t lo = v[l & ~16], hi = v[l | 16];
    return (l & 16) ? swapped{static_cast<uint32_t>(lo >> 32), static_cast<uint32_t>(hi >> 32)}
                    : swapped{static_cast<uint32_t>(lo), static_cast<uint32_t>(hi)};
}
inline swapped __builtin_amdgcn_permlane32_swap(uint32_t a, uint32_t b, bool, bool) {
    const int l = threadIdx.x & 63;
    const auto& v = wavefronts::exchange(static_cast<uint64_t>(b) << 32 | a);
    const uint64_t lo = v[l & ~32], hi = v[l | 32];
    return (l & 32) ? swapped{static_cast<uint32_t>(lo >> 32), static_cast<uint32_t>(hi >> 32)}
                    : swapped{static_cast<uint32_t>(lo), static_cast<uint32_t>(hi)};
}
// The instruction gives no subnormal numbers.
inline float __builtin_amdgcn_exp2f(float x) {
    const float r = exp2f(x);
    return r < 0x1p-126f ? 0.0f : r;
}
inline void __builtin_amdgcn_s_waitcnt(int) {}
#define __builtin_amdgcn_fence(...) ((void)0)
inline void __builtin_amdgcn_wave_barrier() { wavefronts::exchange(0); }
inline void __builtin_amdgcn_s_barrier() { wavefronts::barrier(); }
inline void __syncthreads() { wavefronts::barrier(); }
inline int atomicAdd(int* p, int v) {
    const int r = *p;
    *p += v;
    return r;
}
