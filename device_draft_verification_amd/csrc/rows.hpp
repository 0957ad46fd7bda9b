// A row of logits seen as 16-byte groups whatever its alignment: group g holds
// elements [g W - shift, g W - shift + W) of the row, where shift is the number
// of elements between the 16-byte boundary at or below the row's start and the
// start. Only the first and last groups can hang over the row's ends; they are
// read and written element by element, so no access leaves the row, and an odd
// vocabulary costs one slow group at each end instead of element accesses for
// the whole row.
#pragma once

#include "common.hpp"

namespace specv {

template <int DT>
struct RowGroups {
    static constexpr int W = DT == kBF16 ? 8 : 4;
    static constexpr int ESZ = DT == kBF16 ? 2 : 4;
    using elem_t = typename std::conditional<DT == kBF16, uint16_t, uint32_t>::type;

    const char* start;  // the row's first element
    const char* base;   // the 16-byte boundary at or below it
    int shift;          // elements between them
    int vocab;
    int groups;         // groups that hold an element of the row
    int full0, full1;   // groups [full0, full1) lie wholly inside the row

    __device__ RowGroups(const void* p, int v)
        : start(static_cast<const char*>(p)),
          base(reinterpret_cast<const char*>(reinterpret_cast<uintptr_t>(p) & ~uintptr_t(15))),
          shift(static_cast<int>((reinterpret_cast<uintptr_t>(p) & 15) / ESZ)),
          vocab(v) {
        // in 64 bits: shift + vocab may pass 2^31
        groups = static_cast<int>((static_cast<long>(vocab) + shift + W - 1) / W);
        full0 = shift ? 1 : 0;
        full1 = static_cast<int>((static_cast<long>(vocab) + shift) / W);
    }

    __device__ static uint4 neg_inf() {
        const unsigned w = DT == kBF16 ? 0xFF80FF80u : 0xFF800000u;
        return make_uint4(w, w, w, w);
    }

    // First element of group g (may lie outside the row at its ends).
    __device__ long element(int g) const { return static_cast<long>(g) * W - shift; }

    __device__ bool inside(int g) const { return g >= full0 && g < full1; }

    // A group at an end of the row, -inf outside the row.
    __device__ uint4 load_end(int g) const {
        uint32_t w[4];
        const long e0 = element(g);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (DT == kBF16) {
                const long a = e0 + 2 * i, b = a + 1;
                const uint32_t lo = a >= 0 && a < vocab ? reinterpret_cast<const elem_t*>(start)[a] : 0xFF80u;
                const uint32_t hi = b >= 0 && b < vocab ? reinterpret_cast<const elem_t*>(start)[b] : 0xFF80u;
                w[i] = lo | (hi << 16);
            } else {
                const long a = e0 + i;
                w[i] = a >= 0 && a < vocab ? reinterpret_cast<const elem_t*>(start)[a] : 0xFF800000u;
            }
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }

    // U groups g0 + u * STEP, those at or past `end` as -inf. The whole groups
    // are all requested before any is looked at (groups outside [full0,
    // full1) request the nearest one inside instead).
    template <int U, int STEP>
    __device__ void load(int g0, int end, uint4 (&q)[U]) const {
        typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
        if (full1 > full0) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                int g = g0 + u * STEP;
                g = g < full0 ? full0 : g;
                g = g < full1 ? g : full1 - 1;
                const u32x4 v = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(base) + g);
                q[u] = make_uint4(v.x, v.y, v.z, v.w);
            }
        }
        // The groups at the row's ends: the first can only be this thread's
        // first, the last any one of its groups.
        const int tail = groups - 1;
        const bool has_tail = !inside(tail) && tail >= g0 && tail < end && (tail - g0) % STEP == 0 &&
                              tail - g0 < U * STEP;
        uint4 last = neg_inf();
        if (has_tail)
            last = load_end(tail);
        if (g0 == 0 && end > 0 && tail > 0 && !inside(0))
            q[0] = load_end(0);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int g = g0 + u * STEP;
            if (g >= end)
                q[u] = neg_inf();
            else if (has_tail && g == tail)
                q[u] = last;
        }
    }

    __device__ static void unpack(const uint4& q, float (&z)[W]) {
        Loader<DT, true>::unpack(q, z);
    }

    // The row's element v, as fp32.
    __device__ float at(long v) const {
        const uint32_t b = reinterpret_cast<const elem_t*>(start)[v];
        return __uint_as_float(DT == kBF16 ? b << 16 : b);
    }
};

__device__ inline bool is_finite_f32(float x) { return (__float_as_uint(x) & 0x7F800000u) != 0x7F800000u; }
__device__ inline bool is_finite_f64(double x) {
    return ((static_cast<uint64_t>(__double_as_longlong(x)) >> 52) & 0x7FF) != 0x7FF;
}

}  // namespace specv
