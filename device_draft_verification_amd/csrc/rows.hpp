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

// log2(e) minus its binary32 rounding: the exponent's second term keeps the
// normaliser's error at the rounding of single exponentials instead of 1.3e-8
// times the distance from the row's maximum.
constexpr float kLog2eLow = 1.92596299e-8f;

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
          // by an offset, not through an integer: the compiler then still knows it
          // for global memory (a flat load also counts as an LDS access)
          base(static_cast<const char*>(p) - (reinterpret_cast<uintptr_t>(p) & 15)),
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

    // The group that holds element v of the row (in 64 bits: their sum may pass 2^31).
    __device__ long group_of(int v) const { return (static_cast<long>(v) + shift) / W; }

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

    // U groups base + lane + u * STEP (base the same in the whole workgroup, lane
    // in [0, STEP)), those at or past `end` as -inf. Every step's load is issued
    // before any value is looked at: groups that are not wholly inside the row
    // request the nearest one that is, and are put right afterwards (skipped,
    // by a branch that the workgroup takes together, where there are none).
    // STEPWISE: whole steps among partial ones are left alone, too, so that
    // their loads stay on their way.
    template <int U, int STEP, bool STEPWISE = false>
    __device__ void load(int base, int lane, int end, uint4 (&q)[U]) const {
        if (full1 > full0) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                q[u] = request(base + lane + u * STEP);
        }
        settle<U, STEP, STEPWISE>(base, lane, end, q);
    }

    // Group g, or the nearest one that lies wholly inside the row (which has one).
    __device__ __forceinline__ uint4 request(int g) const {
        typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
        g = g < full0 ? full0 : g;
        g = g < full1 ? g : full1 - 1;
        const u32x4 v = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(base) + g);
        return make_uint4(v.x, v.y, v.z, v.w);
    }

    __device__ uint4 load_any(int g, int end) const {
        if (g >= end)
            return neg_inf();
        return inside(g) ? request(g) : load_end(g);
    }

    template <int U, int STEP, bool STEPWISE>
    __device__ void settle(int base, int lane, int end, uint4 (&q)[U]) const {
        const int stop = end < full1 ? end : full1;
        if (base >= full0 && base + U * STEP <= stop)
            return;
        // The groups at the row's ends: the first can only be this thread's
        // first, the last any one of its groups.
        const int g0 = base + lane, tail = groups - 1;
        const bool has_tail = !inside(tail) && tail >= g0 && tail < end && (tail - g0) % STEP == 0 &&
                              tail - g0 < U * STEP;
        uint4 last = neg_inf();
        if (has_tail)
            last = load_end(tail);
        if (g0 == 0 && end > 0 && tail > 0 && !inside(0))
            q[0] = load_end(0);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (STEPWISE && base + (u + 1) * STEP <= stop)
                continue;
            const int g = g0 + u * STEP;
            if (g >= end)
                q[u] = neg_inf();
            else if (has_tail && g == tail)
                q[u] = last;
        }
    }

    // The group's largest element in an integer order: for a sign-magnitude x,
    // x ^ ((x >> all but the sign) without the sign) rises with x, two bf16 to an
    // instruction. Unlike the floating maximum it needs no step that quiets
    // NaNs; a positive NaN comes out above infinity, a negative one below -inf.
    __device__ static int order_max(const uint4& q) {
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
        if constexpr (DT == kBF16) {
            typedef short s16x2 __attribute__((ext_vector_type(2)));
            s16x2 m;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const s16x2 x = __builtin_bit_cast(s16x2, w[i]);
                const uint32_t sign = __builtin_bit_cast(uint32_t, x >> 15) & 0x7FFF7FFFu;
                const s16x2 o = __builtin_bit_cast(s16x2, w[i] ^ sign);
                m = i ? __builtin_elementwise_max(m, o) : o;
            }
            return m.x > m.y ? m.x : m.y;
        } else {
            int m = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int x = static_cast<int>(w[i]);
                const int o = x ^ ((x >> 31) & 0x7FFFFFFF);
                m = i ? (o > m ? o : m) : o;
            }
            return m;
        }
    }
    static constexpr int kOrderInf = DT == kBF16 ? 0x7F80 : 0x7F800000;  // of +inf
    static constexpr int kOrderNegInf = DT == kBF16 ? -0x7F81 : static_cast<int>(0x807FFFFFu);
    __device__ static int order_of(float z) {
        const int x = static_cast<int>(__float_as_uint(z)) >> (DT == kBF16 ? 16 : 0);
        return x ^ ((x >> 31) & (DT == kBF16 ? 0x7FFF : 0x7FFFFFFF));
    }
    __device__ static float from_order(int o) {
        const int x = o ^ ((o >> 31) & (DT == kBF16 ? 0x7FFF : 0x7FFFFFFF));
        return __uint_as_float(static_cast<uint32_t>(x) << (DT == kBF16 ? 16 : 0));
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
