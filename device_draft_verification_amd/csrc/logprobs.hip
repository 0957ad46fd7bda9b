// Scores of given tokens and their gradient (spec_logprobs.h).
//
//   x = z / T, M = max x, S = sum exp(x - M), H = log S - sum exp(x - M) (x - M) / S;
//   logprob = (x_t - M) - log S, rank = entries before t, the K first entries;
//   grad_v = (a ([v = t] - p_v) - b p_v (log p_v + H)) / T.
//
// Forward: a workgroup goes along a row, or a part of one where there are few
// rows, in steps that stay in registers while the step behind is on its way. A
// thread keeps the largest entry it has seen, and sums of exp(x - M) and of
// exp(x - M) (x - M) against that; the workgroup keeps the K first entries (see
// Selection). Parts of rows are joined by a second kernel. Backward: every
// element for itself, from the normaliser and the entropy.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <new>
#include <type_traits>

#include "lanes.hpp"
#include "launch.hpp"
#include "rows.hpp"
#include "select.hpp"
#include "spec_logprobs.h"
#include "stage.hpp"

namespace specv {
namespace {

constexpr int kT = kBlock;  // threads of a workgroup
constexpr int kU = 4;       // 16-byte groups of a step per thread

// What a part of a row leaves: M (-inf: no entry), S and T = sum e (x - M) log2e, the
// entries before the token.
struct Part {
    float m;
    int before;
    double s, t;
};

struct LogprobsArgs {
    const void* logits;
    const int32_t* token;
    const float* temperature;  // NULL: 1
    float* out_logprob;
    int32_t* out_rank;
    float* out_entropy;
    int32_t* out_top_token;
    float* out_top_logprob;
    float* out_norm;
    int vocab, keep;
};

// ---------------------------------------------------------------- selection ---

// The wavefront's lanes below this one that are in the mask.
__device__ __forceinline__ int lanes_below(uint64_t mask) {
    return static_cast<int>(__builtin_amdgcn_mbcnt_hi(
        static_cast<uint32_t>(mask >> 32), __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(mask), 0)));
}

// The upper half of a key, which rises with the logit, as the logit; its last bits
// may be missing (the result is then lower, or the lowest number).
__device__ inline float logit_at_least(uint32_t upper) {
    return upper < ordered32(kNegMax) ? kNegMax : unordered32(upper);
}

// The k-th largest of 64 N numbers, N in each lane (of the first n chunks), the same
// in every lane, with the bits below LOW zero, or `least` if that is larger: its
// bits from the first in which the largest differs from `least`, two by three
// ballots a chunk.
template <int N, int LOW>
__device__ inline uint32_t kth_largest(const uint32_t (&v)[N], int n, int k, uint32_t least) {
    static_assert(LOW % 2 == 0, "bits go in pairs");
    uint32_t most = v[0];
#pragma unroll
    for (int i = 1; i < N; ++i)
        most = max(most, v[i]);
    most = __builtin_amdgcn_readfirstlane(over_lanes(most, [](uint32_t a, uint32_t b) { return max(a, b); }));
    if (most <= least)
        return least;
    int bit = (31 - __builtin_clz(most ^ least)) & ~1;
    uint32_t t = most & ~(static_cast<uint32_t>((4ull << bit) - 1));
#pragma unroll 1
    for (; bit >= LOW; bit -= 2) {
        const uint32_t one = t | 1u << bit, two = t | 2u << bit, three = t | 3u << bit;
        int reach1 = 0, reach2 = 0, reach3 = 0;
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < n) {
                reach1 += __popcll(__ballot(v[i] >= one));
                reach2 += __popcll(__ballot(v[i] >= two));
                reach3 += __popcll(__ballot(v[i] >= three));
            }
        t = reach3 >= k ? three : reach2 >= k ? two : reach1 >= k ? one : t;
    }
    return max(t, least);
}

// A row's first entries, gathered over segments of it. While a segment goes by,
// each wavefront puts the 16-byte groups aside whose largest entry reaches a bar (few
// do, and single entries would cost all lanes the way through them); at its end
// their entries that reach the bar become keys in a list of the workgroup's, and the
// list's keep-th largest is the next segment's bar. What is kept does not depend on
// the order in which keys arrive.
constexpr int kCap = 512;  // keys

// Wavefronts meet at barriers only: what one reads here behind a barrier is written
// again behind another one. counts and lost, which a segment's end reads and the next
// segment's writes, have that barrier where close() ends (1 to 5 a row).
template <int T>
struct SelectionLds {
    alignas(16) uint64_t lists[2][kCap];
    uint64_t bar;      // of rank(), read by close() behind a barrier and by nobody else
    int counts[2];     // keys put into the lists, also those that one had no place for
    int lost;          // groups that a wavefront had no place for
    uint32_t bars[T / 64];  // the wavefronts' first ones, written once
};

template <int T, int G>
struct GroupLds {
    uint4 data[T / 64][G];
    int at[T / 64][G];
};

// LOW: bits of a key's upper half that need not be looked at.
template <int T, int LOW>
struct Selection {
    SelectionLds<T>& lds;
    const int keep;
    int cur = 0;       // the list in use
    int held = 0;      // keys that earlier segments left in it
    uint64_t bar = 1;  // keys below it are not among the first; 0 marks no key

    __device__ Selection(SelectionLds<T>& l, int k) : lds(l), keep(k) {
        if (threadIdx.x == 0)
            lds.counts[0] = lds.counts[1] = lds.lost = 0;
        lds_barrier();
    }

    // Each lane's keys, where it has them, into list `to`; the whole wavefront calls it.
    template <int N>
    __device__ void put(const bool (&has)[N], const uint64_t (&key)[N], int to) {
        uint64_t mask[N];
        int n = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            mask[i] = __ballot(has[i]);
            n += __popcll(mask[i]);
        }
        if (n == 0)
            return;
        int base = 0;
        if ((threadIdx.x & 63) == 0)
            base = atomicAdd(&lds.counts[to], n);
        base = __builtin_amdgcn_readfirstlane(base);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int slot = base + lanes_below(mask[i]);
            if (has[i] && slot < kCap)
                lds.lists[to][slot] = key[i];
            base += __popcll(mask[i]);
        }
    }

    // A first bar: each of the first `waves` wavefronts, whose threads all have entries,
    // has its share of keep threads whose largest one reaches it.
    __device__ void begin(float most, int waves) {
        waves = min(waves, T / 64);
        if (waves == 0)
            return;
        const uint32_t v[1] = {ordered32(most + 0.0f)};
        const uint32_t least = over_lanes(v[0], [](uint32_t a, uint32_t b) { return min(a, b); });
        const uint32_t mine = kth_largest<1, LOW>(v, 1, (keep + waves - 1) / waves,
                                                  __builtin_amdgcn_readfirstlane(least));
        lds.bars[threadIdx.x >> 6] = static_cast<int>(threadIdx.x >> 6) < waves ? mine : ~0u;
        lds_barrier();
        uint32_t b = lds.bars[0];
#pragma unroll
        for (int w = 1; w < T / 64; ++w)
            b = min(b, lds.bars[w]);
        raise(static_cast<uint64_t>(static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(b))) << 32);
    }

    __device__ void raise(uint64_t to) { bar = to > bar ? to : bar; }

    // After a segment, every thread of the workgroup: f() puts the wavefront's keys
    // that are at least the bar into list `cur`. False: groups were lost, and nothing
    // has changed.
    template <typename F>
    __device__ bool close(bool last, F&& f) {
        int n;
        for (;;) {
            f();
            lds_barrier();
            n = lds.counts[cur];
            const bool lost = lds.lost != 0;
            if (n <= kCap && !lost)
                break;
            // Of the keys that did fit, more than keep are the segment's, and keys are
            // unique: the keep-th largest is a higher bar. Mostly its upper half is.
            const uint64_t before = bar;
            if (!lost) {
                constexpr int N = kCap / 64;
                uint32_t v[N];
#pragma unroll
                for (int i = 0; i < N; ++i)
                    v[i] = static_cast<uint32_t>(lds.lists[cur][64 * i + (threadIdx.x & 63)] >> 32);
                raise(static_cast<uint64_t>(kth_largest<N, LOW>(v, N, keep, static_cast<uint32_t>(bar >> 32))) << 32);
                if (bar == before)
                    rank(kCap);
            }
            lds_barrier();
            if (!lost && bar == before)
                bar = lds.bar;
            if (threadIdx.x == 0) {
                lds.counts[cur] = held;
                lds.lost = 0;
            }
            lds_barrier();
            if (lost)
                return false;
        }
        held = n;
        // Before the last ranking more keys are cheaper than a narrower list.
        if (n > (last ? 3 * keep : keep + 16))
            narrow();
        if (last)  // what follows begins with sort(), which writes the other list
            return true;
        if (held > keep + 64)  // that many are equal
            sort();
        lds_barrier();  // all have read counts and lost, which the next segment writes
        return true;
    }

    // The list's keys that are at least its keep-th largest, into the other list.
    __device__ void narrow() {
        constexpr int N = kCap / 64;
        const int lane = threadIdx.x & 63, chunks = (held + 63) / 64;
        uint64_t key[N];
        uint32_t v[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            key[i] = i < chunks && 64 * i + lane < held ? lds.lists[cur][64 * i + lane] : 0;
            v[i] = static_cast<uint32_t>(key[i] >> 32);
        }
        raise(static_cast<uint64_t>(kth_largest<N, LOW>(v, chunks, keep, static_cast<uint32_t>(bar >> 32))) << 32);
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < chunks && i % (T / 64) == static_cast<int>(threadIdx.x >> 6)) {
                const bool has[1] = {key[i] >= bar};
                const uint64_t one[1] = {key[i]};
                put(has, one, cur ^ 1);
            }
        swap();
    }

    // The list becomes its keep largest keys, largest first.
    __device__ void sort() {
        rank(held);
        if (threadIdx.x == 0)
            lds.counts[cur ^ 1] = min(held, keep);
        swap();
        if (held >= keep)
            bar = lds.lists[cur][keep - 1];
    }

    __device__ void swap() {
        lds_barrier();
        cur ^= 1;
        held = lds.counts[cur];
        if (threadIdx.x == 0)
            lds.counts[cur ^ 1] = 0;  // seen by all behind the next barrier, before its next use
    }

    // The keep largest of the list's first n keys, largest first, into the other list:
    // four lanes to a key, each compares it with a quarter of the list.
    __device__ void rank(int n) const {
        const uint64_t* list = lds.lists[cur];
        const int quarter = static_cast<int>(threadIdx.x) & 3;
#pragma unroll 1
        for (int i = static_cast<int>(threadIdx.x) >> 2; (i & ~15) < n; i += T / 4) {
            const uint64_t mine = i < n ? list[i] : ~0ull;
            int larger = 0;
#pragma unroll 4
            for (int j = 0; j < n; j += 8) {  // what lies behind the n keys does not count
                const int at = j + 2 * quarter;
                const ulonglong2 two = *reinterpret_cast<const ulonglong2*>(list + at);
                larger += two.x > mine && at < n;
                larger += two.y > mine && at + 1 < n;
            }
            larger += lane_move<0xB1>(larger);
            larger += lane_move<0x4E>(larger);
            if (quarter == 0 && i < n && larger < keep) {
                lds.lists[cur ^ 1][larger] = mine;
                if (larger == keep - 1)
                    lds.bar = mine;
            }
        }
    }
};

// ------------------------------------------------------------------- a row ---

// A row's scale: fl32(1/T), NaN of a temperature that makes the whole row NaN.
__device__ inline float row_scale(const float* temperature, long row) {
    if (!temperature)
        return 1.0f;
    float inv_t;
    return temperature_mode(temperature[row], &inv_t) == 1 ? inv_t : __builtin_nanf("");
}

// The largest of three; unlike fmaxf it takes no instructions that quiet NaNs (a
// NaN is lost, or wins: the sums have it).
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
    return r;
}

// The larger of two, a NaN if either is.
__device__ __forceinline__ float maximum(float a, float b) {
    float r;
    asm("v_maximum3_f32 %0, %1, %2, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
}

// A value that is the same in the whole wavefront, known to be so.
__device__ __forceinline__ float uniform(float v) {
    return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(v)));
}

template <int W>
__device__ __forceinline__ float largest(const float (&z)[W]) {
    if constexpr (W == 8)
        return max3(max3(z[0], z[1], z[2]), max3(z[3], z[4], z[5]), max3(z[6], z[7], z[7]));
    else
        return max3(max3(z[0], z[1], z[2]), z[3], z[3]);
}

// Sums of e = 2^y and of e y over some entries, y their distance from a reference in
// units of ln 2. Near the origin (see kReach) the reference is a value of x log2e,
// rounded to binary32, and y one multiply-add; a far one is a value of x itself,
// since beside it x log2e has no digits left for the distances.
struct Sums {
    float ref;
    bool far;
    double s, t;
};

// How far reference `from` lies above `to`, in the same units.
__device__ inline double reference_step(float from, bool from_far, float to, bool to_far) {
    const double a = static_cast<double>(from), b = static_cast<double>(to), c = static_cast<double>(kLog2e);
    if (from_far && to_far)
        return (a - b) * c;
    return (from_far ? a * c : a) - (to_far ? b * c : b);
}

__device__ inline void move_reference(Sums& x, float to, bool to_far) {
    const double d = reference_step(x.ref, x.far, to, to_far);
    x.ref = to;
    x.far = to_far;
    if (d == 0.0 || x.s == 0.0)
        return;
    const double f = static_cast<double>(fast_exp2(static_cast<float>(d)));
    x.t = f == 0.0 ? x.s * f : f * (x.t + x.s * d);  // a NaN stays one
    x.s *= f;
}

// Beyond it binary32 rounds x log2e by more than 2^-3.
constexpr float kReach = 1048576.0f;

// A group's sums are taken against the wavefront's reference so far as long as they
// stay below this; beyond, the reference becomes its largest entry so far.
constexpr float kLazy = 256.0f;

// Joins the threads' parts and single entries edge_x (-inf: none), against the
// largest entry m: in every thread afterwards.
template <int T>
struct JoinLds {
    float m[T / 64];
    int before[T / 64];
    double s[T / 64], t[T / 64];
};

template <int T>
__device__ inline Part join_threads(float m, int before, Sums x, float edge_x, JoinLds<T>& lds) {
    const int wid = threadIdx.x >> 6;
    m = over_lanes(m, [](float a, float b) { return fmaxf(a, b); });
    if ((threadIdx.x & 63) == 0)
        lds.m[wid] = m;
    lds_barrier();
#pragma unroll
    for (int w = 0; w < T / 64; ++w)
        m = fmaxf(m, lds.m[w]);
    move_reference(x, m, true);
    if (!(edge_x == -__builtin_huge_valf())) {
        const float d = (edge_x - m) * kLog2e, e = fast_exp2(d);
        x.s += static_cast<double>(e);
        x.t += static_cast<double>(e * fmaxf(d, kNegMax));
    }
    auto sum = [](auto a, auto b) { return a + b; };
    x.s = over_lanes(x.s, sum);
    x.t = over_lanes(x.t, sum);
    before = over_lanes(before, sum);
    if ((threadIdx.x & 63) == 0) {
        lds.before[wid] = before;
        lds.s[wid] = x.s;
        lds.t[wid] = x.t;
    }
    lds_barrier();
    Part out{m, 0, 0.0, 0.0};
#pragma unroll
    for (int w = 0; w < T / 64; ++w) {
        out.s += lds.s[w];
        out.t += lds.t[w];
        out.before += lds.before[w];
    }
    return out;
}

// The row's outputs, from its sums and its sorted list of n keys (n <= keep).
__device__ inline void write_row(const LogprobsArgs& a, long row, const Part& p, float inv_t, int token,
                                 float z_token, const uint64_t* list, int n) {
    const int tid = threadIdx.x;
    if (tid >= SPEC_LOGPROBS_MAX_K)
        return;
    const float inf = __builtin_huge_valf(), nan = __builtin_nanf("");
    const bool empty = p.m == -inf && p.s == 0.0;
    const bool bad = !empty && !(is_finite_f32(p.m) && is_finite_f64(p.s));
    const double log_s = empty ? 0.0 : log(p.s);
    if (tid == 0) {
        float lp = 0.0f;
        int rank = -1;
        if (token >= 0) {
            lp = empty ? -inf
                       : static_cast<float>((static_cast<double>(z_token * inv_t) - static_cast<double>(p.m)) - log_s);
            rank = empty ? -1 : p.before;
            if (token >= a.vocab) {
                lp = nan;
                rank = -1;
            }
        }
        a.out_logprob[row] = bad ? nan : lp;
        a.out_rank[row] = bad ? -1 : rank;
        a.out_entropy[row] = bad ? nan : empty ? 0.0f : fmaxf(static_cast<float>(log_s - p.t / p.s * (1.0 / static_cast<double>(kLog2e))), 0.0f);
        a.out_norm[2 * row] = bad ? nan : p.m;
        a.out_norm[2 * row + 1] = bad ? nan : static_cast<float>(log_s);
    }
    if (tid < a.keep) {
        int v = -1;
        float lp = bad ? nan : -inf;
        if (!bad && tid < n) {
            const uint64_t key = list[tid];
            const float x = key_logit(key) * inv_t;
            if (x > -inf) {  // scaled below every number: masked as well
                v = key_token(key);
                lp = static_cast<float>((static_cast<double>(x) - static_cast<double>(p.m)) - log_s);
            }
        }
        a.out_top_token[row * a.keep + tid] = v;
        a.out_top_logprob[row * a.keep + tid] = lp;
    }
}

// One pass over a row or a part of one. The reference is the wavefront's and moves only
// when a sum against it grows past kLazy, so an entry costs one multiply-add to its
// distance, its exponential, and one multiply-add and one addition to the sums, about
// ten instructions with the unpacking, the largest entry and the token's rank. Bound by
// those and by the read at nearly the same rate: 2304 x 152064 bf16 take 121 us without
// a list, 5.8 TB/s, and 152 us with lists of 64, 4.6 TB/s (a plain read: 7.1); 1152 x
// 152064 fp32 118 and 132 us. Few rows are bound by latency: 1 x 128256 fp32 with a list
// of 20 takes 9 us and 4.8 to join its 32 parts. Steps of 256 threads x 4 groups: of 512 or 128 threads, of 2 or 6 groups
// measured slower; five workgroups on a compute unit instead of four 160 us for 176.
template <int DT, int T, int U, bool TOP>
__global__ __launch_bounds__(T, 5) void logprobs_kernel(LogprobsArgs a, int splits, int per_split,
                                                     Part* __restrict__ parts, uint64_t* __restrict__ keys) {
    using Row = RowGroups<DT>;
    constexpr int W = Row::W;
    constexpr int kStep = T * U;
    constexpr int kAside = 64 * U;  // a wavefront's groups of a step
    using Select = Selection<T, DT == kBF16 ? 16 : 12>;
    __shared__ typename std::conditional<TOP, SelectionLds<T>, int>::type select_lds;
    __shared__ typename std::conditional<TOP, GroupLds<T, kAside>, int>::type aside;
    __shared__ JoinLds<T> join_lds;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wid = __builtin_amdgcn_readfirstlane(tid >> 6);
    const long row = blockIdx.x / static_cast<unsigned>(splits);
    const int part = static_cast<int>(blockIdx.x % static_cast<unsigned>(splits));
    const Row r(row_ptr(a.logits, DT, row, a.vocab), a.vocab);
    // Steps go over the groups that lie wholly inside the row; what hangs over at its
    // ends, at most 2 W - 2 entries, are the first part's first threads' own.
    const int whole = max(r.full1 - r.full0, 0);
    const int g0 = r.full0 + min(part * per_split, whole);
    const int g1 = r.full0 + min(part * per_split + per_split, whole);
    const int token = a.token[row];
    const float inv_t = row_scale(a.temperature, row);
    const bool unit = inv_t == 1.0f;
    uint4 q[U];
    // Groups past the end request the last one, and are put right when they are used
    // (without a branch: at its end the loads would be waited for).
    auto request = [&](int g) { return r.request_inside(min(g + tid, g1 - 1)); };
    if (g0 < g1) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            q[u] = request(g0 + u * T);
    }
    const float inf = __builtin_huge_valf(), nan = __builtin_nanf("");
    const bool given = token >= 0 && token < a.vocab;
    const float z_token = given ? r.at_global(token) : nan;  // nothing is larger than or equal to a NaN
    // Entries before the token in the order are those above z_token, and in front of it
    // those above the next number below: not (z <= NaN) is true of -inf as well.
    const float z_front = z_token == -inf ? nan : from_order32(z_token == 0.0f ? -2 : order32(z_token) - 1);
    const int token_group = given ? static_cast<int>(r.group_of(token)) : 0;

    float most = -inf;         // the thread's largest logit
    int before = 0, ties = 0;  // the wavefront's entries before the token, the thread's others
    int edge = 0;
    if (part == 0 && tid < a.vocab - whole * W) {  // an entry at an end of the row
        edge = tid < (whole ? (W - r.shift) % W : a.vocab) ? tid : tid + whole * W;
        most = r.at_global(edge);
        ties = most > z_token || (most == z_token && edge < token);
    }
    const float edge_z = most, edge_x = most * inv_t;

    // The wavefront's reference in units of x (-inf: none yet, which is the far one of
    // binary32's lowest value), and whether it has met entries of -inf.
    float ref_x = -inf;
    bool holes = false;
    Sums sum{kNegMax, true, 0.0, 0.0};
    float s_group = 0.0f, t_group = 0.0f;  // of a step, added to sum at its end
    float bar_z = kNegMax;                 // logits below it are not among the first (-inf never is)
    int put_aside = 0;                     // groups, by this wavefront

    // A group's sums, of scaled logits x.
    auto add_up = [&](const float (&x)[W], float top) {
        for (;;) {
            float d[W], e[W];
            if (sum.far) {
#pragma unroll
                for (int i = 0; i < W; ++i)
                    d[i] = (x[i] - sum.ref) * kLog2e;
            } else {
#pragma unroll
                for (int i = 0; i < W; ++i)
                    d[i] = __builtin_fmaf(x[i], kLog2e, -sum.ref);
            }
            if (holes) {  // 0 times the lowest value is 0; a NaN stays one
#pragma unroll
                for (int i = 0; i < W; ++i)
                    d[i] = maximum(d[i], kNegMax);
            }
#pragma unroll
            for (int i = 0; i < W; ++i)
                e[i] = fast_exp2(d[i]);
            float t = e[0] * d[0], t2 = e[1] * d[1];
#pragma unroll
            for (int i = 2; i < W; i += 2) {
                t = __builtin_fmaf(e[i], d[i], t);
                t2 = __builtin_fmaf(e[i + 1], d[i + 1], t2);
            }
            t += t2;
#pragma unroll
            for (int n = W / 2; n > 0; n >>= 1)
#pragma unroll
                for (int i = 0; i < n; ++i)
                    e[i] += e[i + n];
            const float s = e[0];
            // the same in the whole wavefront, and no more often than there are causes
            if (__ballot(!(s <= kLazy) || !(t == t))) {
                if (!holes && __ballot(!(t == t))) {  // an entry of -inf; more are likely
                    holes = true;
                    continue;
                }
                const float best = uniform(over_lanes(max3(most, top, top), [](float a, float b) { return max3(a, b, b); }) * inv_t);
                if (best > ref_x) {
                    ref_x = best;
                    sum.s += static_cast<double>(s_group);
                    sum.t += static_cast<double>(t_group);
                    s_group = t_group = 0.0f;
                    const bool far = !(fabsf(best) < kReach);
                    move_reference(sum, far ? best : best * kLog2e, far);
                    continue;
                }
            }
            s_group += s;
            t_group += t;
            return;
        }
    };
    // The wavefront's groups that reach the bar are put aside.
    auto collect = [&](const uint4& x, float top, int at) {
        if constexpr (TOP) {
            const uint64_t mask = __ballot(top >= bar_z);
            if (mask) {
                const int slot = put_aside + lanes_below(mask);
                if (top >= bar_z && slot < kAside) {
                    aside.data[wid][slot] = x;
                    aside.at[wid][slot] = at;
                }
                put_aside += __popcll(mask);
            }
        }
    };

    // Of the first step's groups, which are all put aside, those that reach the bar.
    auto narrow_aside = [&]() {
        if constexpr (TOP) {
            const int n = put_aside;
            put_aside = 0;
#pragma unroll 1
            for (int i0 = 0; i0 < n; i0 += 64) {
                const int i = min(i0 + lane, kAside - 1);
                const uint4 x = aside.data[wid][i];
                const int at = aside.at[wid][i];
                float z[W];
                Row::unpack(x, z);
                collect(x, i0 + lane < n ? largest(z) : -inf, at);  // to a place at or before its own
            }
        }
    };

    auto body = [&](auto& sel) {
        // Ends the segment [from, to). If it had more groups than there is place for, its
        // steps are gone through again, from memory, each as a segment.
        auto close = [&](int from, int to) {
            if constexpr (TOP) {
                auto end = [&](bool first, bool last) {
                    if (put_aside > kAside)
                        select_lds.lost = 1;
                    wave_order();  // groups are read by other lanes than put them aside
                    if (first) {
                        sel.begin(most, (g1 - g0) / 64);
                        bar_z = logit_at_least(static_cast<uint32_t>(sel.bar >> 32));
                        narrow_aside();
                        wave_order();
                    }
                    const bool done = sel.close(last, [&]() {
                        // Lane by lane the next entry that reaches the bar: most groups have one.
                        const int n = min(put_aside, kAside);
#pragma unroll 1
                        for (int i0 = 0; i0 < n; i0 += 64) {
                            const int i = min(i0 + lane, kAside - 1);
                            float z[W];
                            Row::unpack(aside.data[wid][i], z);
                            const int v0 = static_cast<int>(r.element(aside.at[wid][i]));
                            unsigned hits = 0;
#pragma unroll
                            for (int e = 0; e < W; ++e)
                                hits |= z[e] >= bar_z ? 1u << e : 0u;
                            hits = i0 + lane < n ? hits : 0u;
                            while (__ballot(hits != 0)) {
                                const int e = __builtin_ctz(hits | 1u << W);
                                float y = z[0];
#pragma unroll
                                for (int k = 1; k < W; ++k)
                                    y = e == k ? z[k] : y;
                                const uint64_t key[1] = {make_key(y, v0 + e)};
                                const bool has[1] = {hits != 0 && key[0] >= sel.bar};
                                sel.put(has, key, sel.cur);
                                hits &= hits - 1;
                            }
                        }
                        if (first) {
                            const uint64_t key[1] = {make_key(edge_z, edge)};
                            const bool has[1] = {edge_z >= kNegMax && key[0] >= sel.bar};
                            sel.put(has, key, sel.cur);
                        }
                    });
                    put_aside = 0;
                    bar_z = logit_at_least(static_cast<uint32_t>(sel.bar >> 32));
                    return done;
                };
                if (end(from == g0, to == g1))
                    return;
#pragma unroll 1
                for (int g = from; g < to; g += kStep) {
#pragma unroll 1
                    for (int u = 0; u < U; ++u) {
                        const int at = g + u * T + tid;
                        const uint4 x = at < g1 ? r.request_inside(at) : Row::neg_inf();
                        float z[W];
                        Row::unpack(x, z);
                        collect(x, largest(z), at);
                    }
                    end(false, g + kStep >= g1);
                }
            }
        };

        int segment = g0, segment_end = g0 + kStep;
#pragma unroll 1
        for (int g = g0; g < g1; g += kStep) {
            const bool last = g + kStep > g1;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int at = g + u * T + tid;
                uint4 x = q[u];
                if (last && at >= g1)
                    x = Row::neg_inf();
                float z[W];
                Row::unpack(x, z);
                const float top = largest(z);
                collect(x, top, at);
                q[u] = request(g + kStep + u * T);
                if (__ballot(top >= z_token)) {
                    const float above = at >= g1 ? inf : at < token_group ? z_front : z_token;
#pragma unroll
                    for (int i = 0; i < W; ++i)
                        before += static_cast<int>(__popcll(__ballot(!(z[i] <= above))));
                    if (at == token_group && at < g1) {  // ties in front of the token in its own group
                        const int to = static_cast<int>(token - r.element(at));
#pragma unroll
                        for (int i = 0; i < W; ++i)
                            ties += z[i] == z_token && i < to;
                    }
                }
                if (!unit) {
#pragma unroll
                    for (int i = 0; i < W; ++i)
                        z[i] = scale_logit(z[i], inv_t);
                }
                add_up(z, top);
                most = max3(most, top, top);
            }
            sum.s += static_cast<double>(s_group);
            sum.t += static_cast<double>(t_group);
            s_group = t_group = 0.0f;
            // Segments of 1, 3, 12, 48, .. steps: each makes four times of what has been seen,
            // and lets about 3 keep new keys through.
            if (TOP && (g + kStep >= segment_end || g + kStep >= g1)) {
                close(segment, min(segment_end, g1));
                segment_end += 3 * (segment_end - g0);
                segment = g + kStep;
            }
        }
        if (TOP && g0 == g1)  // a row of no whole group, or a part behind the row's end
            close(g0, g0);
    };
    const uint64_t* list = nullptr;
    int n = 0;
    if constexpr (TOP) {
        Select sel(select_lds, a.keep);
        body(sel);
        sel.sort();
        n = sel.held;
        list = select_lds.lists[sel.cur];
    } else {
        int none = 0;
        body(none);
    }
    const Part p = join_threads<T>(most * inv_t, ties + (lane == 0 ? before : 0), sum, edge_x, join_lds);
    if (splits == 1) {
        write_row(a, row, p, inv_t, token, z_token, list, n);
        return;
    }
    const long at = row * splits + part;
    if (tid == 0)
        parts[at] = p;
    if (TOP && tid < a.keep)
        keys[at * a.keep + tid] = tid < n ? list[tid] : 0;
}

// A row's parts joined, one workgroup per row: sums against the largest part's M, the
// first of all parts' keys. Bound by latency (4.8 us for 32 parts with lists of 20).
template <int DT>
__global__ __launch_bounds__(kT) void logprobs_merge_kernel(LogprobsArgs a, int splits,
                                                            const Part* __restrict__ parts,
                                                            const uint64_t* __restrict__ keys) {
    __shared__ SelectionLds<kT> select_lds;
    __shared__ JoinLds<kT> join_lds;
    const int tid = threadIdx.x;
    const long row = blockIdx.x;
    const int total = splits * a.keep;
    const uint64_t* row_keys = keys + row * total;
    constexpr int kHeld = 4;  // keys of a thread in registers
    uint64_t own[kHeld];
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
        own[i] = tid + i * kT < total ? row_keys[tid + i * kT] : 0;
    const int token = a.token[row];
    const float inv_t = row_scale(a.temperature, row);
    const RowGroups<DT> r(row_ptr(a.logits, DT, row, a.vocab), a.vocab);
    const float z_token = token >= 0 && token < a.vocab ? r.at_global(token) : 0.0f;
    float m = -__builtin_huge_valf();
    Sums sum{m, true, 0.0, 0.0};
    int before = 0;
    for (int i = tid; i < splits; i += kT) {
        const Part p = parts[row * splits + i];
        Sums x{p.m, true, p.s, p.t};
        m = fmaxf(m, p.m);
        move_reference(sum, m, true);
        move_reference(x, m, true);
        sum.s += x.s;
        sum.t += x.t;
        before += p.before;
    }
    Selection<kT, DT == kBF16 ? 16 : 12> sel(select_lds, a.keep);
    if (a.keep) {
        uint64_t best = own[0];
#pragma unroll
        for (int i = 1; i < kHeld; ++i)
            best = own[i] > best ? own[i] : best;
        if (total > kCap / 4)
            sel.begin(best ? key_logit(best) : kNegMax, total / 64);
        sel.close(true, [&]() {
            bool has[kHeld];
#pragma unroll
            for (int i = 0; i < kHeld; ++i)
                has[i] = own[i] >= sel.bar;
            sel.put(has, own, sel.cur);
            for (int i0 = kHeld * kT; i0 < total; i0 += kT) {
                const uint64_t key[1] = {i0 + tid < total ? row_keys[i0 + tid] : 0};
                const bool one[1] = {key[0] >= sel.bar};
                sel.put(one, key, sel.cur);
            }
        });
        sel.sort();
    }
    const Part p = join_threads<kT>(m, before, sum, -__builtin_huge_valf(), join_lds);
    write_row(a, row, p, inv_t, token, z_token, select_lds.lists[sel.cur], sel.held);
}

// ---------------------------------------------------------------- backward ---

struct BackwardArgs {
    const void* logits;
    const int32_t* token;
    const float* temperature;
    const float* norm;
    const float* entropy;
    const float* grad_logprob;
    const float* grad_entropy;  // NULL: 0
    void* out_grad;
    int vocab;
};

// With l = log p = (x - M) - log S: grad = p (c0 + c1 l), c0 = -r (a + b H) and
// c1 = -r b, and r a more at the token. Bound by reading and writing the row. One
// step of a workgroup's loads per split: workgroups follow the rows, so that
// together they read and write one advancing front: 2304 x 152064 bf16 take 223 to 228
// us, 1152 x 152064 fp32 220 to 228, 6.1 to 6.4 TB/s, the rate of a large copy.
constexpr int kBackU = 5;

// The exponential instruction gives 0 for results below 2^-126 (a log p under
// kSubnormal), whose products with large coefficients are ordinary numbers, and with
// others subnormal ones. There it forms 2^120 p, and the coefficient is taken times
// 2^-120: what it still loses, p below 2^-246, times a coefficient of at
// most 1e25 * 201 is less than half of the smallest number. So p is 0 below kNothing
// (at -inf the product with log p would be NaN).
constexpr float kSubnormal = -87.0f, kNothing = -200.0f;
constexpr float kRaise = 120.0f, kLower = 0x1p-120f;

template <int DT>
__global__ __launch_bounds__(kT) void logprobs_backward_kernel(BackwardArgs a, int splits, int per_split) {
    using Row = RowGroups<DT>;
    constexpr int W = Row::W;
    const int tid = threadIdx.x;
    const long row = blockIdx.x / static_cast<unsigned>(splits);
    const int part = static_cast<int>(blockIdx.x % static_cast<unsigned>(splits));
    const Row r(row_ptr(a.logits, DT, row, a.vocab), a.vocab);
    const int g0 = min(part * per_split, r.groups);
    const int g1 = min(g0 + per_split, r.groups);
    char* out = static_cast<char*>(a.out_grad) + row * static_cast<long>(a.vocab) * Row::ESZ;
    const bool whole = (reinterpret_cast<uintptr_t>(out) & 15) == static_cast<uintptr_t>(r.shift) * Row::ESZ;
    uint4 q[kBackU];
    r.template load<kBackU, kT>(g0, tid, g1, q);
    const int token = a.token[row];
    const float m = a.norm[2 * row], log_s = a.norm[2 * row + 1];
    const float inv_t = row_scale(a.temperature, row);
    const float inf = __builtin_huge_valf(), nan = __builtin_nanf("");
    if (m == -inf || !is_finite_f32(m) || !is_finite_f32(log_s) || !(inv_t == inv_t) || token >= a.vocab) {
        const bool empty = m == -inf && inv_t == inv_t && token < a.vocab;
        fill<DT, kT>(r, out, g0, g1, whole, empty ? 0.0f : nan);
        return;
    }
    const double scale = static_cast<double>(inv_t);
    const double ra = token >= 0 ? scale * static_cast<double>(a.grad_logprob[row]) : 0.0;
    const double rb = a.grad_entropy ? scale * static_cast<double>(a.grad_entropy[row]) : 0.0;
    const double d0 = -(ra + (rb == 0.0 ? 0.0 : rb * static_cast<double>(a.entropy[row]))), d1 = -rb;
    const float c0 = static_cast<float>(d0), c1 = static_cast<float>(d1);
    // Coefficients that binary32 holds with room for what they are multiplied by, and
    // that leave nothing of a p below 2^-246; the others (and NaNs) go by binary64.
    const bool near = fabs(d0) <= 1e25 && fabs(d1) <= 1e25;
    const long hot = token >= 0 ? r.group_of(token) : -1;
    for (int g = g0;;) {
#pragma unroll
        for (int u = 0; u < kBackU; ++u) {
            const int at = g + tid + u * kT;
            if (at >= g1)
                continue;
            float z[W], l[W], d[W];
            Row::unpack(q[u], z);
#pragma unroll
            for (int i = 0; i < W; ++i) {
                l[i] = fmaxf((scale_logit(z[i], inv_t) - m) - log_s, kNothing);
                d[i] = fast_exp2(l[i] * kLog2e) * __builtin_fmaf(c1, l[i], c0);
            }
            float least = l[0];
#pragma unroll
            for (int i = 1; i < W; ++i)
                least = fminf(least, l[i]);
            if (least < kSubnormal) {
                bool some = false;  // or masked entries alone
#pragma unroll
                for (int i = 0; i < W; ++i)
                    some |= l[i] < kSubnormal && l[i] > kNothing;
                if (some) {
#pragma unroll
                    for (int i = 0; i < W; ++i)
                        if (l[i] < kSubnormal)
                            d[i] = fast_exp2(__builtin_fmaf(l[i], kLog2e, kRaise)) *
                                   (__builtin_fmaf(c1, l[i], c0) * kLower);
                }
            }
            if (at == hot || !near) {
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    const float x = scale_logit(z[i], inv_t);
                    const double far = fmax((static_cast<double>(x) - static_cast<double>(m)) - static_cast<double>(log_s), -800.0);
                    const bool one = r.element(at) + i == token;
                    if (one || !near)  // a masked entry has none, also of weights that are not finite
                        d[i] = static_cast<float>((one ? ra : 0.0) + (x == -inf ? 0.0 : exp(far) * (d0 + d1 * far)));
                }
            }
            store_group<DT>(r, out, at, whole, d);
        }
        g += kBackU * kT;
        if (g >= g1)
            break;
        r.template load<kBackU, kT>(g, tid, g1, q);
    }
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

constexpr long kMostGroups = (1L << 32) / kT - 1;  // workgroups of one dispatch

// Workgroups that the chip holds at a time (the kernel's launch bounds), and parts of
// rows that a workspace has place for.
constexpr int kAtOnce = 256 * 5;

// Parts of a row when there are `rows`: as many as are at work at once, none shorter
// than a step. Measured against half as many and half as many more (us, bf16, lists of
// 20): 64 rows of 152064 21.4 : 24.2 and 21.2, 256 rows 35.2 : 37.3 and 42.5, 900 rows of
// 32000, which stay whole, 26.0 : 26.0 and 35.3. Rows that leave places empty, or fill
// them a second time in part, are not better off in more parts (of 152064; one part
// first): 600 rows, the last that are split, 59.8 : 55.5 in two; 650 59.1 : 65.0, 800
// 67.0 : 72.2, 1290 98.7 : 100.6, 1500 101.6 : 110.1.
struct Split {
    int splits, per_split;
};

Split split_of(int rows, int vocab, int dtype) {
    const long groups = static_cast<long>(vocab) / (dtype == SPEC_BF16 ? 8 : 4) + 2;  // at any alignment
    constexpr long kStep = kT * kU;
    const long steps = (groups + kStep - 1) / kStep;
    const long want = std::max(1, kAtOnce / rows);
    const long per = (steps + want - 1) / want;
    // Of the same length, in whole lines: a short one at the end has no bar to begin with
    // (1 x 50000 bf16, a list of 20: 13.2 us for 40.4).
    const long splits = (steps + per - 1) / per;
    return {static_cast<int>(splits), static_cast<int>(((groups + splits - 1) / splits + 7) / 8 * 8)};
}

}  // namespace
}  // namespace specv

using namespace specv;

struct spec_logprobs_ctx {
    int rows = 0, V = 0, K = 0, dtype = 0;
    hipStream_t stream = nullptr;
    int device = 0;
    void* ws = nullptr;
    Part* parts = nullptr;
    uint64_t* keys = nullptr;
};

extern "C" {

int spec_logprobs_init(int rows, int vocab, int top_k, int dtype, void* hip_stream,
                       spec_logprobs_ctx** out_ctx) {
    if (!out_ctx)
        return SPEC_EINVAL;
    *out_ctx = nullptr;
    if (rows < 1 || rows > kMostGroups || vocab < 1 || top_k < 0 || top_k > SPEC_LOGPROBS_MAX_K ||
        (dtype != SPEC_F32 && dtype != SPEC_BF16))
        return SPEC_EINVAL;
    spec_logprobs_ctx* ctx = new (std::nothrow) spec_logprobs_ctx();
    if (!ctx)
        return SPEC_ENOMEM;
    ctx->rows = rows;
    ctx->V = vocab;
    ctx->K = top_k;
    ctx->dtype = dtype;
    ctx->stream = static_cast<hipStream_t>(hip_stream);
    if (hipGetDevice(&ctx->device) != hipSuccess) {
        delete ctx;
        return SPEC_EHIP;
    }
    const size_t most = kAtOnce;  // rows that are split have no more parts together
    if (hipMalloc(&ctx->ws, most * (sizeof(Part) + sizeof(uint64_t) * top_k)) != hipSuccess) {
        (void)hipGetLastError();
        delete ctx;
        return SPEC_ENOMEM;
    }
    ctx->parts = static_cast<Part*>(ctx->ws);
    ctx->keys = reinterpret_cast<uint64_t*>(ctx->parts + most);
    *out_ctx = ctx;
    return SPEC_OK;
}

int spec_logprobs_set_stream(spec_logprobs_ctx* ctx, void* hip_stream) {
    if (!ctx)
        return SPEC_EINVAL;
    ctx->stream = static_cast<hipStream_t>(hip_stream);
    return SPEC_OK;
}

int spec_token_logprobs(spec_logprobs_ctx* ctx, int rows, const void* logits, const int32_t* token,
                        const float* temperature, float* out_logprob, int32_t* out_rank,
                        float* out_entropy, int32_t* out_top_token, float* out_top_logprob,
                        float* out_norm) {
    if (!ctx || rows < 0 || rows > ctx->rows)
        return SPEC_EINVAL;
    if (rows == 0)
        return SPEC_OK;
    const size_t esz = ctx->dtype == SPEC_BF16 ? 2 : 4;
    if (!logits || !token || !out_logprob || !out_rank || !out_entropy || !out_norm || !aligned(logits, esz) ||
        !aligned(token, 4) || !aligned(temperature, 4) || !aligned(out_logprob, 4) || !aligned(out_rank, 4) ||
        !aligned(out_entropy, 4) || !aligned(out_norm, 4))
        return SPEC_EINVAL;
    if (ctx->K && (!out_top_token || !out_top_logprob || !aligned(out_top_token, 4) || !aligned(out_top_logprob, 4)))
        return SPEC_EINVAL;
    int device = 0;
    if (hipGetDevice(&device) != hipSuccess)
        return SPEC_EHIP;
    if (device != ctx->device)
        return SPEC_ESTATE;
    const LogprobsArgs a{logits, token, temperature, out_logprob, out_rank, out_entropy,
                         out_top_token, out_top_logprob, out_norm, ctx->V, ctx->K};
    const Split p = split_of(rows, ctx->V, ctx->dtype);
    const dim3 grid(static_cast<unsigned>(static_cast<long>(rows) * p.splits)), block(kT);
    hipStream_t s = ctx->stream;
#define SPEC_LOGPROBS(DT, TOP) \
    logprobs_kernel<DT, kT, kU, TOP><<<grid, block, 0, s>>>(a, p.splits, p.per_split, ctx->parts, ctx->keys)
    const bool bf16 = ctx->dtype == SPEC_BF16;
    if (ctx->K)
        bf16 ? SPEC_LOGPROBS(kBF16, true) : SPEC_LOGPROBS(kF32, true);
    else
        bf16 ? SPEC_LOGPROBS(kBF16, false) : SPEC_LOGPROBS(kF32, false);
#undef SPEC_LOGPROBS
    if (hipGetLastError() != hipSuccess)
        return SPEC_EHIP;
    if (p.splits > 1) {
        const dim3 all(static_cast<unsigned>(rows));
        if (bf16)
            logprobs_merge_kernel<kBF16><<<all, block, 0, s>>>(a, p.splits, ctx->parts, ctx->keys);
        else
            logprobs_merge_kernel<kF32><<<all, block, 0, s>>>(a, p.splits, ctx->parts, ctx->keys);
        if (hipGetLastError() != hipSuccess)
            return SPEC_EHIP;
    }
    return SPEC_OK;
}

int spec_token_logprobs_backward(spec_logprobs_ctx* ctx, int rows, const void* logits,
                                 const int32_t* token, const float* temperature, const float* norm,
                                 const float* entropy, const float* grad_logprob,
                                 const float* grad_entropy, void* out_grad) {
    if (!ctx || rows < 0 || rows > ctx->rows)
        return SPEC_EINVAL;
    if (rows == 0)
        return SPEC_OK;
    const size_t esz = ctx->dtype == SPEC_BF16 ? 2 : 4;
    if (!logits || !token || !norm || !entropy || !grad_logprob || !out_grad || !aligned(logits, esz) ||
        !aligned(token, 4) || !aligned(temperature, 4) || !aligned(norm, 4) || !aligned(entropy, 4) ||
        !aligned(grad_logprob, 4) || !aligned(grad_entropy, 4) || !aligned(out_grad, esz))
        return SPEC_EINVAL;
    if (out_grad != logits) {
        const uintptr_t x = reinterpret_cast<uintptr_t>(logits), y = reinterpret_cast<uintptr_t>(out_grad);
        const uintptr_t n = static_cast<uintptr_t>(rows) * ctx->V * esz;
        if (x < y + n && y < x + n)
            return SPEC_EINVAL;
    }
    int device = 0;
    if (hipGetDevice(&device) != hipSuccess)
        return SPEC_EHIP;
    if (device != ctx->device)
        return SPEC_ESTATE;
    const BackwardArgs a{logits, token, temperature, norm, entropy, grad_logprob, grad_entropy, out_grad, ctx->V};
    const long groups = static_cast<long>(ctx->V) / (ctx->dtype == SPEC_BF16 ? 8 : 4) + 2;  // at any alignment
    const long steps = (groups + kT * kBackU - 1) / (kT * kBackU);
    const long most = kMostGroups / rows;  // of one dispatch
    const long per = (steps + most - 1) / most * (kT * kBackU);
    const long splits = (groups + per - 1) / per;
    const dim3 grid(static_cast<unsigned>(rows * splits)), block(kT);
    if (ctx->dtype == SPEC_BF16)
        logprobs_backward_kernel<kBF16><<<grid, block, 0, ctx->stream>>>(a, static_cast<int>(splits), static_cast<int>(per));
    else
        logprobs_backward_kernel<kF32><<<grid, block, 0, ctx->stream>>>(a, static_cast<int>(splits), static_cast<int>(per));
    return hipGetLastError() == hipSuccess ? SPEC_OK : SPEC_EHIP;
}

int spec_logprobs_destroy(spec_logprobs_ctx* ctx) {
    if (!ctx)
        return SPEC_EINVAL;
    int rc = SPEC_OK;
    if (hipStreamSynchronize(ctx->stream) != hipSuccess)
        rc = SPEC_EHIP;
    if (ctx->ws && hipFree(ctx->ws) != hipSuccess)
        rc = SPEC_EHIP;
    delete ctx;
    return rc;
}

}  // extern "C"
