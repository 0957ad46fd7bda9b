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

#include <cstdint>
#include <new>
#include <type_traits>

#include "launch.hpp"
#include "rows.hpp"
#include "select.hpp"
#include "spec_logprobs.h"
#include "stage.hpp"

namespace specv {
namespace {

constexpr int kT = kBlock;  // threads of a workgroup
constexpr int kU = 4;       // 16-byte groups of a step per thread
constexpr int kCap = 512;   // collected entries

// What a part of a row leaves: M (-inf: no entry), the sums, the entries before
// the token.
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

// A row's first entries, gathered over segments of it: keys that reach a bar are
// put into the list as they are met, and the workgroup looks at the list at the
// end of a segment only, when it is ranked down to its keep largest keys, the last
// of which is the next segment's bar. What is kept does not depend on the order
// in which keys arrive.
struct SelectionLds {
    uint64_t list[kCap];
    uint64_t bar;
    int count;  // keys offered, also those that the list had no place for
};

template <int T>
struct Selection {
    static constexpr int kPer = (kCap + T - 1) / T;  // keys that a thread ranks
    SelectionLds& lds;
    const int keep;
    int held = 0;      // keys that earlier segments left in the list, largest first
    uint64_t bar = 1;  // keys below it are not among the first; 0 marks no key

    __device__ Selection(SelectionLds& l, int k) : lds(l), keep(k) {
        if (threadIdx.x == 0)
            lds.count = 0;
    }

    __device__ void put(uint64_t key) {
        const int slot = atomicAdd(&lds.count, 1);
        if (slot < kCap)
            lds.list[slot] = key;
    }

    // After a segment, every thread of the workgroup. False: the list had no place
    // for some of the segment's keys. The bar is then higher (the keep-th largest key
    // that did fit: more than keep of them are of this segment, and keys are unique),
    // and the segment's keys have to be put again.
    __device__ bool close() {
        lds_barrier();
        const int n = lds.count;
        const bool fits = n <= kCap;
        const int here = fits ? n : kCap;
        uint64_t mine[kPer];
        int place[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int at = static_cast<int>(threadIdx.x) + i * T;
            mine[i] = at < here ? lds.list[at] : 0;
            place[i] = kCap;
            if ((at & ~63) < here) {  // wavefronts without a key have nothing to rank
                int larger = 0;
#pragma unroll 8
                for (int j = 0; j < here; ++j)
                    larger += lds.list[j] > mine[i];
                if (at < here)
                    place[i] = larger;
            }
        }
        lds_barrier();
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            if (fits && place[i] < keep)
                lds.list[place[i]] = mine[i];
            if (place[i] == keep - 1)
                lds.bar = mine[i];
        }
        if (fits)
            held = min(n, keep);
        if (threadIdx.x == 0)
            lds.count = held;
        lds_barrier();
        if (n >= keep)
            bar = lds.bar;
        return fits;
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

template <int W>
__device__ __forceinline__ float largest(const float (&z)[W]) {
    if constexpr (W == 8)
        return max3(max3(z[0], z[1], z[2]), max3(z[3], z[4], z[5]), max3(z[6], z[7], z[7]));
    else
        return max3(max3(z[0], z[1], z[2]), z[3], z[3]);
}

// Sums of e = exp(x - ref) and of e (x - ref) over some entries.
struct Sums {
    float ref;
    double s, t;
};

// The same against another reference.
__device__ inline void move_reference(float from, float to, double& s, double& t) {
    if (from == to || s == 0.0)
        return;
    const float d = from - to;
    const double f = static_cast<double>(fast_exp2(__builtin_fmaf(d, kLog2e, d * kLog2eLow)));
    t = f == 0.0 ? s * f : f * (t + s * static_cast<double>(d));  // d may be -inf; a NaN stays one
    s *= f;
}

// Joins the threads' parts, against the largest entry m: in every thread of the
// first wavefront afterwards.
template <int T>
struct JoinLds {
    float m[T / 64];
    int before[T / 64];
    double s[T / 64], t[T / 64];
};

template <int T>
__device__ inline Part join_threads(float m, int before, Sums x, JoinLds<T>& lds) {
    const int wid = threadIdx.x >> 6;
    m = wave_max(m);
    if ((threadIdx.x & 63) == 0)
        lds.m[wid] = m;
    lds_barrier();
#pragma unroll
    for (int w = 0; w < T / 64; ++w)
        m = fmaxf(m, lds.m[w]);
    move_reference(x.ref, m, x.s, x.t);
    x.s = wave_sum(x.s);
    x.t = wave_sum(x.t);
#pragma unroll
    for (int off = 32; off > 0; off >>= 1)
        before += __shfl_xor(before, off, 64);
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
        a.out_entropy[row] = bad ? nan : empty ? 0.0f : fmaxf(static_cast<float>(log_s - p.t / p.s), 0.0f);
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

// Sums over a step are taken against the reference so far as long as their terms
// stay below this; beyond, the reference becomes the thread's largest entry. A
// thread without an entry has binary32's lowest value for its reference, whose
// terms overflow for every entry above it.
constexpr float kLazy = 256.0f;

template <int DT, int T, int U, bool TOP>
__global__ __launch_bounds__(T) void logprobs_kernel(LogprobsArgs a, int splits, int per_split,
                                                     Part* __restrict__ parts, uint64_t* __restrict__ keys) {
    using Row = RowGroups<DT>;
    constexpr int W = Row::W;
    constexpr int kStep = T * U;
    __shared__ SelectionLds select_lds;
    __shared__ int bars[TOP ? T + 1 : 1];
    __shared__ JoinLds<T> join_lds;
    const int tid = threadIdx.x;
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
    uint4 next[U];
    // Groups past the end request the last one, and are put right before they are used
    // (without a branch: at its end the loads would be waited for).
    auto request = [&](int g) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            next[u] = r.request_inside(min(g + u * T + tid, g1 - 1));
    };
    if (g0 < g1)
        request(g0);
    const float inf = __builtin_huge_valf(), nan = __builtin_nanf("");
    const bool given = token >= 0 && token < a.vocab;
    const float z_token = given ? r.at_global(token) : nan;  // nothing is larger than or equal to a NaN

    float most = -inf;  // the thread's largest logit
    Sums sum{kNegMax, 0.0, 0.0};
    int before = 0;
    int edge = -1;  // the thread's entry at an end of the row
    if (part == 0 && tid < a.vocab - whole * W) {
        edge = tid < (whole ? (W - r.shift) % W : a.vocab) ? tid : tid + whole * W;
        most = r.at_global(edge);
        const float x = scale_logit(most, inv_t);
        if (!(x == -inf))
            sum = Sums{x, static_cast<double>(fast_exp2(x - x)), 0.0};
        before = most > z_token || (most == z_token && edge < token);
    }
    Selection<T> sel(select_lds, a.keep);
    float bar_z = kNegMax;  // logits below it are not among the first (-inf never is)

    // Keys of a step's entries that reach the bar.
    auto collect = [&](const uint4 (&q)[U], const float (&top)[U], int g) {
        unsigned groups = 0;
#pragma unroll
        for (int u = 0; u < U; ++u)
            groups |= top[u] >= bar_z ? 1u << u : 0u;
        while (groups) {
            const int u = __builtin_ctz(groups);
            groups &= groups - 1;
            uint4 x = q[0];
#pragma unroll
            for (int i = 1; i < U; ++i) {
                x.x = u == i ? q[i].x : x.x;
                x.y = u == i ? q[i].y : x.y;
                x.z = u == i ? q[i].z : x.z;
                x.w = u == i ? q[i].w : x.w;
            }
            float z[W];
            Row::unpack(x, z);
            const int v0 = static_cast<int>(r.element(g + tid + u * T));
            unsigned hits = 0;
#pragma unroll
            for (int e = 0; e < W; ++e)
                hits |= z[e] >= bar_z ? 1u << e : 0u;
            while (hits) {
                const int e = __builtin_ctz(hits);
                hits &= hits - 1;
                float y = z[0];
#pragma unroll
                for (int i = 1; i < W; ++i)
                    y = e == i ? z[i] : y;
                const uint64_t key = make_key(y, v0 + e);
                if (key >= sel.bar)
                    sel.put(key);
            }
        }
    };
    auto collect_edge = [&](float z) {
        if (z >= bar_z && edge >= 0) {
            const uint64_t key = make_key(z, edge);
            if (key >= sel.bar)
                sel.put(key);
        }
    };
    auto settle = [&](uint4 (&q)[U], int g) {
        if (g + kStep > g1) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (g + u * T + tid >= g1)
                    q[u] = Row::neg_inf();
        }
    };
    auto tops = [&](const uint4 (&q)[U], float (&top)[U]) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float z[W];
            Row::unpack(q[u], z);
            top[u] = largest(z);
        }
    };
    // Ends the segment [from, to): its list is ranked, after its keys have been put
    // again, from memory, as often as the list did not hold them.
    auto close = [&](int from, int to) {
        for (;;) {
            const bool done = sel.close();
            if (sel.bar > 1)
                bar_z = key_logit(sel.bar);
            if (done)
                return;
#pragma unroll 1
            for (int g = from; g < to; g += kStep) {
                uint4 q[U];
                float top[U];
#pragma unroll
                for (int u = 0; u < U; ++u)
                    q[u] = r.request_inside(min(g + u * T + tid, g1 - 1));
                settle(q, g);
                tops(q, top);
                collect(q, top, g);
            }
            if (from == g0 && edge >= 0)
                collect_edge(r.at_global(edge));
        }
    };

    int segment = g0, segment_end = g0 + kStep;
#pragma unroll 1
    for (int g = g0; g < g1; g += kStep) {
        uint4 q[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            q[u] = next[u];
        settle(q, g);
        request(g + kStep);

        float top[U];  // the largest of each group
        float e_sum, t_sum;
        // exp(x - ref) and its product with x - ref, over the step
        auto add_up = [&]() {
            float e[W], t[W];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float z[W];
                Row::unpack(q[u], z);
                top[u] = largest(z);
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    float d = scale_logit(z[i], inv_t) - sum.ref;
                    const float x = fast_exp2(d * kLog2e);
                    d = fmaxf(d, kNegMax);  // 0 times it is 0 at -inf as well
                    e[i] = u ? e[i] + x : x;
                    t[i] = u ? __builtin_fmaf(x, d, t[i]) : x * d;
                }
            }
#pragma unroll
            for (int n = W / 2; n > 0; n >>= 1)
#pragma unroll
                for (int i = 0; i < n; ++i) {
                    e[i] += e[i + n];
                    t[i] += t[i + n];
                }
            e_sum = e[0];
            t_sum = t[0];
        };
        add_up();
        repack(q);
        float best = top[0];
#pragma unroll
        for (int u = 1; u < U; ++u)
            best = max3(best, top[u], top[u]);
        if (!(e_sum <= kLazy)) {
            const float to = fmaxf(sum.ref, best * inv_t);
            move_reference(sum.ref, to, sum.s, sum.t);
            sum.ref = to;
            add_up();
            repack(q);
        }
        sum.s += static_cast<double>(e_sum);
        sum.t += static_cast<double>(t_sum);

        if (best >= z_token) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (!(top[u] >= z_token) || g + tid + u * T >= g1)
                    continue;
                float z[W];
                Row::unpack(q[u], z);
                // ties count at places [0, to) of the group, before the token
                const long v0 = r.element(g + tid + u * T);
                const int to = static_cast<int>(v0 + W < token ? W : token - v0);
#pragma unroll
                for (int i = 0; i < W; ++i)
                    before += z[i] > z_token || (z[i] == z_token && i < to);
            }
        }
        if constexpr (TOP) {
            if (g == g0) {
                const int held = g1 - g0;
                const int order = bar_of<T, DT == kBF16 ? 16 : 32>(Row::order_of(best), a.keep, held < T ? held : T, bars);
                bar_z = fmaxf(kNegMax, Row::from_order(order));
                collect_edge(most);
            }
            if (best >= bar_z)
                collect(q, top, g);
            // Segments of 1, 1, 2, 4, .. steps: each doubles what has been seen, and lets
            // about keep new keys through.
            if (g + kStep >= segment_end || g + kStep >= g1) {
                close(segment, min(segment_end, g1));
                segment_end += segment_end - g0;
                segment = g + kStep;
            }
        }
        most = max3(most, best, best);
    }
    if (TOP && g0 == g1) {  // a row of no whole group, or a part behind the row's end
        __syncthreads();
        collect_edge(most);
        sel.close();
    }
    const Part p = join_threads<T>(most * inv_t, before, sum, join_lds);
    const int n = sel.held;
    if (splits == 1) {
        write_row(a, row, p, inv_t, token, z_token, select_lds.list, n);
        return;
    }
    const long at = row * splits + part;
    if (tid == 0)
        parts[at] = p;
    if (TOP && tid < a.keep)
        keys[at * a.keep + tid] = tid < n ? select_lds.list[tid] : 0;
}

// A row's parts joined, one workgroup per row.
template <int DT>
__global__ __launch_bounds__(kT) void logprobs_merge_kernel(LogprobsArgs a, int splits,
                                                            const Part* __restrict__ parts,
                                                            const uint64_t* __restrict__ keys) {
    __shared__ SelectionLds select_lds;
    __shared__ int bars[kT + 1];
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
    Sums sum{m, 0.0, 0.0};
    int before = 0;
    for (int i = tid; i < splits; i += kT) {
        Part x = parts[row * splits + i];
        m = fmaxf(sum.ref, x.m);
        move_reference(sum.ref, m, sum.s, sum.t);
        move_reference(x.m, m, x.s, x.t);
        sum = Sums{m, sum.s + x.s, sum.t + x.t};
        before += x.before;
    }
    Selection<kT> sel(select_lds, a.keep);
    if (a.keep) {
        uint64_t best = own[0];
#pragma unroll
        for (int i = 1; i < kHeld; ++i)
            best = own[i] > best ? own[i] : best;
        // the upper half of a key rises with the logit; 0, no key, is the lowest
        const int bar = bar_of<kT, 32>(static_cast<int>(static_cast<uint32_t>(best >> 32) ^ 0x80000000u), a.keep,
                                       total < kT ? total : kT, bars);
        const uint64_t least = static_cast<uint64_t>(static_cast<uint32_t>(bar) ^ 0x80000000u) << 32;
        do {
#pragma unroll
            for (int i = 0; i < kHeld; ++i)
                if (own[i] >= sel.bar && own[i] >= least)
                    sel.put(own[i]);
            for (int i = tid + kHeld * kT; i < total; i += kT) {
                const uint64_t key = row_keys[i];
                if (key >= sel.bar && key >= least)
                    sel.put(key);
            }
        } while (!sel.close());
    }
    const Part p = join_threads<kT>(m, before, sum, join_lds);
    write_row(a, row, p, inv_t, token, z_token, select_lds.list, sel.held);
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
// together they read and write one advancing front.
constexpr int kBackU = 5;

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
    // Coefficients that binary32 holds with room for what they are multiplied by;
    // the others (and NaNs) go by binary64.
    const bool near = fabs(d0) <= 1e30 && fabs(d1) <= 1e30;
    const long hot = token >= 0 ? r.group_of(token) : -1;
    for (int g = g0;;) {
#pragma unroll
        for (int u = 0; u < kBackU; ++u) {
            const int at = g + tid + u * kT;
            if (at >= g1)
                continue;
            float z[W], d[W];
            Row::unpack(q[u], z);
#pragma unroll
            for (int i = 0; i < W; ++i) {
                // below -200 p is 0 (and the product with l would be NaN at -inf)
                const float l = fmaxf((scale_logit(z[i], inv_t) - m) - log_s, -200.0f);
                d[i] = fast_exp2(l * kLog2e) * __builtin_fmaf(c1, l, c0);
            }
            if (at == hot || !near) {
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    const double l = fmax((static_cast<double>(scale_logit(z[i], inv_t)) - static_cast<double>(m)) -
                                              static_cast<double>(log_s), -800.0);
                    const bool one = r.element(at) + i == token;
                    if (one || !near)
                        d[i] = static_cast<float>((one ? ra : 0.0) + exp(l) * (d0 + d1 * l));
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

// Parts of a row when there are `rows`: enough workgroups to fill the chip, none
// shorter than a step.
struct Split {
    int splits, per_split;
};

Split split_of(int rows, int vocab, int dtype) {
    const long groups = static_cast<long>(vocab) / (dtype == SPEC_BF16 ? 8 : 4) + 2;  // at any alignment
    constexpr long kStep = kT * kU;
    const long steps = (groups + kStep - 1) / kStep;
    const long want = (1024 + rows - 1) / rows;
    const long per = (steps + want - 1) / want;
    return {static_cast<int>((steps + per - 1) / per), static_cast<int>(per * kStep)};
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
    // Rows that are split have fewer than 1024 + rows parts together, and only
    // calls of fewer than 1024 rows split them.
    const size_t most = rows < 1024 ? 1024 + static_cast<size_t>(rows) : 2048;
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
