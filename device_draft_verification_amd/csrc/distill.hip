// Distillation from a teacher's top logits, forward and backward
// (spec_distill.h).
//
//   loss = sum_j p_j (log p_j - (x_id(j) - lse)),
//   grad_v = weight / T (P exp(x_v - lse) - sum_{j: id(j) = v} p_j).
//
// Three kernels:
//   distill_forward: one workgroup per row streams it once;
//   distill_backward: a row's groups are split over workgroups (nothing is
//     summed over the vocabulary);
//   distill_loss_grad: one workgroup per row keeps the row in registers between
//     its normaliser and its gradient, so that the logits are read once (of rows
//     that do not fit, the rest is read twice).
// The dense part of the gradient is written first; a barrier later the entries
// of the list, whose students' logits were fetched before anything was
// written, overwrite their places (so the gradient may take the logits' place,
// and no element is rounded twice).
#include <hip/hip_runtime.h>

#include <cstdint>

#include "launch.hpp"
#include "rows.hpp"
#include "spec_distill.h"
#include "stage.hpp"

namespace specv {
namespace {

struct DistillArgs {
    const void* logits;
    const int32_t* ids;
    const float* teacher;
    const double* teacher_lse;  // NULL: the list's own normaliser
    const float* temperature;
    const double* lse_in;       // backward alone: the forward pass's normalisers
    const float* weight;
    float* out_loss;
    double* out_lse;
    void* out_grad;
    int vocab, top_k;
};

// ----------------------------------------------------------------- the list ---

// A row's teacher list after reduction, the same in every thread.
struct RowList {
    bool empty;    // nothing to learn: loss and gradient 0
    bool bad;      // loss and gradient NaN
    float inv_t;
    double mass;   // P
    double inner;  // sum_j p_j (log p_j - x_id(j)), so that loss = inner + P lse
};

// A thread's own entry (threads past the list hold none).
struct Entry {
    int id;    // -1: unused
    float x;   // the student's scaled logit there
    double p;  // the teacher's probability
};

struct ListLds {
    int id[SPEC_DISTILL_MAX_K];
    double p[SPEC_DISTILL_MAX_K];
    float most[4];
    int flags[4];
    double sum[4], inner[4];
};

struct ListFetch {
    float t;      // the row's temperature
    float y;      // the thread's teacher logit
    double norm;  // teacher_lse, where given
};

// The thread's entry, and then (gather) the student's logit at it. Issued
// before the row's own loads: loads return in order, so waiting for these then
// waits for nothing else.
__device__ __forceinline__ ListFetch fetch_list(const DistillArgs& a, long row, Entry& mine) {
    const int tid = threadIdx.x;
    ListFetch f{a.temperature[row], 0.0f, a.teacher_lse ? a.teacher_lse[row] : 0.0};
    mine = Entry{-1, 0.0f, 0.0};
    if (tid < a.top_k) {
        mine.id = a.ids[row * a.top_k + tid];
        f.y = a.teacher[row * a.top_k + tid];
    }
    return f;
}

template <int DT>
__device__ __forceinline__ void gather(const DistillArgs& a, const RowGroups<DT>& r, Entry& mine) {
    if (mine.id >= 0 && mine.id < a.vocab)
        mine.x = r.at(mine.id);
}

// With e_j = exp(y_j - m): over the list (teacher_lse NULL, m its largest y)
// p_j = e_j / S and log p_j = y_j - m - log S, S = sum e; so sum p (log p - x)
// = T / S - log S with T = sum e (y - m - x): S and T in one exchange. With
// the teacher's own normaliser as m, p = e, P = S and the sum is T.
__device__ inline RowList reduce_list(const DistillArgs& a, const ListFetch& f, Entry& mine, ListLds& lds) {
    const int tid = threadIdx.x, wid = tid >> 6;
    const float inf = __builtin_huge_valf();
    RowList out{};
    const bool t_ok = temperature_mode(f.t, &out.inv_t) == 1;
    const bool used = mine.id >= 0;
    const float y = used ? f.y * out.inv_t : -inf;
    // The student's logit has to be here before anybody writes the gradient,
    // which may take the logits' place.
    asm volatile("" : "+v"(mine.x));
    mine.x *= out.inv_t;
    const bool holds = wid * 64 < a.top_k;  // the wavefront holds part of the list
    if (holds) {
        const bool any_used = __ballot(used) != 0, any_out = __ballot(used && mine.id >= a.vocab) != 0,
                   any_mass = __ballot(used && !(y == -inf)) != 0;
        const float m = wave_max(y);
        if ((tid & 63) == 0) {
            lds.most[wid] = m;
            lds.flags[wid] = (any_used ? 1 : 0) | (any_out ? 2 : 0) | (any_mass ? 4 : 0);
        }
    } else if (tid % 64 == 0 && tid < SPEC_DISTILL_MAX_K) {
        lds.most[wid] = -inf;
        lds.flags[wid] = 0;
        lds.sum[wid] = lds.inner[wid] = 0.0;
    }
    lds_barrier();
    const int flags = lds.flags[0] | lds.flags[1] | lds.flags[2] | lds.flags[3];
    const bool own_norm = a.teacher_lse != nullptr;
    out.bad = !t_ok || (flags & 2);
    out.empty = !(flags & 1) || (!out.bad && !own_norm && !(flags & 4));
    const double m = own_norm ? f.norm
                              : static_cast<double>(fmaxf(fmaxf(lds.most[0], lds.most[1]),
                                                          fmaxf(lds.most[2], lds.most[3])));
    double e = 0.0;
    if (holds) {
        double t = 0.0;
        if (used) {
            const double d = static_cast<double>(y) - m;
            e = exp(d);
            if (!(e == 0.0))
                t = e * (d - static_cast<double>(mine.x));
        }
        const double s = wave_sum(e), w = wave_sum(t);
        if ((tid & 63) == 0) {
            lds.sum[wid] = s;
            lds.inner[wid] = w;
        }
    }
    lds_barrier();
    const double s = (lds.sum[0] + lds.sum[1]) + (lds.sum[2] + lds.sum[3]);
    const double t = (lds.inner[0] + lds.inner[1]) + (lds.inner[2] + lds.inner[3]);
    out.bad = out.bad || !is_finite_f64(m) || !is_finite_f64(s);
    out.mass = own_norm ? s : 1.0;
    out.inner = own_norm ? t : t / s - log(s);
    mine.p = own_norm ? e : e / s;
    if (tid < a.top_k) {
        lds.id[tid] = mine.id;
        lds.p[tid] = mine.p;
    }
    return out;
}

// ---------------------------------------------------------- the normaliser ---

// Running (ref, s) of a thread, s = sum 2^(x log2e - ref): a batch is summed
// against the current reference, and only where that passes 2^8 a group the
// reference is moved to the batch's maximum first. Terms then stay within 2^8
// of 1, so the rounding of their exponents grows by at most 8 steps of 2^-24.
// All of that holds while the reference, a rounded x log2e, is within a fraction
// of the product: within 2^-2 below 2^22. References start at -2^22 or above, so
// that what lies below adds nothing, and a row whose own largest entry lies
// outside (in_reach) is summed by far_row instead.
constexpr float kLazy = 256.0f;
constexpr float kReach = 4194304.0f;

template <int DT>
__device__ inline float group_sum(const uint4& q, float inv_t, float ref) {
    constexpr int W = RowGroups<DT>::W;
    float z[W], t[W];
    RowGroups<DT>::unpack(q, z);
#pragma unroll
    for (int e = 0; e < W; ++e)
        t[e] = fast_exp2(__builtin_fmaf(scale_logit(z[e], inv_t), kLog2e, -ref));
#pragma unroll
    for (int n = W / 2; n > 0; n >>= 1)
#pragma unroll
        for (int e = 0; e < n; ++e)
            t[e] += t[e + n];
    return t[0];
}

template <int DT>
__device__ inline float group_max(const uint4& q) {
    constexpr int W = RowGroups<DT>::W;
    float z[W];
    RowGroups<DT>::unpack(q, z);
    float m = z[0];
#pragma unroll
    for (int e = 1; e < W; ++e)
        m = fmaxf(m, z[e]);
    return m;
}

template <int DT>
__device__ __forceinline__ void online_add(const uint4& q, float inv_t, float& ref, double& s) {
    float g = group_sum<DT>(q, inv_t, ref);
    if (!(g <= kLazy)) {
        const float next = fmaxf(ref, scale_logit(group_max<DT>(q), inv_t) * kLog2e);
        s *= static_cast<double>(fast_exp2(ref - next));
        ref = next;
        g = group_sum<DT>(q, inv_t, ref);
    }
    s += static_cast<double>(g);
}

// The first reference: the wavefront's largest entry of its first groups, or
// the least one allowed where those hold nothing above it.
template <int DT>
__device__ __forceinline__ float first_reference(const uint4& q, float inv_t) {
    return fmaxf(-kReach, scale_logit(wave_max(group_max<DT>(q)), inv_t) * kLog2e);
}

// The threads' pairs joined in two steps, lds holding a (reference, sum) for each
// wavefront in between: what a row's end looks at decides how much of the second
// step each wavefront does.
template <int WAVES>
__device__ inline void join_waves(float ref, double s, double* lds) {
    const float m = wave_max(ref);
    s = wave_sum(s * static_cast<double>(ref == m ? 1.0f : fast_exp2(ref - m)));
    if ((threadIdx.x & 63) == 0) {
        lds[2 * (threadIdx.x >> 6)] = static_cast<double>(m);
        lds[2 * (threadIdx.x >> 6) + 1] = s;
    }
    lds_barrier();
}

// Whether the sums hold, before they are joined: a reference above the least one
// is an entry of its own wavefront, whose term is then within 2^-2 of 1 in the
// exponent; where all are the least one, a sum says whether entries lie close
// enough. A NaN fails. For a pass that needs the row's sum in one thread: with the
// sum itself in a condition of the workgroup all 16 wavefronts would form it (0.5 us
// of a row of 20011 floats).
template <int WAVES>
__device__ inline bool in_reach(const double* lds) {
    const double* pair = lds + 2 * (threadIdx.x % WAVES);
    const bool fits = pair[0] <= static_cast<double>(kReach) && is_finite_f64(pair[1]);
    const bool some = pair[0] > -static_cast<double>(kReach) || pair[1] >= 0.25;
    return __ballot(!fits) == 0 && __ballot(some) != 0;
}

// The same of the joined sum: nothing but a reference in reach with a sum of at
// least its own term gives such a value. The same in every thread, and made so for
// the compiler: a branch of single lanes would keep the row's registers alive over
// far_row.
__device__ inline bool lse_in_reach(double lse2) {
    return __builtin_amdgcn_readfirstlane(fabs(lse2) <= static_cast<double>(kReach)) != 0;
}

// lse * log2e of the row.
template <int WAVES>
__device__ inline double join(const double* lds) {
    double top = lds[0];
#pragma unroll
    for (int w = 1; w < WAVES; ++w)
        top = fmax(top, lds[2 * w]);
    double sum = 0.0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
        const float d = static_cast<float>(lds[2 * w] - top);
        sum += lds[2 * w + 1] * static_cast<double>(fast_exp2(d));
    }
    return top + log2(sum);
}

// ------------------------------------------------------------ the gradient ---

// The row's coefficients: exp(x - lse) = 2^(x log2e - ref) * 2^(ref - lse log2e),
// the second factor (within 2^-2 in the exponent below kReach) taken into the
// coefficient.
struct GradScale {
    float ref, dense;
    double coef;
};

__device__ inline GradScale grad_scale(float weight, const RowList& l, double lse2) {
    GradScale g;
    g.ref = static_cast<float>(lse2);
    g.coef = static_cast<double>(weight) * static_cast<double>(l.inv_t);
    g.dense = static_cast<float>(g.coef * l.mass * exp2(static_cast<double>(g.ref) - lse2));
    return g;
}

// The dense part's coefficient stays inside binary32, before it is formed (which
// takes registers that this does not). The same in every thread, and made so.
__device__ inline bool coef_in_reach(float weight, const RowList& l) {
    const bool in = fabsf(weight * l.inv_t) * static_cast<float>(l.mass) <= 1e38f;
    return __builtin_amdgcn_readfirstlane(in) != 0;
}

template <int DT>
__device__ __forceinline__ void grad_group(const RowGroups<DT>& r, char* out, int g, bool whole,
                                           const uint4& q, float inv_t, const GradScale& c) {
    constexpr int W = RowGroups<DT>::W;
    float z[W], d[W];
    RowGroups<DT>::unpack(q, z);
#pragma unroll
    for (int e = 0; e < W; ++e)
        d[e] = c.dense * fast_exp2(__builtin_fmaf(scale_logit(z[e], inv_t), kLog2e, -c.ref));
    store_group<DT>(r, out, g, whole, d);
}

// A group wholly inside a row whose gradient has the row's alignment.
template <int DT>
__device__ __forceinline__ void grad_group_inside(const RowGroups<DT>& r, char* out, int g, const uint4& q,
                                                  float inv_t, const GradScale& c) {
    constexpr int W = RowGroups<DT>::W;
    float z[W], d[W];
    RowGroups<DT>::unpack(q, z);
#pragma unroll
    for (int e = 0; e < W; ++e)
        d[e] = c.dense * fast_exp2(__builtin_fmaf(scale_logit(z[e], inv_t), kLog2e, -c.ref));
    reinterpret_cast<u32x4*>(out - r.shift * RowGroups<DT>::ESZ)[g] = pack_group<DT>(d);
}

// The listed places, after the dense part: the first entry of an id writes the
// sum over all entries of that id. q: the student's probability at the thread's
// own entry.
template <int DT>
__device__ inline void grad_list(const DistillArgs& a, const RowList& l, const Entry& mine,
                                 const ListLds& lds, double q, double coef, char* out) {
    double sum = 0.0;
    bool first = true;
    for (int j = 0; j < a.top_k; ++j) {
        if (lds.id[j] == mine.id) {
            sum += lds.p[j];
            first = first && j >= static_cast<int>(threadIdx.x);
        }
    }
    if (first)
        store_element<DT>(out, mine.id, static_cast<float>(coef * (l.mass * q - sum)));
}

template <int DT>
__device__ inline char* grad_row(const DistillArgs& a, long row, const RowGroups<DT>& r, bool* whole) {
    char* out = static_cast<char*>(a.out_grad) + row * static_cast<long>(a.vocab) * RowGroups<DT>::ESZ;
    *whole = (reinterpret_cast<uintptr_t>(out) & 15) == static_cast<uintptr_t>(r.shift) * RowGroups<DT>::ESZ;
    return out;
}

// ---------------------------------------------------------------- far rows ---

// The largest, or the sum, of all threads' values, the same in every thread.
template <int THREADS, bool MAX>
__device__ inline double over_workgroup(double v, double* lds) {
    // The lane's number under another name: exchange addresses that the wavefront
    // sums above could share would stay in registers over the whole kernel.
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) {
        const int2 b = __builtin_bit_cast(int2, v);
        const int at = (lane ^ off) * 4;
        const double o = __builtin_bit_cast(
            double, make_int2(__builtin_amdgcn_ds_bpermute(at, b.x), __builtin_amdgcn_ds_bpermute(at, b.y)));
        v = MAX ? fmax(v, o) : v + o;
    }
    __syncthreads();
    if ((threadIdx.x & 63) == 0)
        lds[threadIdx.x >> 6] = v;
    __syncthreads();
    v = lds[0];
#pragma unroll
    for (int w = 1; w < THREADS / 64; ++w)
        v = MAX ? fmax(v, lds[w]) : v + lds[w];
    return v;
}

// A row whose largest scaled logit M lies so far out (a row masked with a large
// finite constant) that M log2e has no digits left for the sum, or whose weight *
// P / T is past binary32: everything is taken against M itself, and M and
// log S = log sum exp(x - M) stay apart,
//   q_v = exp(x_v - M) / S, loss = sum_j p_j (log p_j - (x_j - M)) + P log S,
// one element at a time, by one workgroup, from memory: such rows are rare (128256
// bf16: one row 52 us forward, 126 in one call; 640 rows 260 and 840). Every thread of
// the workgroup calls this, after reduce_list and before anything of the row's
// gradient is written.
template <int DT, int THREADS, bool LOSS, bool GRAD>
__device__ inline void far_row(const DistillArgs& a, long row, const RowGroups<DT>& r, const RowList& l,
                               const Entry& mine, const ListLds& list, double* lds, char* out) {
    const int tid = threadIdx.x;
    const float inf = __builtin_huge_valf(), nan = __builtin_nanf("");
    float m = -inf;
    bool wild = false;  // a NaN, or infinite above
    for (long v = tid; v < r.vocab; v += THREADS) {
        const float x = scale_logit(r.at(v), l.inv_t);
        wild = wild || !(x < inf);
        m = fmaxf(m, x);
    }
    const double top = over_workgroup<THREADS, true>(static_cast<double>(wild ? inf : m), lds);
    m = static_cast<float>(top);
    if (!is_finite_f64(top)) {
        if (LOSS && tid == 0) {
            a.out_loss[row] = nan;
            a.out_lse[row] = static_cast<double>(nan);
        }
        if (GRAD)
            for (long v = tid; v < r.vocab; v += THREADS)
                store_element<DT>(out, v, nan);
        return;
    }
    // exp(x - M); its second term keeps log2e's own rounding out of it
    auto term = [&](long v) {
        const float t = scale_logit(r.at(v), l.inv_t) - m;
        return fast_exp2(__builtin_fmaf(t, kLog2e, t * kLog2eLow));
    };
    double s = 0.0;
    for (long v = tid; v < r.vocab; v += THREADS)
        s += static_cast<double>(term(v));
    s = over_workgroup<THREADS, false>(s, lds);
    if (LOSS) {
        double t = 0.0;
        const double p = mine.id >= 0 ? list.p[tid] : 0.0;
        if (p > 0.0)
            t = p * (log(p) - (static_cast<double>(mine.x) - top));
        t = over_workgroup<THREADS, false>(t, lds);
        const double log_s = log(s);
        if (tid == 0) {
            a.out_loss[row] = static_cast<float>(t + l.mass * log_s);
            a.out_lse[row] = top + log_s;
        }
    }
    if (GRAD) {
        const double coef = static_cast<double>(a.weight[row]) * static_cast<double>(l.inv_t);
        const double dense = coef * l.mass / s;
        for (long v = tid; v < r.vocab; v += THREADS)
            store_element<DT>(out, v, static_cast<float>(dense * static_cast<double>(term(v))));
        __syncthreads();  // the dense part is written
        if (mine.id >= 0)
            grad_list<DT>(a, l, mine, list, exp(static_cast<double>(mine.x) - top) / s, coef, out);
    }
}

// ----------------------------------------------------------------- kernels ---

// One workgroup per row, bound by the read of the logits (640 rows of 128256 bf16:
// 33 us, 4.9 TB/s, 2.5 rows per CU). Few rows take 1024 threads each, for more loads
// in flight; many take 512, so that one row's reductions hide behind another's
// loads (1024 threads, 256, or 8 groups per thread at a time cost 8 to 16 us
// more). 37 rows of 20011 floats: 7.7 us, latency. A row is one workgroup's however
// few there are: 1 to 128 rows of 152064 bf16 take 14 to 17 us.
template <int DT, int THREADS, int U>
__global__ __launch_bounds__(THREADS) void distill_forward_kernel(DistillArgs a) {
    using Row = RowGroups<DT>;
    __shared__ ListLds list;
    __shared__ double lds[2 * THREADS / 64];
    const int tid = threadIdx.x;
    const long row = blockIdx.x;
    const Row r(row_ptr(a.logits, DT, row, a.vocab), a.vocab);
    Entry mine;
    const ListFetch f = fetch_list(a, row, mine);
    gather<DT>(a, r, mine);
    uint4 q[U];
    r.template load<U, THREADS, true>(0, tid, r.groups, q);
    const RowList l = reduce_list(a, f, mine, list);
    const float nan = __builtin_nanf("");
    if (l.empty || l.bad) {
        if (tid == 0) {
            a.out_loss[row] = l.empty ? 0.0f : nan;
            a.out_lse[row] = static_cast<double>(nan);
        }
        return;
    }
    float ref = first_reference<DT>(q[0], l.inv_t);
    double s = 0.0;
    for (int g0 = 0;;) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            online_add<DT>(q[u], l.inv_t, ref, s);
        g0 += U * THREADS;
        if (g0 >= r.groups)
            break;
        r.template load<U, THREADS>(g0, tid, r.groups, q);
    }
    join_waves<THREADS / 64>(ref, s, lds);
    if (!in_reach<THREADS / 64>(lds)) {
        far_row<DT, THREADS, true, false>(a, row, r, l, mine, list, lds, nullptr);
        return;
    }
    const double lse = join<THREADS / 64>(lds) / static_cast<double>(kLog2e);
    if (tid == 0) {
        a.out_loss[row] = static_cast<float>(l.inner + l.mass * lse);
        a.out_lse[row] = lse;
    }
}

// Every element is read, scaled and written once: bound by those two streams (640
// rows of 128256 bf16: 61 us, 5.4 TB/s; the backward pass cannot keep what the
// forward pass read). Each workgroup reduces the row's list (at most 256 entries)
// for itself while its part of the row is on its way.
template <int DT, int THREADS, int U>
__global__ __launch_bounds__(THREADS) void distill_backward_kernel(DistillArgs a, int splits, int per_split) {
    using Row = RowGroups<DT>;
    __shared__ ListLds list;
    __shared__ double lds[THREADS / 64];
    const int tid = threadIdx.x;
    const long row = blockIdx.x / static_cast<unsigned>(splits);
    const int part = static_cast<int>(blockIdx.x % static_cast<unsigned>(splits));
    const Row r(row_ptr(a.logits, DT, row, a.vocab), a.vocab);
    const int g0 = min(part * per_split, r.groups);
    const int g1 = min(g0 + per_split, r.groups);
    bool whole;
    char* out = grad_row<DT>(a, row, r, &whole);
    Entry mine;
    const ListFetch f = fetch_list(a, row, mine);
    const double lse = a.lse_in[row];
    const float weight = a.weight[row];
    gather<DT>(a, r, mine);
    uint4 q[U];
    r.template load<U, THREADS>(g0, tid, g1, q);
    const RowList l = reduce_list(a, f, mine, list);
    if (l.empty || l.bad || !is_finite_f64(lse)) {
        fill<DT, THREADS>(r, out, g0, g1, whole, l.empty ? 0.0f : __builtin_nanf(""));
        return;
    }
    const double lse2 = lse * static_cast<double>(kLog2e);
    const GradScale c = grad_scale(weight, l, lse2);
    // The normaliser has lost its logarithm of the sum, or soon will have: formed
    // again, by one workgroup for the whole row (which may be its own gradient). So
    // is a row whose coefficient binary32 does not hold.
    if (!lse_in_reach(lse2) || !is_finite_f32(c.dense)) {
        if (part == 0)
            far_row<DT, THREADS, false, true>(a, row, r, l, mine, list, lds, out);
        return;
    }
    for (int g = g0;;) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (g + tid + u * THREADS < g1)
                grad_group<DT>(r, out, g + tid + u * THREADS, whole, q[u], l.inv_t, c);
        g += U * THREADS;
        if (g >= g1)
            break;
        r.template load<U, THREADS>(g, tid, g1, q);
    }
    __syncthreads();  // the dense part is written
    if (mine.id >= 0) {
        const long at = r.group_of(mine.id);
        if (at >= g0 && at < g1)
            grad_list<DT>(a, l, mine, list, exp(static_cast<double>(mine.x) - lse), c.coef, out);
    }
}

// The row's first R * THREADS groups stay in registers; those behind them
// (TAIL), kTailUnroll per thread at a time, are read again for the gradient.
// 2304 rows of 152064 bf16 (1.4 GB read and written): 340-355 us, 4.0-4.1 TB/s; a
// copy with one workgroup per row takes 267 us, one along a single front 217, and
// the two passes above, which read the row twice, 345 (110 and 235; in chunks of 420
// rows, whose second read may come from the last-level cache, 445). What is left over
// the copy is a row's own order: its first gradient waits for its last logit, and
// with 304 KB of a CU's 512 KB of registers in one row there is no second workgroup
// to cover for the wait; the 160 KB of LDS hold no part of a row so far. 1024 rows
// of 128256 floats, 40 % of each read again: 260 us, the two passes 258. Few long
// rows are one workgroup each: 1 to 64 rows of 152064 bf16 32-35 us, where the two
// passes, the second of them split, take 24-30. (Workgroups
// that stay for several rows and load the next row's groups as the gradients free
// their registers: 339-381 us; 16 groups in registers and the rest read again, which
// fits twice on a CU: 390; 20 groups so: 385; 1024 threads of 10 and the rest read
// again: 419; 1024 threads of 19 groups spill.)
constexpr int kTailUnroll = 4;

template <int DT, int THREADS, int R, bool TAIL>
__global__ __launch_bounds__(THREADS) void distill_loss_grad_kernel(DistillArgs a) {
    using Row = RowGroups<DT>;
    __shared__ ListLds list;
    __shared__ double lds[2 * THREADS / 64];
    const int tid = threadIdx.x;
    const long row = blockIdx.x;
    const Row r(row_ptr(a.logits, DT, row, a.vocab), a.vocab);
    bool whole;
    char* out = grad_row<DT>(a, row, r, &whole);
    Entry mine;
    const ListFetch f = fetch_list(a, row, mine);
    const float weight = a.weight[row];
    gather<DT>(a, r, mine);
    uint4 q[R];
    r.template load<R, THREADS, true>(0, tid, r.groups, q);
    const RowList l = reduce_list(a, f, mine, list);
    const float nan = __builtin_nanf("");
    float ref = -kReach;
    double s = 0.0;
    if (!l.empty && !l.bad) {
        ref = first_reference<DT>(q[0], l.inv_t);
#pragma unroll
        for (int u = 0; u < R; ++u)
            online_add<DT>(q[u], l.inv_t, ref, s);
        if constexpr (TAIL)
            for (int g0 = R * THREADS; g0 < r.groups; g0 += kTailUnroll * THREADS) {
                uint4 t[kTailUnroll];
                r.template load<kTailUnroll, THREADS>(g0, tid, r.groups, t);
#pragma unroll
                for (int u = 0; u < kTailUnroll; ++u)
                    online_add<DT>(t[u], l.inv_t, ref, s);
            }
    }
    join_waves<THREADS / 64>(ref, s, lds);
    const double lse2 = join<THREADS / 64>(lds);
    const double lse = lse2 / static_cast<double>(kLog2e);
    const bool none = l.empty || l.bad;
    const bool far = !none && (!lse_in_reach(lse2) || !coef_in_reach(weight, l));
    if (tid == 0 && !far) {
        a.out_loss[row] = l.empty ? 0.0f : l.bad ? nan : static_cast<float>(l.inner + l.mass * lse);
        a.out_lse[row] = none ? static_cast<double>(nan) : lse;
    }
    if (none || far) {
        if (far)
            far_row<DT, THREADS, true, true>(a, row, r, l, mine, list, lds, out);
        else
            fill<DT, THREADS>(r, out, 0, r.groups, whole, l.empty ? 0.0f : nan);
        return;
    }
    const GradScale c = grad_scale(weight, l, lse2);
    // Steps that lie wholly inside the row go out as 16-byte stores from
    // registers; the others, at the row's ends (or of a gradient that is
    // aligned otherwise than its row), are read again.
    auto from_registers = [&](int u) {
        return whole && u < R && u * THREADS >= r.full0 && (u + 1) * THREADS <= r.full1;
    };
#pragma unroll
    for (int u = 0; u < R; ++u)
        if (from_registers(u))
            grad_group_inside<DT>(r, out, tid + u * THREADS, q[u], l.inv_t, c);
    const int steps = (r.groups + THREADS - 1) / THREADS;
#pragma unroll 1
    for (int u = 0; u < steps; ++u) {
        const int g = tid + u * THREADS;
        if (!from_registers(u) && g < r.groups)
            grad_group<DT>(r, out, g, whole, r.load_any(g, r.groups), l.inv_t, c);
    }
    __syncthreads();  // the dense part is written
    if (mine.id >= 0)
        grad_list<DT>(a, l, mine, list, exp(static_cast<double>(mine.x) - lse), c.coef, out);
}

template <int DT>
void launch_forward(int rows, const DistillArgs& a, hipStream_t s) {
    if (rows <= 256)
        distill_forward_kernel<DT, 1024, 4><<<dim3(rows), dim3(1024), 0, s>>>(a);
    else
        distill_forward_kernel<DT, 512, 4><<<dim3(rows), dim3(512), 0, s>>>(a);
}

template <int DT>
void launch_backward(int rows, const DistillArgs& a, hipStream_t s) {
    // One step of a workgroup's loads per split: workgroups follow the rows, so
    // that together they read and write one advancing front. Both passes of 640
    // rows of 128256 bf16: 5 to 7 groups a thread 93 us, 4 96 us, 8 95 us, two steps
    // of 4 96 us, 2048 workgroups with longer splits 100 us (shorter steps reduce
    // the list more often, longer ones leave fewer workgroups to cover for it).
    constexpr int kT = 256, kU = 5;
    const long groups = static_cast<long>(a.vocab) / RowGroups<DT>::W + 2;  // at any alignment
    const long steps = (groups + kT * kU - 1) / (kT * kU);
    const long most = ((1L << 32) / kT - 1) / rows;  // of one dispatch
    const long per = (steps + most - 1) / most * (kT * kU);
    const long splits = (groups + per - 1) / per;
    distill_backward_kernel<DT, kT, kU><<<dim3(static_cast<unsigned>(rows * splits)), dim3(kT), 0, s>>>(
        a, static_cast<int>(splits), static_cast<int>(per));
}

template <int DT>
void launch_loss_grad(int rows, const DistillArgs& a, hipStream_t s) {
    // The smallest size that holds the row; the largest is what the registers hold
    // (38 groups take 152 of a thread's 256, beside about 48 others), the others leave
    // room for more workgroups on the CU. At any alignment of the row's start:
    const long groups = (static_cast<long>(a.vocab) + RowGroups<DT>::W - 1) / RowGroups<DT>::W + 1;
#define SPEC_RESIDENT(T, R)                                                                \
    if (groups <= (T) * (R)) {                                                             \
        distill_loss_grad_kernel<DT, T, R, false><<<dim3(rows), dim3(T), 0, s>>>(a);       \
        return;                                                                            \
    }
    SPEC_RESIDENT(256, 4)
    SPEC_RESIDENT(256, 8)
    SPEC_RESIDENT(256, 16)
    SPEC_RESIDENT(512, 16)
    SPEC_RESIDENT(512, 24)
    SPEC_RESIDENT(512, 38)
#undef SPEC_RESIDENT
    distill_loss_grad_kernel<DT, 512, 38, true><<<dim3(rows), dim3(512), 0, s>>>(a);
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

template <bool LOSS, bool GRAD>
int run(int rows, int dtype, const DistillArgs& a, void* hip_stream) {
    if (rows < 0 || a.vocab < 1 || (dtype != SPEC_F32 && dtype != SPEC_BF16) || a.top_k < 1 ||
        a.top_k > SPEC_DISTILL_MAX_K || rows >= (1L << 32) / 1024)
        return SPEC_EINVAL;
    if (rows == 0)
        return SPEC_OK;
    const size_t esz = dtype == SPEC_BF16 ? 2 : 4;
    if (!a.logits || !a.ids || !a.teacher || !a.temperature || !aligned(a.logits, esz) ||
        !aligned(a.ids, 4) || !aligned(a.teacher, 4) || !aligned(a.temperature, 4) ||
        (a.teacher_lse && !aligned(a.teacher_lse, 8)))
        return SPEC_EINVAL;
    if (LOSS && (!a.out_loss || !a.out_lse || !aligned(a.out_loss, 4) || !aligned(a.out_lse, 8)))
        return SPEC_EINVAL;
    if (!LOSS && (!a.lse_in || !aligned(a.lse_in, 8)))
        return SPEC_EINVAL;
    if (GRAD && (!a.weight || !a.out_grad || !aligned(a.weight, 4) || !aligned(a.out_grad, esz)))
        return SPEC_EINVAL;
    if (GRAD && a.out_grad != a.logits) {
        const uintptr_t x = reinterpret_cast<uintptr_t>(a.logits), y = reinterpret_cast<uintptr_t>(a.out_grad);
        const uintptr_t n = static_cast<uintptr_t>(rows) * a.vocab * esz;
        if (x < y + n && y < x + n)
            return SPEC_EINVAL;
    }
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    const bool bf16 = dtype == SPEC_BF16;
    if (LOSS && GRAD)
        bf16 ? launch_loss_grad<kBF16>(rows, a, s) : launch_loss_grad<kF32>(rows, a, s);
    else if (LOSS)
        bf16 ? launch_forward<kBF16>(rows, a, s) : launch_forward<kF32>(rows, a, s);
    else
        bf16 ? launch_backward<kBF16>(rows, a, s) : launch_backward<kF32>(rows, a, s);
    return hipGetLastError() == hipSuccess ? SPEC_OK : SPEC_EHIP;
}

}  // namespace
}  // namespace specv

extern "C" {

int spec_distill_forward(int rows, int vocab, int dtype, int top_k, const void* logits,
                         const int32_t* ids, const float* teacher, const double* teacher_lse,
                         const float* temperature, float* out_loss, double* out_lse,
                         void* hip_stream) {
    const specv::DistillArgs a{logits, ids, teacher, teacher_lse, temperature, nullptr, nullptr,
                               out_loss, out_lse, nullptr, vocab, top_k};
    return specv::run<true, false>(rows, dtype, a, hip_stream);
}

int spec_distill_backward(int rows, int vocab, int dtype, int top_k, const void* logits,
                          const int32_t* ids, const float* teacher, const double* teacher_lse,
                          const float* temperature, const double* lse, const float* weight,
                          void* out_grad, void* hip_stream) {
    const specv::DistillArgs a{logits, ids, teacher, teacher_lse, temperature, lse, weight,
                               nullptr, nullptr, out_grad, vocab, top_k};
    return specv::run<false, true>(rows, dtype, a, hip_stream);
}

int spec_distill_loss_grad(int rows, int vocab, int dtype, int top_k, const void* logits,
                           const int32_t* ids, const float* teacher, const double* teacher_lse,
                           const float* temperature, const float* weight, float* out_loss,
                           double* out_lse, void* out_grad, void* hip_stream) {
    const specv::DistillArgs a{logits, ids, teacher, teacher_lse, temperature, nullptr, weight,
                               out_loss, out_lse, out_grad, vocab, top_k};
    return specv::run<true, true>(rows, dtype, a, hip_stream);
}

}  // extern "C"
