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

#include "launch.hpp"
#include "rows.hpp"
#include "select.hpp"
#include "spec_logprobs.h"
#include "stage.hpp"

namespace specv {
namespace {

constexpr int kT = kBlock;     // threads of a workgroup
constexpr int kU = 4;          // 16-byte groups of a step per thread
constexpr int kStep = kT * kU;
constexpr int kCap = 512;      // collected entries: two per thread when ranked

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

// The `keep` largest keys of those offered so far, and some more: keys reach the
// list when they are at least the bar, which is the keep-th largest key at the
// time the list was last ranked. Every thread calls every function; what is kept
// does not depend on the order in which keys arrive.
struct SelectionLds {
    uint64_t list[kCap];
    uint64_t bar;
    int counts[3];  // keys offered in a round; rounds take turns
};

struct Selection {
    SelectionLds& lds;
    int keep;
    int n = 0;         // keys in the list, the same in every thread
    int round = 0;
    uint64_t bar = 1;  // 0 marks no candidate

    __device__ Selection(SelectionLds& l, int k) : lds(l), keep(k) {
        if (threadIdx.x < 3)
            lds.counts[threadIdx.x] = 0;
        lds_barrier();
    }

    // f(push) pushes this thread's keys that are at least the bar. Where a round
    // overflows the list, the keep-th largest key that did fit is a higher bar (the
    // list holds more than keep keys of this round, and keys are unique): again with that.
    template <typename F>
    __device__ void offer(F&& f) {
        for (;;) {
            int* count = &lds.counts[round % 3];
            f([&](uint64_t key) {
                const int slot = n + atomicAdd(count, 1);
                if (slot < kCap)
                    lds.list[slot] = key;
            });
            // Of three counters one is written, one may still be read by a thread that
            // has just passed the barrier before, and one is free.
            if (threadIdx.x == 0)
                lds.counts[(round + 1) % 3] = 0;
            lds_barrier();
            const int more = *count;
            ++round;
            if (n + more <= kCap) {
                n += more;
                if (n > 2 * keep + 64)
                    rank();
                return;
            }
            uint64_t mine[2];
            int place[2];
            places(kCap, mine, place);
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (place[i] == keep - 1)
                    lds.bar = mine[i];
            lds_barrier();
            bar = lds.bar;
        }
    }

    // The list becomes its keep largest keys, largest first.
    __device__ void rank() {
        uint64_t mine[2];
        int place[2];
        places(n, mine, place);
        lds_barrier();
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (place[i] < keep)
                lds.list[place[i]] = mine[i];
        lds_barrier();
        if (n >= keep) {
            n = keep;
            bar = lds.list[keep - 1];
        }
    }

    // This thread's keys among the first `held` of the list, and how many of those
    // are larger (kCap where there is none).
    __device__ void places(int held, uint64_t (&mine)[2], int (&place)[2]) const {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int at = static_cast<int>(threadIdx.x) + i * kT;
            mine[i] = at < held ? lds.list[at] : 0;
            place[i] = kCap;
            if ((at & ~63) < held) {  // wavefronts without a key have nothing to rank
                int larger = 0;
#pragma unroll 8
                for (int j = 0; j < held; ++j)
                    larger += lds.list[j] > mine[i];
                if (at < held)
                    place[i] = larger;
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

// (M, S, T) of the same entries against a larger M: T = sum e (x - M).
__device__ inline void move_reference(float from, float to, double& s, double& t) {
    if (from == -__builtin_huge_valf() || from == to)
        return;  // nothing but entries of -inf so far: the sums are 0 (or NaN)
    const float d = from - to;
    const double f = static_cast<double>(fast_exp2(__builtin_fmaf(d, kLog2e, d * kLog2eLow)));
    t = f * (t + s * static_cast<double>(d));
    s *= f;
}

// Joins the threads' parts: in every thread of the first wavefront afterwards.
struct JoinLds {
    float m[kWaves];
    int before[kWaves];
    double s[kWaves], t[kWaves];
};

__device__ inline Part join_threads(Part p, JoinLds& lds) {
    const int wid = threadIdx.x >> 6;
    float m = wave_max(p.m);
    move_reference(p.m, m, p.s, p.t);
    p.s = wave_sum(p.s);
    p.t = wave_sum(p.t);
#pragma unroll
    for (int off = 32; off > 0; off >>= 1)
        p.before += __shfl_xor(p.before, off, 64);
    if ((threadIdx.x & 63) == 0) {
        lds.m[wid] = m;
        lds.before[wid] = p.before;
        lds.s[wid] = p.s;
        lds.t[wid] = p.t;
    }
    lds_barrier();
    m = lds.m[0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w)
        m = fmaxf(m, lds.m[w]);
    Part out{m, 0, 0.0, 0.0};
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        double s = lds.s[w], t = lds.t[w];
        move_reference(lds.m[w], m, s, t);
        out.s += s;
        out.t += t;
        out.before += lds.before[w];
    }
    return out;
}

// The row's outputs, from its sums and its sorted list of n keys (n <= keep).
__device__ inline void write_row(const LogprobsArgs& a, long row, const Part& p, float inv_t, int token,
                                 float z_token, const uint64_t* list, int n) {
    const int tid = threadIdx.x;
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

template <int DT, bool TOP>
__global__ __launch_bounds__(kT) void logprobs_kernel(LogprobsArgs a, int splits, int per_split,
                                                      Part* __restrict__ parts, uint64_t* __restrict__ keys) {
    using Row = RowGroups<DT>;
    constexpr int W = Row::W;
    __shared__ SelectionLds select_lds;
    __shared__ int bars[TOP ? kT + 1 : 1];
    __shared__ JoinLds join_lds;
    const int tid = threadIdx.x;
    const long row = blockIdx.x / static_cast<unsigned>(splits);
    const int part = static_cast<int>(blockIdx.x % static_cast<unsigned>(splits));
    const Row r(row_ptr(a.logits, DT, row, a.vocab), a.vocab);
    const int g0 = min(part * per_split, r.groups);
    const int g1 = min(g0 + per_split, r.groups);
    const int token = a.token[row];
    const float inv_t = row_scale(a.temperature, row);
    uint4 next[kU];
    auto request = [&](int g) {
        if (r.full1 > r.full0) {
#pragma unroll
            for (int u = 0; u < kU; ++u)
                next[u] = r.request(g + tid + u * kT);
        }
    };
    request(g0);
    const bool given = token >= 0 && token < a.vocab;
    const float z_token = given ? r.at(token) : 0.0f;
    // Both zeros are one logit: a token's of +0 is tied by entries of -0.
    const int token_order = given ? Row::order_of(z_token) - (z_token == 0.0f ? 1 : 0) : 0x7FFFFFFF;

    const float inf = __builtin_huge_valf();
    float m = -inf;
    double s = 0.0, t = 0.0;
    int before = 0;
    Selection sel(select_lds, a.keep);
    // In the order of the logits: below it lie none of the K first entries so far.
    int bar_o = Row::kOrderNegInf + 1;  // -inf is no candidate
#pragma unroll 1
    for (int g = g0; g < g1; g += kStep) {
        uint4 q[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u)
            q[u] = next[u];
        r.template settle<kU, kT, false>(g, tid, g1, q);
        if (g + kStep < g1)
            request(g + kStep);

        int most[kU];  // the largest of each group, in integer order
        int best = Row::kOrderNegInf;
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            most[u] = Row::order_max(q[u]);
            best = max(best, most[u]);
        }
        const float x_best = Row::from_order(best) * inv_t;
        if (x_best > m) {
            move_reference(m, x_best, s, t);
            m = x_best;
        }
        const float ref = m == -inf ? 0.0f : m;
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            float z[W], e[W], et[W];
            Row::unpack(q[u], z);
#pragma unroll
            for (int i = 0; i < W; ++i) {
                const float d = scale_logit(z[i], inv_t) - ref;
                e[i] = fast_exp2(d * kLog2e);
                et[i] = e[i] * fmaxf(d, kNegMax);  // 0 at -inf
            }
#pragma unroll
            for (int n = W / 2; n > 0; n >>= 1)
#pragma unroll
                for (int i = 0; i < n; ++i) {
                    e[i] += e[i + n];
                    et[i] += et[i + n];
                }
            s += static_cast<double>(e[0]);
            t += static_cast<double>(et[0]);
        }
        if (best >= token_order) {
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                if (most[u] < token_order || g + tid + u * kT >= g1)
                    continue;
                float z[W];
                Row::unpack(q[u], z);
                const long v0 = r.element(g + tid + u * kT);
#pragma unroll
                for (int i = 0; i < W; ++i)
                    before += z[i] > z_token || (z[i] == z_token && v0 + i < token && v0 + i >= 0);
            }
        }
        if constexpr (TOP) {
            if (g == g0) {
                const int held = g1 - g0;
                bar_o = max(bar_o, bar_of<kT, DT == kBF16 ? 16 : 32>(best, a.keep, held < kT ? held : kT, bars));
            }
            sel.offer([&](auto&& push) {
                if (sel.bar > 1)
                    bar_o = max(bar_o, Row::order_of(key_logit(sel.bar)));
                const int from = bar_o == 0 ? -1 : bar_o;  // a bar at +0 lets -0 through
                const float from_z = Row::from_order(from);
                unsigned groups = 0;
#pragma unroll
                for (int u = 0; u < kU; ++u)
                    groups |= most[u] >= from ? 1u << u : 0u;
                while (groups) {
                    const int u = __builtin_ctz(groups);
                    groups &= groups - 1;
                    uint4 x = q[0];
#pragma unroll
                    for (int i = 1; i < kU; ++i) {
                        x.x = u == i ? q[i].x : x.x;
                        x.y = u == i ? q[i].y : x.y;
                        x.z = u == i ? q[i].z : x.z;
                        x.w = u == i ? q[i].w : x.w;
                    }
                    float z[W];
                    Row::unpack(x, z);
                    const int v0 = static_cast<int>(r.element(g + tid + u * kT));
                    unsigned hits = 0;
#pragma unroll
                    for (int e = 0; e < W; ++e)
                        hits |= z[e] >= from_z ? 1u << e : 0u;
                    while (hits) {
                        const int e = __builtin_ctz(hits);
                        hits &= hits - 1;
                        float y = z[0];
#pragma unroll
                        for (int i = 1; i < W; ++i)
                            y = e == i ? z[i] : y;
                        const uint64_t key = make_key(y, v0 + e);
                        if (key >= sel.bar)
                            push(key);
                    }
                }
            });
        }
    }
    if (TOP)
        sel.rank();
    const Part p = join_threads(Part{m, before, s, t}, join_lds);
    const int n = min(sel.n, a.keep);
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
    __shared__ JoinLds join_lds;
    const int tid = threadIdx.x;
    const long row = blockIdx.x;
    const int token = a.token[row];
    const float inv_t = row_scale(a.temperature, row);
    const RowGroups<DT> r(row_ptr(a.logits, DT, row, a.vocab), a.vocab);
    const float z_token = token >= 0 && token < a.vocab ? r.at(token) : 0.0f;
    Part p{-__builtin_huge_valf(), 0, 0.0, 0.0};
    for (int i = tid; i < splits; i += kT) {
        Part x = parts[row * splits + i];
        const float m = fmaxf(p.m, x.m);
        move_reference(p.m, m, p.s, p.t);
        move_reference(x.m, m, x.s, x.t);
        p = Part{m, p.before + x.before, p.s + x.s, p.t + x.t};
    }
    Selection sel(select_lds, a.keep);
    const int total = splits * a.keep;
    for (int i0 = 0; i0 < total; i0 += kT) {
        const uint64_t key = i0 + tid < total ? keys[row * total + i0 + tid] : 0;
        sel.offer([&](auto&& push) {
            if (key >= sel.bar)
                push(key);
        });
    }
    if (a.keep)
        sel.rank();
    p = join_threads(p, join_lds);
    write_row(a, row, p, inv_t, token, z_token, select_lds.list, min(sel.n, a.keep));
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
    logprobs_kernel<DT, TOP><<<grid, block, 0, s>>>(a, p.splits, p.per_split, ctx->parts, ctx->keys)
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
