// Beam selection over beams and vocabulary, and the reordering of the beams'
// states (spec_beam.h).
//
//   value(w, v) = score[w] + (z[w][v] - lse[w]), the K best of W * V.
//
// Within a beam the value never falls with the logit, so a beam's part of the
// answer is among the K first of its row in the order (larger z, lower v), and
// that order is the order of one 64-bit integer, (ordered bits of z) << 32 |
// ~v. Two kernels:
//   beam_piece: one workgroup per piece of a row; the piece stays in registers
//     while its K largest keys are found, so the logits are read once;
//   beam_merge: one workgroup per sequence; forms the binary64 values of the
//     pieces' keys and keeps the K best over the beams.
// Both narrow by a bar that at least K entries reach and few more do (from the
// threads' largest entries, and from a histogram of the values), collect what
// reaches it in LDS, and rank the collected entries by counting. Collected in any
// order, ranked by a total order: the result does not depend on timing.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <new>

#include "rows.hpp"
#include "spec_beam.h"

namespace specv {
namespace {

constexpr int kPieceUnroll = 8;  // 16-byte groups of a piece per thread
constexpr int kCollect = 256;    // collected entries: one per thread when ranked

struct NormPart {
    float m;  // the piece's largest finite logit (-inf: none)
    int pad;
    double s;  // sum of exp(z - m)  (m = 0 when there is none)
};

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

// The K largest keys of piece p of row `row`, largest first, 0 where the piece
// has fewer candidates; with NORM also the piece's part of the normaliser.
//
// 256 threads of eight 16-byte groups: 32 KiB of a row in 32 registers a thread,
// enough workgroups per CU to load while others select. Bound by the read of the
// logits (256 x 8 beams of 152064 bf16, K = 8: 83 us, 7.5 TB/s, part of it from the
// last-level cache; 4 groups 99 us, 12 90 us; 64 x 16 beams of 128256, K = 32: 38
// us, 6.8 TB/s). Forming the normalisers takes an exponential for each entry beside
// that: 120 and 56 us. Small calls are a chain of latencies (4 beams of 32000 floats:
// 6 us).
template <int DT, int T, int U, bool NORM>
__global__ __launch_bounds__(T) void beam_piece_kernel(
    const void* __restrict__ logits, const float* __restrict__ score,
    const double* __restrict__ lse, int vocab, int keep, int pieces, int per_piece,
    uint64_t* __restrict__ keys, NormPart* __restrict__ norm) {
    using Row = RowGroups<DT>;
    constexpr int W = Row::W;
    const long row = blockIdx.x / static_cast<unsigned>(pieces);
    const int p = static_cast<int>(blockIdx.x % static_cast<unsigned>(pieces));
    uint64_t* out = keys + (row * pieces + p) * keep;
    const int tid = threadIdx.x;

    const float sc = score[row];
    if (!is_finite_f32(sc) || (!NORM && !is_finite_f64(lse[row]))) {
        if (tid < keep)
            out[tid] = 0;
        return;
    }
    const Row r(row_ptr(logits, DT, row, vocab), vocab);
    const int g0 = min(p * per_piece, r.groups);
    const int g1 = min(g0 + per_piece, r.groups);
    uint4 q[U];
    r.template load<U, T>(g0, tid, g1, q);

    __shared__ int bars[T + 1];
    __shared__ uint64_t list[kCollect];
    __shared__ double wave_sums[T / 64];
    __shared__ float wave_most[T / 64];
    __shared__ uint64_t next_bar;
    __shared__ int count;
    if (tid == 0)
        count = 0;

    const float inf = __builtin_huge_valf();
    int most[U];  // the largest of each group, in integer order
    int best = Row::kOrderNegInf;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        most[u] = Row::order_max(q[u]);
        best = max(best, most[u]);
    }
    if (best >= Row::kOrderInf) {  // an infinite logit or a NaN is no candidate
        best = Row::kOrderNegInf;
        repack(q);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float z[W];
            Row::unpack(q[u], z);
            most[u] = Row::kOrderNegInf;
#pragma unroll
            for (int e = 0; e < W; ++e)
                if (is_finite_f32(z[e]))
                    most[u] = max(most[u], Row::order_of(z[e]));
            best = max(best, most[u]);
        }
    }
    const int held = g1 - g0;
    const int bar = bar_of<T, DT == kBF16 ? 16 : 32>(best, keep, held < T ? held : T, bars);

    repack(q);
    if constexpr (NORM) {
        float m = wave_max(Row::from_order(best));
        if ((tid & 63) == 0)
            wave_most[tid >> 6] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < T / 64; ++w)
            m = fmaxf(m, wave_most[w]);
        const float ref = m == -inf ? 0.0f : m;
        double s = 0.0;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float z[W];
            Row::unpack(q[u], z);
            float g = 0.0f;
#pragma unroll
            for (int e = 0; e < W; ++e) {
                const float t = z[e] - ref;
                g += fast_exp2(__builtin_fmaf(t, kLog2e, t * kLog2eLow));
            }
            s += static_cast<double>(g);
        }
        s = wave_sum(s);
        if ((tid & 63) == 0)
            wave_sums[tid >> 6] = s;
        __syncthreads();
        if (tid == 0) {
            s = wave_sums[0];
#pragma unroll
            for (int w = 1; w < T / 64; ++w)
                s += wave_sums[w];
            norm[row * pieces + p] = NormPart{m, 0, s};
        }
    }

    // Collect the entries that reach the bar. If the list overflows (ties at the
    // bar, or a vocabulary whose best entries lie together), the keep-th largest
    // key that did fit is a higher bar, and keys are unique: again with that.
    auto with_zeros = [](int o) { return o == 0 ? -1 : o; };  // a bar at +0 lets -0 through
    int bar_o = with_zeros(max(bar, Row::kOrderNegInf + 1));  // -inf is no candidate
    uint64_t bar_key = 0;
    const int v0 = static_cast<int>(r.element(g0 + tid));
    for (;;) {
        repack(q);
        const float bar_z = Row::from_order(bar_o);
        // Hits are few and lie in different groups of different threads: each thread
        // picks its own next group that has one, so that the wavefront goes round as
        // often as its busiest thread, not once for every group with a hit anywhere.
        unsigned groups = 0;
#pragma unroll
        for (int u = 0; u < U; ++u)
            groups |= most[u] >= bar_o ? 1u << u : 0u;
        while (groups) {
            const int u = __builtin_ctz(groups);
            groups &= groups - 1;
            uint4 g = q[0];
#pragma unroll
            for (int i = 1; i < U; ++i) {
                g.x = u == i ? q[i].x : g.x;
                g.y = u == i ? q[i].y : g.y;
                g.z = u == i ? q[i].z : g.z;
                g.w = u == i ? q[i].w : g.w;
            }
            float z[W];
            Row::unpack(g, z);
            unsigned hits = 0;
#pragma unroll
            for (int e = 0; e < W; ++e)
                hits |= z[e] >= bar_z ? 1u << e : 0u;
            while (hits) {
                const int e = __builtin_ctz(hits);
                hits &= hits - 1;
                float x = z[0];
#pragma unroll
                for (int i = 1; i < W; ++i)
                    x = e == i ? z[i] : x;
                const uint64_t key = make_key(x, v0 + u * T * W + e);
                if (x < inf && key >= bar_key) {
                    const int slot = atomicAdd(&count, 1);
                    if (slot < kCollect)
                        list[slot] = key;
                }
            }
        }
        __syncthreads();
        const int n = count;
        const int held_keys = n < kCollect ? n : kCollect;
        const uint64_t mine = tid < held_keys ? list[tid] : 0;
        int place = kCollect;
        if ((tid & ~63) < held_keys) {  // wavefronts without an entry have nothing to rank
            place = 0;
#pragma unroll 8
            for (int i = 0; i < held_keys; ++i)
                place += list[i] > mine;
        }
        if (n <= kCollect) {
            if (tid < n) {
                if (place < keep)
                    out[place] = mine;
            } else if (tid < keep) {
                out[tid] = 0;
            }
            return;
        }
        if (tid < held_keys && place == keep - 1)
            next_bar = mine;
        __syncthreads();
        bar_key = next_bar;
        bar_o = with_zeros(Row::order_of(key_logit(bar_key)));
        if (tid == 0)
            count = 0;
        __syncthreads();
    }
}

// A candidate of the merge in its total order: value, then the lower beam, then
// the larger key (larger logit, lower token).
struct Cand {
    double value;
    uint64_t key;
    int beam;
};

__device__ inline bool before(const Cand& a, const Cand& b) {
    if (a.value != b.value)
        return a.value > b.value;
    if (a.beam != b.beam)
        return a.beam < b.beam;
    return a.key > b.key;
}

constexpr int kMergeThreads = 512;
constexpr int kMergeWaves = kMergeThreads / 64;
// The merge's bar: entries are counted in bins of 1/32 below the best value, and
// all entries of the bins up to the one that holds the keep-th are collected.
// The last bin holds everything 16 or more below.
constexpr float kBinsPerUnit = 32.0f;
constexpr int kEntryChunk = 8;  // keys a thread has in flight
// A formed normaliser beyond this (a beam masked with a large finite constant) has
// lost too much of its logarithm: its largest logit and the logarithm stay apart.
// Below it binary64's own rounding is 2^-31 at most.
constexpr double kFarNormaliser = 4194304.0;

// The K best of a sequence's beams * pieces * K keys. One workgroup per sequence:
// the keys are few (16 beams x 8 pieces x 32 of 64 sequences: 2 MB beside the logits' 263),
// so its time is the latency of its steps (read, histogram, collect, rank): 5.7 us
// for one sequence, 6.6 us for 256 of 8 beams and K = 8, 11.3 us for the 4096 keys
// above. Up to 4096 keys stay in registers over the steps; more are read again in
// each (40960 of 64 beams, K = 64: 65 us, more than their pieces' 58).
template <bool NORM>
__global__ __launch_bounds__(kMergeThreads) void beam_merge_kernel(
    const float* score /* may be out_score */, const double* __restrict__ lse, int beams, int keep,
    int pieces, const uint64_t* __restrict__ keys, const NormPart* __restrict__ norm,
    int32_t* out_parent, int32_t* out_token, float* out_score, float* out_logq) {
    __shared__ double b_score[SPEC_BEAM_MAX], b_lse[SPEC_BEAM_MAX];
    __shared__ double b_off[NORM ? SPEC_BEAM_MAX : 1];  // taken from a beam's logits first
    __shared__ int alive[SPEC_BEAM_MAX];
    __shared__ int hist[kMergeThreads], wave_total[kMergeWaves], limit;
    __shared__ double wave_best[kMergeWaves];
    __shared__ Cand list[kCollect];
    __shared__ Cand next_bar;
    __shared__ int count;
    const long b = blockIdx.x;
    const int tid = threadIdx.x, lane = tid & 63, wid = tid >> 6;
    const double none = -static_cast<double>(__builtin_huge_valf());
    const int per_beam = pieces * keep, total = beams * per_beam;
    const uint64_t* k_b = keys + b * total;
    // Keys c0 + i * kMergeThreads, 0 past the end.
    struct Chunk {
        uint64_t key[kEntryChunk];
        int beam[kEntryChunk];
        double value[kEntryChunk];  // no candidate: none
    };
    auto load = [&](Chunk& x, int c0) {
#pragma unroll
        for (int i = 0; i < kEntryChunk; ++i) {
            const int c = c0 + i * kMergeThreads;
            x.key[i] = c < total ? k_b[c] : 0;
            x.beam[i] = c < total ? c / per_beam : 0;
        }
    };
    // The first keys are on their way while the beams' scores are read.
    Chunk own;
    load(own, tid);
    if (tid == 0) {
        count = 0;
        limit = kMergeThreads - 1;
    }
    hist[tid] = 0;
    if constexpr (NORM) {
        // 16 lanes to a beam: log sum over its pieces, against the largest
        // piece maximum (a piece without a finite logit has sum 0, NaN or inf)
        for (int w = tid >> 4; w < beams; w += kMergeThreads / 16) {
            const long row = b * beams + w;
            const float sc = score[row];
            const bool ok = is_finite_f32(sc);  // else the pieces were not formed
            const NormPart* part = norm + row * pieces;
            float m = -__builtin_huge_valf();
            for (int p = tid & 15; ok && p < pieces; p += 16)
                m = fmaxf(m, part[p].m);
#pragma unroll
            for (int off = 1; off < 16; off <<= 1)
                m = fmaxf(m, __shfl_xor(m, off, 64));
            double s = 0.0;
            for (int p = tid & 15; ok && p < pieces; p += 16) {
                const NormPart x = part[p];
                s += x.m == -__builtin_huge_valf()
                         ? x.s
                         : x.s * exp(static_cast<double>(x.m) - static_cast<double>(m));
            }
#pragma unroll
            for (int off = 1; off < 16; off <<= 1)
                s += __shfl_xor(s, off, 64);
            if ((tid & 15) == 0) {
                const double log_s = log(s), l = static_cast<double>(m) + log_s;
                const bool far = fabs(l) > kFarNormaliser;
                b_score[w] = static_cast<double>(sc);
                b_off[w] = far ? static_cast<double>(m) : 0.0;
                b_lse[w] = far ? log_s : l;
                alive[w] = ok && is_finite_f64(l);
            }
        }
    } else if (tid < beams) {
        const float sc = score[b * beams + tid];
        const double l = lse[b * beams + tid];
        b_score[tid] = static_cast<double>(sc);
        b_lse[tid] = l;
        alive[tid] = is_finite_f32(sc) && is_finite_f64(l);
    }
    __syncthreads();
    auto logq = [&](uint64_t key, int w) {
        const double z = static_cast<double>(key_logit(key));
        if constexpr (NORM)
            return (z - b_off[w]) - b_lse[w];
        else
            return z - b_lse[w];
    };
    auto values = [&](Chunk& x) {
#pragma unroll
        for (int i = 0; i < kEntryChunk; ++i) {
            const int w = x.beam[i];
            x.value[i] = x.key[i] != 0 && alive[w]
                             ? b_score[w] + logq(x.key[i], w)
                             : none;
        }
    };
    values(own);
    // Every candidate of the sequence: a thread's first kEntryChunk from its
    // registers, any further ones read again each time.
    auto for_each = [&](auto&& f) {
#pragma unroll
        for (int i = 0; i < kEntryChunk; ++i)
            if (own.value[i] > none)
                f(Cand{own.value[i], own.key[i], own.beam[i]});
        for (int c0 = tid + kEntryChunk * kMergeThreads; c0 < total; c0 += kEntryChunk * kMergeThreads) {
            Chunk x;
            load(x, c0);
            values(x);
#pragma unroll
            for (int i = 0; i < kEntryChunk; ++i)
                if (x.value[i] > none)
                    f(Cand{x.value[i], x.key[i], x.beam[i]});
        }
    };
    double best = none;
    for_each([&](const Cand& x) { best = fmax(best, x.value); });
#pragma unroll
    for (int off = 32; off > 0; off >>= 1)
        best = fmax(best, __shfl_xor(best, off, 64));
    if (lane == 0)
        wave_best[wid] = best;
    __syncthreads();
    best = wave_best[0];
#pragma unroll
    for (int w = 1; w < kMergeWaves; ++w)
        best = fmax(best, wave_best[w]);
    auto bin_of = [&](double v) {
        return static_cast<int>(fminf(static_cast<float>(best - v) * kBinsPerUnit,
                                      static_cast<float>(kMergeThreads - 1)));
    };
    for_each([&](const Cand& x) {
        const int bin = bin_of(x.value);
        if (bin < kMergeThreads - 1)  // nobody asks how many the last one holds
            atomicAdd(&hist[bin], 1);
    });
    __syncthreads();
    {
        int upto = hist[tid];
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const int o = __shfl_up(upto, off, 64);
            upto += lane >= off ? o : 0;
        }
        if (lane == 63)
            wave_total[wid] = upto;
        __syncthreads();
        for (int w = 0; w < wid; ++w)
            upto += wave_total[w];
        if (upto >= keep && upto - hist[tid] < keep)
            limit = tid;
        __syncthreads();
    }
    const int last_bin = limit;
    auto emit = [&](int j, const Cand& x, bool some) {
        const long at = b * keep + j;
        out_parent[at] = some ? x.beam : -1;
        out_token[at] = some ? key_token(x.key) : -1;
        out_score[at] = some ? static_cast<float>(x.value) : -__builtin_huge_valf();
        if (out_logq)
            out_logq[at] = some ? static_cast<float>(logq(x.key, x.beam)) : -__builtin_huge_valf();
    };
    Cand bar{none, 0, SPEC_BEAM_MAX};  // behind every candidate
    for (;;) {
        for_each([&](const Cand& x) {
            if (bin_of(x.value) > last_bin || before(bar, x))
                return;
            const int slot = atomicAdd(&count, 1);
            if (slot < kCollect)
                list[slot] = x;
        });
        __syncthreads();
        const int n = count;
        const int held = n < kCollect ? n : kCollect;
        Cand mine{none, 0, SPEC_BEAM_MAX};
        int place = kCollect;
        if (tid - lane < held) {
            if (tid < held)
                mine = list[tid];
            place = 0;
            int same = 0;
#pragma unroll 8
            for (int i = 0; i < held; ++i) {
                const double v = list[i].value;
                place += v > mine.value;
                same += v == mine.value;
            }
            if (same > 1)  // more than itself
                for (int i = 0; i < held; ++i)
                    place += list[i].value == mine.value && before(list[i], mine);
        }
        if (n <= kCollect) {
            if (tid < n) {
                if (place < keep)
                    emit(place, mine, true);
            } else if (tid < keep) {
                emit(tid, mine, false);
            }
            return;
        }
        // Overflow (ties, or a crowded bin): the keep-th best of those that fit
        // is a higher bar, and no two candidates are equal in the order.
        if (tid < held && place == keep - 1)
            next_bar = mine;
        __syncthreads();
        bar = next_bar;
        if (tid == 0)
            count = 0;
        __syncthreads();
    }
}

// ---------------------------------------------------------------- reorder ---

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

// In place: one thread owns one T-sized column of every slot of a (layer,
// sequence), at most NB, and reads the parents' columns before it writes any
// slot, so that a permutation needs no other order. Reads and writes each moved
// slot once; small states are one latency (4 layers x 4 beams of 16 KiB: 3 us), large
// ones move at 5.8-6.0 TB/s of what is moved (8 layers x 32 sequences x 8 beams of 512
// KiB, 1.67 GB: 284 us; 4 x 16 x 64 beams of 256 KiB, 2.07 GB: 355).
template <typename T, int NB>
__global__ __launch_bounds__(kBlock) void beam_reorder_kernel(long states, int batch, int beams,
                                                              const int32_t* __restrict__ parent,
                                                              char* state, long stride, long cols) {
    const long blocks_per = (cols + kBlock - 1) / kBlock;
#pragma unroll 1
    for (long blk = blockIdx.x; blk < states * blocks_per; blk += gridDim.x) {
        const long lb = blk / blocks_per;
        const long col = (blk - lb * blocks_per) * kBlock + threadIdx.x;
        if (col >= cols)
            continue;
        const int32_t* par = parent + (lb % batch) * beams;
        char* s = state + lb * beams * stride + col * static_cast<long>(sizeof(T));
        auto moves = [&](int j, int* w) {
            *w = j < beams ? par[j] : -1;
            return *w >= 0 && *w < beams && *w != j;
        };
        T r[NB] = {};
        int w;
#pragma unroll
        for (int j = 0; j < NB; ++j)
            if (moves(j, &w))
                r[j] = *reinterpret_cast<const T*>(s + w * stride);
#pragma unroll
        for (int j = 0; j < NB; ++j)
            if (moves(j, &w))
                *reinterpret_cast<T*>(s + j * stride) = r[j];
    }
}

// Into another array: a workgroup copies one run of kCopyUnroll * kBlock Ts of a
// slot. Workgroups follow the destination's order, so that together they write
// one advancing front (8 layers x 32 sequences x 8 beams of 512 KiB: 270-280 us,
// 7.8 TB/s counting each slot's read though parents repeat; a workgroup per column
// of all slots 476 us). The destination is not read again here: its stores go past
// the caches (270 us; plain stores 307). Two loads a thread are enough in flight
// (four 281, eight 510).
constexpr int kCopyUnroll = 2;

template <typename T>
__global__ __launch_bounds__(kBlock) void beam_copy_kernel(
    long states, int batch, int beams_in, int beams_out, const int32_t* __restrict__ parent,
    const char* __restrict__ src, long src_stride, char* __restrict__ dst, long dst_stride, long cols,
    long runs) {
#pragma unroll 1
    for (long blk = blockIdx.x; blk < states * beams_out * runs; blk += gridDim.x) {
        const long slot = blk / runs, lb = slot / beams_out;
        const int j = static_cast<int>(slot - lb * beams_out);
        const int w = parent[(lb % batch) * beams_out + j];
        if (w < 0 || w >= beams_in)
            continue;
        const long c0 = (blk - slot * runs) * (kCopyUnroll * kBlock) + threadIdx.x;
        const T* s = reinterpret_cast<const T*>(src + (lb * beams_in + w) * src_stride);
        T* d = reinterpret_cast<T*>(dst + slot * dst_stride);
        T r[kCopyUnroll] = {};
#pragma unroll
        for (int u = 0; u < kCopyUnroll; ++u)
            if (c0 + u * kBlock < cols)
                r[u] = s[c0 + u * kBlock];
#pragma unroll
        for (int u = 0; u < kCopyUnroll; ++u)
            if (c0 + u * kBlock < cols)
                __builtin_nontemporal_store(r[u], d + c0 + u * kBlock);
    }
}

template <typename T>
hipError_t launch_reorder(long states, int batch, int beams_in, int beams_out,
                          const int32_t* parent, const void* src, long src_stride, void* dst,
                          long dst_stride, long bytes, bool in_place, hipStream_t stream) {
    const long cols = bytes / static_cast<long>(sizeof(T));
    const char* s = static_cast<const char*>(src);
    char* d = static_cast<char*>(dst);
    auto grid = [](long blocks) { return dim3(static_cast<unsigned>(blocks < (1L << 23) ? blocks : 1L << 23)); };
    if (!in_place) {
        const long runs = (cols + kCopyUnroll * kBlock - 1) / (kCopyUnroll * kBlock);
        beam_copy_kernel<T><<<grid(states * beams_out * runs), dim3(kBlock), 0, stream>>>(
            states, batch, beams_in, beams_out, parent, s, src_stride, d, dst_stride, cols, runs);
        return hipGetLastError();
    }
    const long blocks = states * ((cols + kBlock - 1) / kBlock);
#define SPEC_REORDER(NB)                                                                  \
    beam_reorder_kernel<T, NB><<<grid(blocks), dim3(kBlock), 0, stream>>>(                \
        states, batch, beams_out, parent, d, dst_stride, cols)
    if (beams_out <= 4)
        SPEC_REORDER(4);
    else if (beams_out <= 16)  // (an instance of 8 takes three times its registers and is slower)
        SPEC_REORDER(16);
    else if (beams_out <= 32)
        SPEC_REORDER(32);
    else
        SPEC_REORDER(64);
#undef SPEC_REORDER
    return hipGetLastError();
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool overlap(const void* a, uint64_t na, const void* b, uint64_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

}  // namespace
}  // namespace specv

using namespace specv;

struct spec_beam_ctx {
    int B = 0, W = 0, K = 0, V = 0, dtype = 0, pieces = 0;
    int per_piece = 0;  // groups of a piece (the last has the rest)
    hipStream_t stream = nullptr;
    int device = 0;
    void* ws = nullptr;
    uint64_t* keys = nullptr;
    NormPart* norm = nullptr;
};

extern "C" {

int spec_beam_init(int batch, int beams, int keep, int vocab, int dtype, void* hip_stream,
                   spec_beam_ctx** out_ctx) {
    if (!out_ctx)
        return SPEC_EINVAL;
    *out_ctx = nullptr;
    if (batch < 1 || beams < 1 || beams > SPEC_BEAM_MAX || keep < 1 || keep > SPEC_BEAM_MAX ||
        vocab < 1 || (dtype != SPEC_F32 && dtype != SPEC_BF16))
        return SPEC_EINVAL;
    // A row holds at most one group more than its elements need (its first
    // and last groups may both hang over).
    const long W = dtype == SPEC_BF16 ? 8 : 4;
    const long groups = (static_cast<long>(vocab) + W - 1) / W + 1;
    const long per_piece = static_cast<long>(kPieceUnroll) * kBlock;
    const long pieces = (groups + per_piece - 1) / per_piece;
    const long rows = static_cast<long>(batch) * beams;
    if (rows * pieces >= (1L << 32) / kBlock || batch >= (1L << 32) / kMergeThreads || static_cast<long>(beams) * pieces * keep >= (1L << 30))
        return SPEC_EINVAL;
    spec_beam_ctx* ctx = new (std::nothrow) spec_beam_ctx();
    if (!ctx)
        return SPEC_ENOMEM;
    ctx->B = batch;
    ctx->W = beams;
    ctx->K = keep;
    ctx->V = vocab;
    ctx->dtype = dtype;
    ctx->pieces = static_cast<int>(pieces);
    ctx->per_piece = static_cast<int>(per_piece);
    ctx->stream = static_cast<hipStream_t>(hip_stream);
    if (hipGetDevice(&ctx->device) != hipSuccess) {
        delete ctx;
        return SPEC_EHIP;
    }
    const size_t key_bytes = static_cast<size_t>(rows) * pieces * keep * sizeof(uint64_t);
    const size_t norm_bytes = static_cast<size_t>(rows) * pieces * sizeof(NormPart);
    if (hipMalloc(&ctx->ws, key_bytes + norm_bytes) != hipSuccess) {
        (void)hipGetLastError();
        delete ctx;
        return SPEC_ENOMEM;
    }
    // 16-byte entries first: the keys behind them stay aligned
    ctx->norm = static_cast<NormPart*>(ctx->ws);
    ctx->keys = reinterpret_cast<uint64_t*>(static_cast<char*>(ctx->ws) + norm_bytes);
    *out_ctx = ctx;
    return SPEC_OK;
}

int spec_beam_set_stream(spec_beam_ctx* ctx, void* hip_stream) {
    if (!ctx)
        return SPEC_EINVAL;
    ctx->stream = static_cast<hipStream_t>(hip_stream);
    return SPEC_OK;
}

int spec_beam_select(spec_beam_ctx* ctx, const void* logits, const float* score,
                     const double* lse, int32_t* out_parent, int32_t* out_token,
                     float* out_score, float* out_logq) {
    if (!ctx || !logits || !score || !out_parent || !out_token || !out_score)
        return SPEC_EINVAL;
    const size_t esz = ctx->dtype == SPEC_BF16 ? 2 : 4;
    if (!aligned(logits, esz) || !aligned(score, 4) || (lse && !aligned(lse, 8)) ||
        !aligned(out_parent, 4) || !aligned(out_token, 4) || !aligned(out_score, 4) ||
        (out_logq && !aligned(out_logq, 4)))
        return SPEC_EINVAL;
    int device = 0;
    if (hipGetDevice(&device) != hipSuccess)
        return SPEC_EHIP;
    if (device != ctx->device)
        return SPEC_ESTATE;
    const dim3 grid(static_cast<unsigned>(static_cast<long>(ctx->B) * ctx->W * ctx->pieces));
    hipStream_t s = ctx->stream;
#define SPEC_PIECE(DT, NORM)                                                                   \
    beam_piece_kernel<DT, kBlock, kPieceUnroll, NORM><<<grid, dim3(kBlock), 0, s>>>(           \
        logits, score, lse, ctx->V, ctx->K, ctx->pieces, ctx->per_piece, ctx->keys, ctx->norm)
    if (ctx->dtype == SPEC_BF16) {
        if (lse)
            SPEC_PIECE(kBF16, false);
        else
            SPEC_PIECE(kBF16, true);
    } else {
        if (lse)
            SPEC_PIECE(kF32, false);
        else
            SPEC_PIECE(kF32, true);
    }
#undef SPEC_PIECE
    if (hipGetLastError() != hipSuccess)
        return SPEC_EHIP;
    const dim3 seqs(static_cast<unsigned>(ctx->B));
    if (lse)
        beam_merge_kernel<false><<<seqs, dim3(kMergeThreads), 0, s>>>(
            score, lse, ctx->W, ctx->K, ctx->pieces, ctx->keys, ctx->norm, out_parent, out_token,
            out_score, out_logq);
    else
        beam_merge_kernel<true><<<seqs, dim3(kMergeThreads), 0, s>>>(
            score, lse, ctx->W, ctx->K, ctx->pieces, ctx->keys, ctx->norm, out_parent, out_token,
            out_score, out_logq);
    return hipGetLastError() == hipSuccess ? SPEC_OK : SPEC_EHIP;
}

int spec_beam_destroy(spec_beam_ctx* ctx) {
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

int spec_beam_reorder(int layers, int batch, int beams_in, int beams_out, const int32_t* parent,
                      const void* src, int64_t src_stride, void* dst, int64_t dst_stride,
                      int64_t bytes, void* hip_stream) {
    if (layers < 0 || batch < 0 || beams_in < 1 || beams_in > SPEC_BEAM_MAX || beams_out < 1 ||
        beams_out > SPEC_BEAM_MAX || bytes < 0 || src_stride < bytes || dst_stride < bytes)
        return SPEC_EINVAL;
    if (layers == 0 || batch == 0 || bytes == 0)
        return SPEC_OK;
    if (!parent || !src || !dst || !aligned(parent, 4))
        return SPEC_EINVAL;
    const long states = static_cast<long>(layers) * batch;
    // Every byte offset has to fit 63 bits.
    if (src_stride > (INT64_MAX / SPEC_BEAM_MAX) / states || dst_stride > (INT64_MAX / SPEC_BEAM_MAX) / states)
        return SPEC_EINVAL;
    const uint64_t src_bytes = static_cast<uint64_t>(states * beams_in - 1) * src_stride + bytes;
    const uint64_t dst_bytes = static_cast<uint64_t>(states * beams_out - 1) * dst_stride + bytes;
    const bool in_place = src == dst && src_stride == dst_stride && beams_in == beams_out;
    if (!in_place && overlap(src, src_bytes, dst, dst_bytes))
        return SPEC_EINVAL;
    const uint64_t parent_bytes = static_cast<uint64_t>(batch) * beams_out * sizeof(int32_t);
    if (overlap(parent, parent_bytes, src, src_bytes) || overlap(parent, parent_bytes, dst, dst_bytes))
        return SPEC_EINVAL;
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    auto fits = [&](int a) {
        return aligned(src, a) && aligned(dst, a) && src_stride % a == 0 && dst_stride % a == 0 &&
               bytes % a == 0;
    };
    hipError_t e;
    if (fits(16))
        e = launch_reorder<u32x4>(states, batch, beams_in, beams_out, parent, src, src_stride, dst,
                                  dst_stride, bytes, in_place, s);
    else if (fits(4))
        e = launch_reorder<uint32_t>(states, batch, beams_in, beams_out, parent, src, src_stride,
                                     dst, dst_stride, bytes, in_place, s);
    else
        e = launch_reorder<uint8_t>(states, batch, beams_in, beams_out, parent, src, src_stride,
                                    dst, dst_stride, bytes, in_place, s);
    return e == hipSuccess ? SPEC_OK : SPEC_EHIP;
}

}  // extern "C"
