// Distillation from a teacher's top logits, forward and backward
// (spec_distill.h).
//
//   loss = sum_j p_j (log p_j - (x_id(j) - lse)),
//   grad_v = weight / T (P exp(x_v - lse) - sum_{j: id(j) = v} p_j).
//
// One workgroup per row. The dense part of the gradient is written first; a
// barrier later the entries of the list, whose students' logits were fetched
// before anything was written, overwrite their places (so the gradient may
// take the logits' place, and no element is rounded twice).
#include <hip/hip_runtime.h>

#include <cstdint>

#include "launch.hpp"
#include "rows.hpp"
#include "spec_distill.h"

namespace specv {
namespace {

constexpr int kThreads = 1024;
constexpr int kRowWaves = kThreads / 64;
constexpr int kUnroll = 4;

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

struct ListEntry {
    int id;       // -1: unused
    float x;      // the student's scaled logit there
    double p;     // the teacher's probability
};

__device__ inline double row_sum(double v, double* lds) {
    v = wave_sum(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0)
        lds[threadIdx.x >> 6] = v;
    __syncthreads();
    double s = lds[0];
#pragma unroll
    for (int w = 1; w < kRowWaves; ++w)
        s += lds[w];
    return s;
}

__device__ inline float row_max(float v, float* lds) {
    v = wave_max(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0)
        lds[threadIdx.x >> 6] = v;
    __syncthreads();
    float m = lds[0];
#pragma unroll
    for (int w = 1; w < kRowWaves; ++w)
        m = fmaxf(m, lds[w]);
    return m;
}

template <int DT>
__device__ inline void store_element(void* row, long v, float g) {
    if constexpr (DT == kBF16) {
        const __bf16 h = static_cast<__bf16>(g);
        reinterpret_cast<__bf16*>(row)[v] = h;
    } else {
        reinterpret_cast<float*>(row)[v] = g;
    }
}

// Group g of the row's gradient; `whole`: it can go out as one 16-byte store.
template <int DT>
__device__ inline void store_group(const RowGroups<DT>& r, char* out, int g, bool whole,
                                   const float (&d)[RowGroups<DT>::W]) {
    constexpr int W = RowGroups<DT>::W;
    const long e0 = r.element(g);
    if (whole && r.inside(g)) {
        typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
        u32x4 v;
        if constexpr (DT == kBF16) {
            typedef float f32x2 __attribute__((ext_vector_type(2)));
            typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{d[2 * i], d[2 * i + 1]}, bf16x2));
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] = __float_as_uint(d[i]);
        }
        *reinterpret_cast<u32x4*>(out + e0 * RowGroups<DT>::ESZ) = v;
        return;
    }
#pragma unroll
    for (int i = 0; i < W; ++i)
        if (e0 + i >= 0 && e0 + i < r.vocab)
            store_element<DT>(out, e0 + i, d[i]);
}

template <int DT, bool LOSS, bool GRAD>
__global__ __launch_bounds__(kThreads) void distill_kernel(DistillArgs a) {
    using Row = RowGroups<DT>;
    constexpr int W = Row::W;
    __shared__ ListEntry list[SPEC_DISTILL_MAX_K];
    __shared__ double lds_d[kRowWaves];
    __shared__ float lds_f[kRowWaves];
    const int tid = threadIdx.x;
    const long row = blockIdx.x;
    const float inf = __builtin_huge_valf();
    const Row r(row_ptr(a.logits, DT, row, a.vocab), a.vocab);
    char* out = GRAD ? static_cast<char*>(a.out_grad) + row * static_cast<long>(a.vocab) * Row::ESZ : nullptr;
    const bool whole = GRAD && (reinterpret_cast<uintptr_t>(out) & 15) == static_cast<uintptr_t>(r.shift) * Row::ESZ;

    // The list: the teacher's probabilities and the student's logits there.
    float inv_t = 0.0f;
    const bool t_ok = temperature_mode(a.temperature[row], &inv_t) == 1;
    int id = -1;
    float y = -inf;
    if (tid < a.top_k) {
        id = a.ids[row * a.top_k + tid];
        if (id >= 0)
            y = a.teacher[row * a.top_k + tid] * inv_t;
        else
            id = -1;
    }
    const bool used = id >= 0;
    const bool outside = id >= a.vocab;
    float x_id = 0.0f;
    if (used && !outside)
        x_id = r.at(id) * inv_t;
    const bool any_used = __syncthreads_or(used);
    const bool any_outside = __syncthreads_or(outside);
    const bool any_mass = __syncthreads_or(used && !(y == -inf));
    auto fill = [&](float v) {
        if constexpr (GRAD) {
            float d[W];
#pragma unroll
            for (int e = 0; e < W; ++e)
                d[e] = v;
            for (int g = tid; g < r.groups; g += kThreads)
                store_group<DT>(r, out, g, whole, d);
        }
    };
    const float nan = __builtin_nanf("");
    if (!any_used || (t_ok && !any_outside && !any_mass && !a.teacher_lse)) {
        fill(0.0f);
        if (LOSS && tid == 0) {
            a.out_loss[row] = 0.0f;
            a.out_lse[row] = nan;
        }
        return;
    }
    double lse_t;
    if (a.teacher_lse) {
        lse_t = a.teacher_lse[row];
    } else {
        const float m = row_max(y, lds_f);
        const double s = row_sum(used ? exp(static_cast<double>(y) - static_cast<double>(m)) : 0.0, lds_d);
        lse_t = static_cast<double>(m) + log(s);
    }
    bool bad = !t_ok || any_outside || !is_finite_f64(lse_t);
    const double logp = static_cast<double>(y) - lse_t;
    const double p = used ? exp(logp) : 0.0;
    const double mass = row_sum(p, lds_d);
    if (tid < a.top_k)
        list[tid] = ListEntry{id, x_id, p};

    // The row's normaliser: s = sum 2^(x log2e - m), log-normaliser in base-2
    // units of the rounded constant, as the verifier keeps it.
    float m = 0.0f;
    double lse2 = 0.0;  // lse * kLog2e
    if constexpr (LOSS) {
        float mx = -inf;
        double s = 0.0;
        if (!bad) {
            float ref = kNegMax;
            for (int g0 = tid; g0 - tid < r.groups; g0 += kUnroll * kThreads) {
                uint4 q[kUnroll];
                r.template load<kUnroll, kThreads>(g0, r.groups, q);
                float bm = -inf;
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) {
                    float z[W];
                    Row::unpack(q[u], z);
#pragma unroll
                    for (int e = 0; e < W; ++e)
                        bm = fmaxf(bm, z[e]);
                }
                const float nr = fmaxf(ref, scale_logit(bm, inv_t) * kLog2e);
                s *= nr == ref ? 1.0 : static_cast<double>(fast_exp2(ref - nr));
                ref = nr;
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) {
                    float z[W];
                    Row::unpack(q[u], z);
                    float gs = 0.0f;
#pragma unroll
                    for (int e = 0; e < W; ++e)
                        gs += fast_exp2(__builtin_fmaf(scale_logit(z[e], inv_t), kLog2e, -ref));
                    s += static_cast<double>(gs);
                }
            }
            mx = ref;
        }
        m = row_max(mx, lds_f);
        s = row_sum(bad ? 0.0 : s * static_cast<double>(mx == m ? 1.0f : fast_exp2(mx - m)), lds_d);
        lse2 = static_cast<double>(m) + log2(s);
    } else {
        lse2 = a.lse_in[row] * static_cast<double>(kLog2e);
    }
    const double lse = LOSS ? lse2 / static_cast<double>(kLog2e) : a.lse_in[row];
    bad = bad || !is_finite_f64(lse);
    if constexpr (LOSS) {
        double term = 0.0;
        if (!bad && p > 0.0)
            term = p * (logp - (static_cast<double>(x_id) - lse));
        term = row_sum(term, lds_d);
        if (tid == 0) {
            a.out_loss[row] = bad ? nan : static_cast<float>(term);
            a.out_lse[row] = bad ? static_cast<double>(nan) : lse;
        }
    }
    if constexpr (GRAD) {
        if (bad) {
            fill(nan);
            return;
        }
        // exp(x - lse) = 2^(x log2e - ref) * 2^(ref - lse log2e), the second
        // factor (below 1 step of ref from 1) taken into the row's coefficient.
        const float ref = static_cast<float>(lse2);
        const double coef = static_cast<double>(a.weight[row]) * static_cast<double>(inv_t);
        const double dense = coef * mass * exp2(static_cast<double>(ref) - lse2);
        const float df = static_cast<float>(dense);
        __syncthreads();  // the list is written, and every gathered logit read
        for (int g0 = tid; g0 - tid < r.groups; g0 += kUnroll * kThreads) {
            uint4 q[kUnroll];
            r.template load<kUnroll, kThreads>(g0, r.groups, q);
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                if (g0 + u * kThreads >= r.groups)
                    break;
                float z[W], d[W];
                Row::unpack(q[u], z);
#pragma unroll
                for (int e = 0; e < W; ++e)
                    d[e] = df * fast_exp2(__builtin_fmaf(scale_logit(z[e], inv_t), kLog2e, -ref));
                store_group<DT>(r, out, g0 + u * kThreads, whole, d);
            }
        }
        __syncthreads();  // the dense part is written
        if (tid < a.top_k && used) {
            // The first entry of an id writes the sum of all entries of that id.
            double sum = 0.0;
            bool first = true;
            for (int j = 0; j < a.top_k; ++j) {
                if (list[j].id == id) {
                    sum += list[j].p;
                    first = first && j >= tid;
                }
            }
            if (first) {
                const double q = exp(static_cast<double>(x_id) - lse);
                store_element<DT>(out, id, static_cast<float>(coef * (mass * q - sum)));
            }
        }
    }
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

template <bool LOSS, bool GRAD>
int run(int rows, int dtype, const DistillArgs& a, void* hip_stream) {
    if (rows < 0 || a.vocab < 1 || (dtype != SPEC_F32 && dtype != SPEC_BF16) || a.top_k < 1 ||
        a.top_k > SPEC_DISTILL_MAX_K || rows >= (1L << 32) / kThreads)
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
    if (dtype == SPEC_BF16)
        distill_kernel<kBF16, LOSS, GRAD><<<dim3(rows), dim3(kThreads), 0, s>>>(a);
    else
        distill_kernel<kF32, LOSS, GRAD><<<dim3(rows), dim3(kThreads), 0, s>>>(a);
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
