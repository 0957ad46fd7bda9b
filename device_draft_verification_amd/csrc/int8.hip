// Quantisation of rows to 8 bits, and the product of two quantised matrices
// with a scale for each row of either (spec_int8.h):
//
//   scale = fl32(max |x| / 127), q = rne(x / scale);
//   out[n][v] = (sum_k a[n][k] w[v][k]) * a_scale[n] * w_scale[v].
#include <hip/hip_runtime.h>

#include <cstdint>

#include "rows.hpp"
#include "spec_int8.h"

namespace specv {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// ------------------------------------------------------------ quantisation ---

// x / scale rounded to the nearest integer, ties to even, from the exact
// quotient. rint(x * fl32(1/scale)) is within one of it (the reciprocal of the
// smallest subnormal scales overflows; those divide); for the right integer r
// the remainder x - r * scale is a multiple of the smaller operand's last place
// and at most half a scale in size, so the fma below is exact and decides.
__device__ inline float exact_quotient(float x, float scale, float inv) {
    float r = __builtin_rintf(inv == __builtin_huge_valf() ? x / scale : x * inv);
    const float rem = __builtin_fmaf(-r, scale, x);
    const float twice = 2.0f * fabsf(rem);
    const bool odd = (static_cast<int>(r) & 1) != 0;
    if (twice > scale || (twice == scale && odd))
        r += rem > 0.0f ? 1.0f : -1.0f;
    return fminf(fmaxf(r, -127.0f), 127.0f);
}

template <int DT>
__global__ __launch_bounds__(kBlock) void quantize_rows_kernel(const void* __restrict__ x, int cols,
                                                              int8_t* __restrict__ out_q,
                                                              float* __restrict__ out_scale) {
    using Row = RowGroups<DT>;
    constexpr int W = Row::W;
    __shared__ float lds_f[kWaves];
    const long row = blockIdx.x;
    const Row r(row_ptr(x, DT, row, cols), cols);
    int8_t* q_row = out_q + row * cols;
    float m = 0.0f;
    bool wild = false;
    for (int g = threadIdx.x; g < r.groups; g += kBlock) {
        uint4 q[1];
        r.template load<1, kBlock>(g, r.groups, q);
        float z[W];
        Row::unpack(q[0], z);
#pragma unroll
        for (int e = 0; e < W; ++e) {
            const long k = r.element(g) + e;
            if (k >= 0 && k < cols) {
                wild = wild || !is_finite_f32(z[e]);
                m = fmaxf(m, fabsf(z[e]));
            }
        }
    }
    wild = __syncthreads_or(wild);
    m = block_max(m, lds_f);
    float scale = m / 127.0f;  // correctly rounded
    if (wild)
        scale = __builtin_nanf("");
    if (threadIdx.x == 0)
        out_scale[row] = scale;
    const bool zero = !(scale > 0.0f);
    const float inv = 1.0f / scale;
    for (int g = threadIdx.x; g < r.groups; g += kBlock) {
        uint4 q[1];
        r.template load<1, kBlock>(g, r.groups, q);
        float z[W];
        Row::unpack(q[0], z);
#pragma unroll
        for (int e = 0; e < W; ++e) {
            const long k = r.element(g) + e;
            if (k >= 0 && k < cols)
                q_row[k] = zero ? 0 : static_cast<int8_t>(exact_quotient(z[e], scale, inv));
        }
    }
}

// ----------------------------------------------------------------- product ---

// One 128 (vocabulary) x 128 (rows) tile per workgroup of four wavefronts, each
// 64 x 64 as 2 x 2 tiles of v_mfma_i32_32x32x32_i8; K in chunks of 64 staged
// through LDS. The vocabulary is the M side: a lane then holds runs of four
// consecutive outputs of one row.
constexpr int kTileV = 128, kTileN = 128, kTileK = 64;
constexpr int kPadK = kTileK + 16;  // bytes per staged row

template <int OUT>
__device__ inline void store_out(void* out, size_t at, float v) {
    if constexpr (OUT == kBF16)
        reinterpret_cast<__bf16*>(out)[at] = static_cast<__bf16>(v);
    else
        reinterpret_cast<float*>(out)[at] = v;
}

template <int OUT>
__global__ __launch_bounds__(kBlock) void int8_product_kernel(
    const int8_t* __restrict__ a, const float* __restrict__ a_scale, const int8_t* __restrict__ w,
    const float* __restrict__ w_scale, int rows, int depth, int cols, int tiles_v,
    void* __restrict__ out) {
    __shared__ __align__(16) int8_t lds_w[kTileV * kPadK];
    __shared__ __align__(16) int8_t lds_a[kTileN * kPadK];
    const int tid = threadIdx.x, lane = tid & 63, wid = tid >> 6;
    const int v0 = static_cast<int>(blockIdx.x % tiles_v) * kTileV;
    const int n0 = static_cast<int>(blockIdx.x / tiles_v) * kTileN;
    const int wv = (wid & 1) * 64, wn = (wid >> 1) * 64;
    i32x16 acc[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
            acc[i][j] = i32x16{};
    for (int k0 = 0; k0 < depth; k0 += kTileK) {
        __syncthreads();
        // 128 rows x 4 chunks of 16 bytes for either side; rows past the end
        // repeat the last one (never stored), chunks past the depth are zero
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int c = tid + i * kBlock, rr = c >> 2, kk = (c & 3) * 16;
            const bool in = k0 + kk < depth;
            const int v = v0 + rr < cols ? v0 + rr : cols - 1;
            const int n = n0 + rr < rows ? n0 + rr : rows - 1;
            const int k = in ? k0 + kk : 0;
            uint4 x = *reinterpret_cast<const uint4*>(w + static_cast<size_t>(v) * depth + k);
            uint4 y = *reinterpret_cast<const uint4*>(a + static_cast<size_t>(n) * depth + k);
            if (!in)
                x = y = make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4*>(lds_w + rr * kPadK + kk) = x;
            *reinterpret_cast<uint4*>(lds_a + rr * kPadK + kk) = y;
        }
        __syncthreads();
#pragma unroll
        for (int ks = 0; ks < kTileK; ks += 32) {
            i32x4 fw[2], fa[2];
            const int kb = ks + 16 * (lane >> 5);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                fw[i] = *reinterpret_cast<const i32x4*>(lds_w + (wv + 32 * i + (lane & 31)) * kPadK + kb);
                fa[i] = *reinterpret_cast<const i32x4*>(lds_a + (wn + 32 * i + (lane & 31)) * kPadK + kb);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fw[i], fa[j], acc[i][j], 0, 0, 0);
        }
    }
    // Lane l holds rows 8 (r / 4) + 4 (l / 32) + r % 4 and column l % 32 of a
    // 32 x 32 tile.
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int n = n0 + wn + 32 * j + (lane & 31);
        if (n >= rows)
            continue;
        const float sa = a_scale[n];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int v = v0 + wv + 32 * i + 8 * (e >> 2) + 4 * (lane >> 5) + (e & 3);
                if (v < cols)
                    store_out<OUT>(out, static_cast<size_t>(n) * cols + v,
                                   static_cast<float>(acc[i][j][e]) * sa * w_scale[v]);
            }
    }
}

}  // namespace
}  // namespace specv

using namespace specv;

extern "C" {

int spec_quantize_rows(int rows, int cols, int dtype, const void* x, int8_t* out_q,
                       float* out_scale, void* hip_stream) {
    if (rows < 0 || cols < 1 || (dtype != SPEC_F32 && dtype != SPEC_BF16) || rows >= (1L << 32) / kBlock)
        return SPEC_EINVAL;
    if (rows == 0)
        return SPEC_OK;
    if (!x || !out_q || !out_scale || !aligned(x, dtype == SPEC_BF16 ? 2 : 4) || !aligned(out_scale, 4))
        return SPEC_EINVAL;
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    if (dtype == SPEC_BF16)
        quantize_rows_kernel<kBF16><<<dim3(rows), dim3(kBlock), 0, s>>>(x, cols, out_q, out_scale);
    else
        quantize_rows_kernel<kF32><<<dim3(rows), dim3(kBlock), 0, s>>>(x, cols, out_q, out_scale);
    return hipGetLastError() == hipSuccess ? SPEC_OK : SPEC_EHIP;
}

int spec_int8_product(int rows, int depth, int cols, const int8_t* a, const float* a_scale,
                      const int8_t* w, const float* w_scale, int out_dtype, void* out,
                      void* hip_stream) {
    if (rows < 0 || cols < 1 || depth < 16 || depth % 16 != 0 || depth > SPEC_INT8_MAX_DEPTH ||
        (out_dtype != SPEC_F32 && out_dtype != SPEC_BF16))
        return SPEC_EINVAL;
    if (rows == 0)
        return SPEC_OK;
    if (!a || !a_scale || !w || !w_scale || !out || !aligned(a, 16) || !aligned(w, 16) ||
        !aligned(a_scale, 4) || !aligned(w_scale, 4) || !aligned(out, out_dtype == SPEC_BF16 ? 2 : 4))
        return SPEC_EINVAL;
    const long tiles_v = (static_cast<long>(cols) + kTileV - 1) / kTileV;
    const long tiles_n = (static_cast<long>(rows) + kTileN - 1) / kTileN;
    if (tiles_v * tiles_n >= (1L << 32) / kBlock)
        return SPEC_EINVAL;
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    const dim3 grid(static_cast<unsigned>(tiles_v * tiles_n));
    if (out_dtype == SPEC_BF16)
        int8_product_kernel<kBF16><<<grid, dim3(kBlock), 0, s>>>(a, a_scale, w, w_scale, rows, depth, cols,
                                                                 static_cast<int>(tiles_v), out);
    else
        int8_product_kernel<kF32><<<grid, dim3(kBlock), 0, s>>>(a, a_scale, w, w_scale, rows, depth, cols,
                                                                static_cast<int>(tiles_v), out);
    return hipGetLastError() == hipSuccess ? SPEC_OK : SPEC_EHIP;
}

}  // extern "C"
