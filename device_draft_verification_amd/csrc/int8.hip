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

// One workgroup per row, the row in registers between its maximum and its
// quotients (U groups per thread; U = 0: a longer row, read twice).
template <int DT, int U>
__global__ __launch_bounds__(kBlock) void quantize_rows_kernel(const void* __restrict__ x, int cols,
                                                              int8_t* __restrict__ out_q,
                                                              float* __restrict__ out_scale) {
    using Row = RowGroups<DT>;
    constexpr int W = Row::W;
    constexpr int N = U ? U : 4;  // groups in registers at a time
    __shared__ float lds_f[kWaves];
    const long row = blockIdx.x;
    const int tid = threadIdx.x;
    const Row r(row_ptr(x, DT, row, cols), cols);
    int8_t* q_row = out_q + row * cols;
    // a group's 8-bit values go out as one W-byte store
    const bool whole = ((reinterpret_cast<uintptr_t>(q_row) - r.shift) & (W - 1)) == 0;
    uint4 q[N];
    float m = 0.0f;
    uint32_t wild = 0;  // all exponent bits of any element set: a NaN or infinity
    // places outside the row are loaded as -inf: they are made zero here
    auto scan = [&](int g0) {
        r.template load<N, kBlock>(g0 - tid, tid, r.groups, q);
#pragma unroll
        for (int u = 0; u < N; ++u) {
            const int g = g0 + u * kBlock;
            float z[W];
            Row::unpack(q[u], z);
            if (g >= r.groups)
                continue;
#pragma unroll
            for (int e = 0; e < W; ++e) {
                const long k = r.element(g) + e;
                const bool in = r.inside(g) || (k >= 0 && k < cols);
                const uint32_t mag = in ? __float_as_uint(z[e]) & 0x7FFFFFFFu : 0u;
                wild |= mag >= 0x7F800000u;
                m = fmaxf(m, __uint_as_float(mag));
            }
        }
    };
    for (int g0 = tid; g0 - tid < r.groups; g0 += N * kBlock) {
        scan(g0);
        if (U)
            break;
    }
    m = wave_max(m);
    if ((tid & 63) == 0)
        lds_f[tid >> 6] = m;
    const bool any_wild = __syncthreads_or(wild != 0);
    m = fmaxf(fmaxf(lds_f[0], lds_f[1]), fmaxf(lds_f[2], lds_f[3]));
    float scale = m / 127.0f;  // correctly rounded
    if (any_wild)
        scale = __builtin_nanf("");
    if (tid == 0)
        out_scale[row] = scale;
    const bool zero = !(scale > 0.0f);
    const float inv = 1.0f / scale;
    for (int g0 = tid; g0 - tid < r.groups; g0 += N * kBlock) {
        if (!U)
            r.template load<N, kBlock>(g0 - tid, tid, r.groups, q);
#pragma unroll
        for (int u = 0; u < N; ++u) {
            const int g = g0 + u * kBlock;
            if (g >= r.groups)
                continue;
            float z[W];
            Row::unpack(q[u], z);
            uint32_t b[2] = {0, 0};
#pragma unroll
            for (int e = 0; e < W; ++e) {
                const int v = zero ? 0 : static_cast<int>(exact_quotient(z[e], scale, inv));
                b[e >> 2] |= (static_cast<uint32_t>(v) & 0xFFu) << (8 * (e & 3));
            }
            const long k0 = r.element(g);
            if (whole && r.inside(g)) {
                if constexpr (W == 8)
                    *reinterpret_cast<uint2*>(q_row + k0) = make_uint2(b[0], b[1]);
                else
                    *reinterpret_cast<uint32_t*>(q_row + k0) = b[0];
            } else {
#pragma unroll
                for (int e = 0; e < W; ++e)
                    if (k0 + e >= 0 && k0 + e < cols)
                        q_row[k0 + e] = static_cast<int8_t>(b[e >> 2] >> (8 * (e & 3)));
            }
        }
        if (U)
            break;
    }
}

template <int DT>
hipError_t launch_quantize(int rows, int cols, const void* x, int8_t* out_q, float* out_scale,
                           hipStream_t s) {
    constexpr int W = RowGroups<DT>::W;
    const long groups = (static_cast<long>(cols) + W - 1) / W + 1;  // at any alignment
    const dim3 grid(rows), block(kBlock);
    if (groups <= kBlock)
        quantize_rows_kernel<DT, 1><<<grid, block, 0, s>>>(x, cols, out_q, out_scale);
    else if (groups <= 2 * kBlock + 1)
        quantize_rows_kernel<DT, 3><<<grid, block, 0, s>>>(x, cols, out_q, out_scale);
    else if (groups <= 8 * kBlock)
        quantize_rows_kernel<DT, 8><<<grid, block, 0, s>>>(x, cols, out_q, out_scale);
    else
        quantize_rows_kernel<DT, 0><<<grid, block, 0, s>>>(x, cols, out_q, out_scale);
    return hipGetLastError();
}

// ----------------------------------------------------------------- product ---

// A workgroup of WV x WN wavefronts forms a TV (vocabulary) x TN (rows) tile of
// the output, each wavefront TV / WV x TN / WN as 32 x 32 tiles of
// v_mfma_i32_32x32x32_i8. The vocabulary is the M side: a lane then holds runs
// of four consecutive outputs of one row.
//
// K in stages of 64 bytes through a ring of LDS slots, loaded straight into LDS
// RING - 1 stages ahead: one barrier per stage, after which the slot of the
// stage before is refilled. A slot holds TV + TN rows of 64 bytes; a row's four
// 16-byte chunks sit at positions XORed with (row / 2) % 4, so the eight rows
// that a phase of a fragment read touches lie in eight different 16-byte
// places of 128.
// Rows past the end repeat the last one (their outputs are not stored), chunks
// past the depth come from a page of zeros.
constexpr int kStageK = 64;

__device__ int4 zero_chunk;  // zero from load on, never written

__device__ constexpr int wait_loads(int n) {
    // s_waitcnt operand: vmcnt n (bits 3:0 and 15:14), lgkmcnt 0 (bits 11:8), expcnt not waited
    return (n & 0xF) | ((n >> 4) << 14) | (0x7 << 4);
}

// At most n global loads and no LDS access of this wavefront outstanding, then
// the workgroup's barrier. Unlike __syncthreads it leaves the n youngest loads
// in flight; the empty asm keeps the compiler from moving memory accesses across.
template <int N>
__device__ __forceinline__ void stage_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(wait_loads(N));
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

template <int TV, int TN, int WV, int WN, int RING, int OUT>
__global__ __launch_bounds__(64 * WV * WN, 2) void int8_product_kernel(
    const int8_t* __restrict__ a, const float* __restrict__ a_scale, const int8_t* __restrict__ w,
    const float* __restrict__ w_scale, int rows, int depth, int cols, int tiles_n, int tiles,
    void* __restrict__ out) {
    constexpr int kWavesHere = WV * WN;
    constexpr int MV = TV / WV / 32, MN = TN / WN / 32;
    constexpr int kSlot = (TV + TN) * kStageK;
    constexpr int kLoads = (TV + TN) / 16 / kWavesHere;  // 1 KiB each, per wavefront and stage
    static_assert((TV + TN) / 16 % kWavesHere == 0, "every wavefront issues the same loads");
    // The epilogue turns a wavefront's 32 rows x 32 MV entries through LDS.
    constexpr int ESZ = OUT == kBF16 ? 2 : 4;
    constexpr int kRowBytes = 32 * MV * ESZ + 16;
    constexpr int kTurn = 32 * kRowBytes;
    constexpr int kLds = RING * kSlot > kWavesHere * kTurn ? RING * kSlot : kWavesHere * kTurn;
    __shared__ __align__(16) int8_t lds[kLds];
    const int lane = threadIdx.x & 63;
    const int wid = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
    // Workgroups go round the eight XCDs: each XCD takes a contiguous run of
    // tiles, rows fastest, so that the tiles that share weights share an L2.
    const int blk = blockIdx.x, xcd = blk & 7, at = blk >> 3;
    const int per = tiles >> 3, extra = tiles & 7;
    const int tile = xcd * per + (xcd < extra ? xcd : extra) + at;
    const int v0 = tile / tiles_n * TV;
    const int n0 = tile % tiles_n * TN;

    // This lane's chunk of each of its wavefront's loads.
    const int8_t* src[kLoads];
    int chunk[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int row = (wid + kWavesHere * i) * 16 + (lane >> 2);
        chunk[i] = ((lane & 3) ^ ((row >> 1) & 3)) * 16;
        if (row < TV) {
            const int v = v0 + row;
            src[i] = w + static_cast<size_t>(v < cols ? v : cols - 1) * depth + chunk[i];
        } else {
            const int n = n0 + row - TV;
            src[i] = a + static_cast<size_t>(n < rows ? n : rows - 1) * depth + chunk[i];
        }
    }
    const int stages = (depth + kStageK - 1) / kStageK;
    const int8_t* zeros = reinterpret_cast<const int8_t*>(&zero_chunk);
    asm volatile("" : "+s"(zeros));  // looked up once, not in every stage
    auto issue = [&](int s) {
        int8_t* slot = lds + (s % RING) * kSlot;
        const int k = s * kStageK;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            // stages past the end load zeros into slots that nobody reads
            const int8_t* from = k + kStageK <= depth || k + chunk[i] < depth ? src[i] + k : zeros;
            __builtin_amdgcn_global_load_lds(reinterpret_cast<const void*>(from),
                                             slot + (wid + kWavesHere * i) * 1024, 16, 0, 0);
        }
    };
    i32x16 acc[MV][MN];
#pragma unroll
    for (int i = 0; i < MV; ++i)
#pragma unroll
        for (int j = 0; j < MN; ++j)
            acc[i][j] = i32x16{};
#pragma unroll
    for (int s = 0; s < RING - 1; ++s)
        issue(s);
    const int wv = wid % WV * (TV / WV), wn = wid / WV * (TN / WN);
    const int frag_row = lane & 31;
    const int swz = (frag_row >> 1) & 3;  // rows of a tile start at multiples of 32
    // Half a stage (32 of K) is multiplied while the next half's fragments are
    // read: of stage s - 1 the second half waits in registers over the barrier.
    i32x4 fw[2][MV], fa[2][MN];
    auto read = [&](int s, int half) {
        const int8_t* slot = lds + (s % RING) * kSlot;
        const int pos = ((2 * half + (lane >> 5)) ^ swz) * 16;
#pragma unroll
        for (int j = 0; j < MN; ++j)
            fa[half][j] = *reinterpret_cast<const i32x4*>(slot + (TV + wn + 32 * j + frag_row) * kStageK + pos);
#pragma unroll
        for (int i = 0; i < MV; ++i)
            fw[half][i] = *reinterpret_cast<const i32x4*>(slot + (wv + 32 * i + frag_row) * kStageK + pos);
    };
    auto multiply = [&](int half) {
#pragma unroll
        for (int i = 0; i < MV; ++i)
#pragma unroll
            for (int j = 0; j < MN; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fw[half][i], fa[half][j], acc[i][j], 0, 0, 0);
    };
    for (int s = 0; s < stages; ++s) {
        // Stage s has landed once at most the RING - 2 stages after it are out;
        // past the barrier every wavefront has also read all of stage s - 1.
        stage_barrier<kLoads*(RING - 2)>();
        issue(s + RING - 1);
        read(s, 0);
        __builtin_amdgcn_sched_barrier(0);
        if (s > 0)
            multiply(1);
        read(s, 1);
        __builtin_amdgcn_sched_barrier(0);
        multiply(0);
    }
    multiply(1);
    // No load may still be on its way into LDS when it is used again.
    stage_barrier<0>();

    // Lane l holds entries 8 (e / 4) + 4 (l / 32) + e % 4 of row l % 32 of a
    // 32 x 32 tile. Turned through LDS (each wavefront in its own part), they go
    // out as 16-byte stores along the rows.
    int8_t* turn = lds + wid * kTurn;
    const bool whole = (static_cast<size_t>(cols) * ESZ) % 16 == 0 &&
                       (reinterpret_cast<uintptr_t>(out) & 15) == 0;
#pragma unroll
    for (int j = 0; j < MN; ++j) {
        const int nb = n0 + wn + 32 * j;
        const int n = nb + (lane & 31);
        const float sa = a_scale[n < rows ? n : rows - 1];
#pragma unroll
        for (int i = 0; i < MV; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int at_v = 32 * i + 8 * e + 4 * (lane >> 5);
                float z[4];
#pragma unroll
                for (int f = 0; f < 4; ++f) {
                    const int v = v0 + wv + at_v + f;
                    z[f] = static_cast<float>(acc[i][j][4 * e + f]) * sa * w_scale[v < cols ? v : cols - 1];
                }
                int8_t* to = turn + (lane & 31) * kRowBytes + at_v * ESZ;
                if constexpr (OUT == kBF16) {
                    typedef float f32x2 __attribute__((ext_vector_type(2)));
                    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
                    *reinterpret_cast<uint2*>(to) = make_uint2(
                        __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{z[0], z[1]}, bf16x2)),
                        __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{z[2], z[3]}, bf16x2)));
                } else {
                    *reinterpret_cast<float4*>(to) = make_float4(z[0], z[1], z[2], z[3]);
                }
            }
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        constexpr int kEntries = 32 * MV;
        if (whole) {
            constexpr int kPer = 16 / ESZ;               // entries per store
            constexpr int kLanes = kEntries / kPer;      // lanes per row
#pragma unroll
            for (int t = 0; t < 32 * kLanes / 64; ++t) {
                const int r = t * (64 / kLanes) + lane / kLanes, c = lane % kLanes * kPer;
                const uint4 x = *reinterpret_cast<const uint4*>(turn + r * kRowBytes + c * ESZ);
                const int v = v0 + wv + c;
                if (nb + r < rows && v < cols)
                    *reinterpret_cast<uint4*>(static_cast<char*>(out) +
                                              (static_cast<size_t>(nb + r) * cols + v) * ESZ) = x;
            }
        } else {
            using elem_t = typename std::conditional<OUT == kBF16, uint16_t, uint32_t>::type;
            for (int r = 0; r < 32 && nb + r < rows; ++r)
#pragma unroll
                for (int c = lane; c < kEntries; c += 64)
                    if (v0 + wv + c < cols)
                        static_cast<elem_t*>(out)[static_cast<size_t>(nb + r) * cols + v0 + wv + c] =
                            *reinterpret_cast<const elem_t*>(turn + r * kRowBytes + c * ESZ);
        }
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    }
}

template <int TV, int TN, int WV, int WN, int RING>
hipError_t launch_tile(int rows, int depth, int cols, const int8_t* a, const float* a_scale,
                       const int8_t* w, const float* w_scale, int out_dtype, void* out, hipStream_t s) {
    const long tiles_v = (static_cast<long>(cols) + TV - 1) / TV;
    const long tiles_n = (static_cast<long>(rows) + TN - 1) / TN;
    if (tiles_v * tiles_n >= (1L << 32) / (64 * WV * WN))
        return hipErrorInvalidValue;
    const dim3 grid(static_cast<unsigned>(tiles_v * tiles_n)), block(64 * WV * WN);
    if (out_dtype == SPEC_BF16)
        int8_product_kernel<TV, TN, WV, WN, RING, kBF16><<<grid, block, 0, s>>>(
            a, a_scale, w, w_scale, rows, depth, cols, static_cast<int>(tiles_n),
            static_cast<int>(tiles_v * tiles_n), out);
    else
        int8_product_kernel<TV, TN, WV, WN, RING, kF32><<<grid, block, 0, s>>>(
            a, a_scale, w, w_scale, rows, depth, cols, static_cast<int>(tiles_n),
            static_cast<int>(tiles_v * tiles_n), out);
    return hipGetLastError();
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
    const hipError_t e = dtype == SPEC_BF16 ? launch_quantize<kBF16>(rows, cols, x, out_q, out_scale, s)
                                            : launch_quantize<kF32>(rows, cols, x, out_q, out_scale, s);
    return e == hipSuccess ? SPEC_OK : SPEC_EHIP;
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
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    const long big = ((static_cast<long>(cols) + 255) / 256) * ((static_cast<long>(rows) + 127) / 128);
    hipError_t e;
    if (rows > 64 && big >= 256)
        e = launch_tile<256, 128, 2, 2, 3>(rows, depth, cols, a, a_scale, w, w_scale, out_dtype, out, s);
    else if (rows > 32)
        e = launch_tile<128, 64, 2, 2, 4>(rows, depth, cols, a, a_scale, w, w_scale, out_dtype, out, s);
    else
        e = launch_tile<128, 32, 2, 1, 4>(rows, depth, cols, a, a_scale, w, w_scale, out_dtype, out, s);
    return e == hipSuccess ? SPEC_OK : e == hipErrorInvalidValue ? SPEC_EINVAL : SPEC_EHIP;
}

}  // extern "C"
