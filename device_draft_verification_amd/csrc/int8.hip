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
__device__ inline int exact_quotient(float x, float scale, float inv) {
    float r = __builtin_rintf(inv == __builtin_huge_valf() ? x / scale : x * inv);
    const float rem = __builtin_fmaf(-r, scale, x);
    const float twice = 2.0f * fabsf(rem);
    const bool odd = (static_cast<int>(r) & 1) != 0;
    if (twice > scale || (twice == scale && odd))
        r += rem > 0.0f ? 1.0f : -1.0f;
    return static_cast<int>(fminf(fmaxf(r, -127.0f), 127.0f));
}

// A group's quotients as bytes. Adding 1.5 * 2^23 rounds to an integer, ties to
// even, and leaves it in the low byte; only where a remainder reaches half a
// scale (a tie, or a product x * inv on the wrong side of one) the group takes
// the exact way.
template <int W>
__device__ inline void quantize_group(const float (&x)[W], float scale, float inv, uint32_t (&b)[2]) {
    constexpr float kMagic = 12582912.0f;
    const float half = 0.5f * scale;
    uint32_t w[W];
    bool near = !(scale >= 1.17549435e-38f);  // subnormal: half a scale may not be exact
#pragma unroll
    for (int e = 0; e < W; ++e) {
        const float m = __builtin_amdgcn_fmed3f(x[e] * inv, -127.0f, 127.0f) + kMagic;
        w[e] = __float_as_uint(m);
        near = near || fabsf(__builtin_fmaf(-(m - kMagic), scale, x[e])) >= half;
    }
    if (near) {
#pragma unroll
        for (int e = 0; e < W; ++e)
            w[e] = static_cast<uint32_t>(exact_quotient(x[e], scale, inv));
    }
#pragma unroll
    for (int i = 0; i < W / 4; ++i) {
        // v_perm_b32(a, b, s): byte k of the result is byte s[k] of {a, b}, b's first
        const uint32_t lo = __builtin_amdgcn_perm(w[4 * i + 1], w[4 * i], 0x0c0c0400u);
        const uint32_t hi = __builtin_amdgcn_perm(w[4 * i + 3], w[4 * i + 2], 0x04000c0cu);
        b[i] = lo | hi;
    }
}

// One workgroup of T threads per row, the row in registers between its maximum
// and its quotients (U groups per thread; LONG: a longer row, read twice). Bound by
// the read of x and the write of the bytes: 2304 rows of 4096 bf16 (28 MB) 8 us,
// 3.5 TB/s, of which about 4 are the launch, the load's latency and the reduction.
template <int DT, int T, int U, bool LONG>
__global__ __launch_bounds__(T) void quantize_rows_kernel(const void* __restrict__ x, int cols,
                                                          int8_t* __restrict__ out_q,
                                                          float* __restrict__ out_scale) {
    using Row = RowGroups<DT>;
    constexpr int W = Row::W;
    __shared__ uint32_t lds_m[T / 64];
    const long row = blockIdx.x;
    const int tid = threadIdx.x;
    const Row r(row_ptr(x, DT, row, cols), cols);
    int8_t* q_row = out_q + row * cols;
    // a group's 8-bit values go out as one W-byte store
    const bool whole = ((reinterpret_cast<uintptr_t>(q_row) - r.shift) & (W - 1)) == 0;
    uint4 q[U];
    // The largest magnitude as an integer: the order of floats without a sign
    // is the order of their bits, and a NaN or infinity comes out on top.
    uint32_t m = 0;
    for (int g0 = 0; g0 < r.groups; g0 += U * T) {
        r.template load<U, T>(g0, tid, r.groups, q);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int g = g0 + tid + u * T;
            float z[W];
            Row::unpack(q[u], z);
            if (g >= r.groups)
                continue;
            const bool inside = r.inside(g);
            const long k0 = r.element(g);
#pragma unroll
            for (int e = 0; e < W; ++e) {
                // places outside the row are loaded as -inf: they do not count
                const uint32_t mag = __float_as_uint(z[e]) & 0x7FFFFFFFu;
                if (inside || (k0 + e >= 0 && k0 + e < cols))
                    m = mag > m ? mag : m;
            }
        }
        if (!LONG)
            break;
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) {
        const uint32_t o = __shfl_xor(m, off, 64);
        m = o > m ? o : m;
    }
    if constexpr (T > 64) {
        if ((tid & 63) == 0)
            lds_m[tid >> 6] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < T / 64; ++w) {
            const uint32_t o = lds_m[w];
            m = o > m ? o : m;
        }
    }
    const float scale = m >= 0x7F800000u ? __builtin_nanf("") : __uint_as_float(m) / 127.0f;  // correctly rounded
    if (tid == 0)
        out_scale[row] = scale;
    const bool zero = !(scale > 0.0f);
    const float inv = 1.0f / scale;
    for (int g0 = 0; g0 < r.groups; g0 += U * T) {
        if (LONG)
            r.template load<U, T>(g0, tid, r.groups, q);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int g = g0 + tid + u * T;
            if (g >= r.groups)
                continue;
            float z[W];
            Row::unpack(q[u], z);
            uint32_t b[2] = {0, 0};
            if (!zero)
                quantize_group<W>(z, scale, inv, b);
            const long k0 = r.element(g);
            if (whole && r.inside(g)) {
                if constexpr (W == 8)
                    __builtin_nontemporal_store(static_cast<uint64_t>(b[1]) << 32 | b[0],
                                                reinterpret_cast<uint64_t*>(q_row + k0));
                else
                    __builtin_nontemporal_store(b[0], reinterpret_cast<uint32_t*>(q_row + k0));
            } else {
#pragma unroll
                for (int e = 0; e < W; ++e)
                    if (k0 + e >= 0 && k0 + e < cols)
                        q_row[k0 + e] = static_cast<int8_t>(b[e >> 2] >> (8 * (e & 3)));
            }
        }
        if (!LONG)
            break;
    }
}

template <int DT>
hipError_t launch_quantize(int rows, int cols, const void* x, int8_t* out_q, float* out_scale,
                           hipStream_t s) {
    constexpr int W = RowGroups<DT>::W;
    const bool even = cols % W == 0 && aligned(x, 16);
    const long groups = (static_cast<long>(cols) + W - 1) / W + (even ? 0 : 1);  // at any alignment
#define SPEC_QUANTIZE(T, U, LONG)                                                              \
    quantize_rows_kernel<DT, T, U, LONG><<<dim3(rows), dim3(T), 0, s>>>(x, cols, out_q, out_scale)
    // Two groups per thread: enough loads in flight, and short chains of
    // quotients (2304 rows of 4096 bf16: 8 us; four per thread 10, eight 14).
    // So many rows that one dispatch does not hold the wider workgroups (2^32
    // work-items) take the narrow one that reads a row twice.
    auto fits = [&](long threads) { return rows * threads < (1L << 32); };
    if (groups <= 128)
        SPEC_QUANTIZE(64, 2, false);
    else if (groups <= 256)
        SPEC_QUANTIZE(128, 2, false);
    else if (groups <= 512)
        SPEC_QUANTIZE(256, 2, false);
    else if (groups <= 1024 && fits(512))
        SPEC_QUANTIZE(512, 2, false);
    else if (groups <= 2048 && fits(1024))
        SPEC_QUANTIZE(1024, 2, false);
    else
        SPEC_QUANTIZE(256, 8, true);
#undef SPEC_QUANTIZE
    return hipGetLastError();
}

// ----------------------------------------------------------------- product ---

// A workgroup of WV x WN wavefronts forms a TV (vocabulary) x TN (rows) tile of
// the output, each wavefront TV / WV x TN / WN as 32 x 32 tiles of
// v_mfma_i32_32x32x32_i8. The vocabulary is the M side: a lane then holds runs
// of four consecutive outputs of one row.
//
// K in stages of BK bytes through a ring of LDS slots, loaded straight into LDS
// RING - 1 stages ahead: one barrier per stage, after which the slot of the
// stage before is refilled. A slot holds TV + TN rows of BK bytes; a row's
// 16-byte chunks sit at positions XORed with the row's number in units of the
// banks' 256 bytes (row / 4 for BK = 64), so the sixteen rows that a phase of a
// fragment read touches lie in sixteen different 16-byte places of them (row / 2
// for BK = 64 measured one conflict cycle for every useful one).
// Rows past the end repeat the last one (their outputs are not stored), chunks
// past the depth come from a page of zeros.
//
// Many rows are bound by the matrix cores: 2304 x 152064, D = 4096 takes 1260-1360 us
// (2.1-2.3 POP/s; a library's int8 product of the shape 1413), the cores multiplying
// 62 % of the cycles at the 1.65 GHz that the load leaves. In 256 x 256 tiles a
// wavefront reads 6 fragments for 8 multiplications (in 128 x 128, 4 for 4); 8
// wavefronts, 2 per SIMD (4 wavefronts of 128 x 128 each 1395 us;
// 64-byte stages in a ring of 4 1380; raised wave priority around the products
// 1641). Few rows are bound by the read of the weights: 1 row x 152064,
// D = 4096 127 us, 64 rows at D = 512 19 us, 5 TB/s each.
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

template <int TV, int TN, int WV, int WN, int BK, int RING, int OUT>
__global__ __launch_bounds__(64 * WV * WN, 2) void int8_product_kernel(
    const int8_t* __restrict__ a, const float* __restrict__ a_scale, const int8_t* __restrict__ w,
    const float* __restrict__ w_scale, int rows, int depth, int cols, int tiles_n, int tiles,
    void* __restrict__ out) {
    constexpr int kWavesHere = WV * WN;
    constexpr int MV = TV / WV / 32, MN = TN / WN / 32;
    constexpr int kSlot = (TV + TN) * BK;
    constexpr int kChunks = BK / 16;                  // of a row in a slot
    constexpr int kRowsPerLoad = 64 / kChunks;        // a load covers 1 KiB
    constexpr int kLoads = kSlot / 1024 / kWavesHere;  // per wavefront and stage
    constexpr int kSteps = BK / 32;                   // of K = 32 each
    static_assert(kSlot / 1024 % kWavesHere == 0, "every wavefront issues the same loads");
    static_assert(kSteps % 2 == 0 && 256 % BK == 0, "two sets of fragments take turns");
    auto swizzle = [](int row) { return row / (256 / BK) % kChunks; };
    // The epilogue turns a wavefront's 32 rows x 32 MV entries through LDS.
    constexpr int ESZ = OUT == kBF16 ? 2 : 4;
    constexpr int kRowBytes = 32 * MV * ESZ + 16;
    constexpr int kTurn = 32 * kRowBytes;
    constexpr int kLds = RING * kSlot > kWavesHere * kTurn ? RING * kSlot : kWavesHere * kTurn;
    // One LDS object: with two the compiler keeps their accesses apart by alias
    // scopes, and then waits for every load into LDS before any read of it.
    __shared__ __align__(16) int8_t lds[kLds + TV * sizeof(float)];
    float* scale_v = reinterpret_cast<float*>(lds + kLds);
    const int lane = threadIdx.x & 63;
    const int wid = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
    // Workgroups go round the eight XCDs: each XCD takes a contiguous run of
    // tiles, rows fastest, so that the tiles that share weights share an L2.
    const int blk = blockIdx.x, xcd = blk & 7, at = blk >> 3;
    const int per = tiles >> 3, extra = tiles & 7;
    const int tile = xcd * per + (xcd < extra ? xcd : extra) + at;
    const int v0 = tile / tiles_n * TV;
    const int n0 = tile % tiles_n * TN;
    for (int t = threadIdx.x; t < TV; t += 64 * WV * WN)  // read behind the loop's barriers
        scale_v[t] = w_scale[v0 + t < cols ? v0 + t : cols - 1];

    // This lane's chunk of each of its wavefront's loads.
    const int8_t* src[kLoads];
    int chunk[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int row = (wid + kWavesHere * i) * kRowsPerLoad + lane / kChunks;
        chunk[i] = (lane % kChunks ^ swizzle(row)) * 16;
        if (row < TV) {
            const int v = v0 + row;
            src[i] = w + static_cast<size_t>(v < cols ? v : cols - 1) * depth + chunk[i];
        } else {
            const int n = n0 + row - TV;
            src[i] = a + static_cast<size_t>(n < rows ? n : rows - 1) * depth + chunk[i];
        }
    }
    const int stages = (depth + BK - 1) / BK;
    const int8_t* zeros = reinterpret_cast<const int8_t*>(&zero_chunk);
    asm volatile("" : "+s"(zeros));  // looked up once, not in every stage
    auto issue = [&](int s, int i) {
        int8_t* slot = lds + (s % RING) * kSlot;
        const int k = s * BK;
        // stages past the end load zeros into slots that nobody reads
        const int8_t* from = k + BK <= depth || k + chunk[i] < depth ? src[i] + k : zeros;
        __builtin_amdgcn_global_load_lds(reinterpret_cast<const void*>(from),
                                         slot + (wid + kWavesHere * i) * 1024, 16, 0, 0);
    };
    i32x16 acc[MV][MN];
#pragma unroll
    for (int i = 0; i < MV; ++i)
#pragma unroll
        for (int j = 0; j < MN; ++j)
            acc[i][j] = i32x16{};
#pragma unroll
    for (int s = 0; s < RING - 1; ++s)
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            issue(s, i);
    const int wv = wid % WV * (TV / WV), wn = wid / WV * (TN / WN);
    const int frag_row = lane & 31;
    const int swz = swizzle(frag_row);  // rows of a tile start at multiples of 32
    // A step (32 of K) is multiplied while the next one's fragments are read: of
    // stage s - 1 the last step waits in registers over the barrier. The fragment
    // reads and loads go between the matrix instructions, in whose shadow they
    // issue: in one run before them, all wavefronts issue theirs together behind
    // the barrier with the matrix cores idle (1486 us against 1380 at N = 2304,
    // D = 4096, V = 152064).
    constexpr int kReads = MV + MN, kMul = MV * MN;
    i32x4 fw[2][MV], fa[2][MN];
    auto read = [&](int s, int step, int i) {
        const int8_t* slot = lds + (s % RING) * kSlot;
        const int pos = ((2 * step + (lane >> 5)) ^ swz) * 16;
        if (i < MN)
            fa[step & 1][i] = *reinterpret_cast<const i32x4*>(slot + (TV + wn + 32 * i + frag_row) * BK + pos);
        else
            fw[step & 1][i - MN] =
                *reinterpret_cast<const i32x4*>(slot + (wv + 32 * (i - MN) + frag_row) * BK + pos);
    };
    auto multiply = [&](int step, int m) {
        const int i = m / MN, j = m % MN;
        acc[i][j] =
            __builtin_amdgcn_mfma_i32_32x32x32_i8(fw[step & 1][i], fa[step & 1][j], acc[i][j], 0, 0, 0);
    };
    // Of `work` pieces spread over `steps` steps, the first of step n.
    auto share = [](int n, int steps, int work) { return (n * work + steps - 1) / steps; };
    for (int s = 0; s < stages; ++s) {
        // Stage s has landed once at most the RING - 2 stages after it are out;
        // past the barrier every wavefront has also read all of stage s - 1.
        stage_barrier<kLoads*(RING - 2)>();
#pragma unroll
        for (int h = 0; h < kSteps; ++h) {
            const int pieces = h == 0 ? kReads + kLoads : kReads;
#pragma unroll
            for (int m = 0; m < kMul; ++m) {
                if (h > 0 || s > 0)
                    multiply(h + 1, m);  // the step before this one
#pragma unroll
                for (int p = share(m, kMul, pieces); p < share(m + 1, kMul, pieces); ++p) {
                    if (p < kReads)
                        read(s, h, p);
                    else
                        issue(s + RING - 1, p - kReads);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    }
#pragma unroll
    for (int m = 0; m < kMul; ++m)
        multiply(1, m);
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
                const float4 sw = *reinterpret_cast<const float4*>(scale_v + wv + at_v);
                const float z[4] = {static_cast<float>(acc[i][j][4 * e]) * sa * sw.x,
                                    static_cast<float>(acc[i][j][4 * e + 1]) * sa * sw.y,
                                    static_cast<float>(acc[i][j][4 * e + 2]) * sa * sw.z,
                                    static_cast<float>(acc[i][j][4 * e + 3]) * sa * sw.w};
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

template <int TV, int TN, int WV, int WN, int BK, int RING>
hipError_t launch_tile(int rows, int depth, int cols, const int8_t* a, const float* a_scale,
                       const int8_t* w, const float* w_scale, int out_dtype, void* out, hipStream_t s) {
    const long tiles_v = (static_cast<long>(cols) + TV - 1) / TV;
    const long tiles_n = (static_cast<long>(rows) + TN - 1) / TN;
    if (tiles_v * tiles_n >= (1L << 32) / (64 * WV * WN))
        return hipErrorInvalidValue;
    const dim3 grid(static_cast<unsigned>(tiles_v * tiles_n)), block(64 * WV * WN);
    if (out_dtype == SPEC_BF16)
        int8_product_kernel<TV, TN, WV, WN, BK, RING, kBF16><<<grid, block, 0, s>>>(
            a, a_scale, w, w_scale, rows, depth, cols, static_cast<int>(tiles_n),
            static_cast<int>(tiles_v * tiles_n), out);
    else
        int8_product_kernel<TV, TN, WV, WN, BK, RING, kF32><<<grid, block, 0, s>>>(
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
    auto tiles = [&](long tv, long tn) { return ((cols + tv - 1) / tv) * ((rows + tn - 1) / tn); };
    // The largest tile that still gives the chip about enough workgroups
    // (microseconds at D = 4096, V = 152064 unless another V and D stand there):
    //   256 x 256, a workgroup per CU: 512 rows 325 (128 x 128: 404), 128 rows 197
    //     (172); 512 rows of V = 32000, D = 2048, 250 tiles, 39 (47), of V = 8192,
    //     64 tiles, 44 (128 x 64, 512 tiles: 25);
    //   128 x 128: 128 rows 172 (128 x 64: 182); 256 rows of V = 32000, D = 2048,
    //     500 tiles, 27 (37);
    //   128 x 64: 64 rows 149 (64 x 32: 160); of V = 32000, D = 2048, 250 tiles,
    //     17.3 (15.6);
    //   64 x 32: 1 row 127 (128 x 64: 132), 16 rows of V = 8192 13.0 (20.2).
    hipError_t e;
#define SPEC_TILE(...) \
    e = launch_tile<__VA_ARGS__>(rows, depth, cols, a, a_scale, w, w_scale, out_dtype, out, s)
    if (rows > 128 && tiles(256, 256) >= 224)
        SPEC_TILE(256, 256, 2, 4, 128, 2);
    else if (rows > 64 && tiles(128, 128) >= 448)
        SPEC_TILE(128, 128, 2, 2, 128, 2);
    else if (rows > 32 && tiles(128, 64) >= 400)
        SPEC_TILE(128, 64, 4, 1, 128, 2);
    else
        SPEC_TILE(64, 32, 2, 1, 128, 3);
#undef SPEC_TILE
    return e == hipSuccess ? SPEC_OK : e == hipErrorInvalidValue ? SPEC_EINVAL : SPEC_EHIP;
}

}  // extern "C"
