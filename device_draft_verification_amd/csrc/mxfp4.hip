// Quantisation of rows to 4-bit floating point with a scale for every 32
// entries, and the product of two matrices so quantised (spec_mxfp4.h):
//
//   e = floor(log2 max |x|) - 2, code = e2m1(x / 2^e);
//   out[n][v] = sum_b 2^(ea + ew) sum_{k in block b} a[n][k] w[v][k].
#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "common.hpp"
#include "spec_mxfp4.h"
#include "stage.hpp"

namespace specv {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 __attribute__((aligned(2))) u32x4_any;  // rows of an odd length start at any element

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// ------------------------------------------------------------ quantisation ---

// The larger of a lane's value and that of another lane of its four (CTRL: the
// permutation, two bits a lane).
template <int CTRL>
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
    const uint32_t o = __builtin_amdgcn_mov_dpp(v, CTRL, 0xF, 0xF, true);
    return o > v ? o : v;
}

// v, or'ed over the 16 lanes of a row of lanes that are 4 or 8 places apart.
__device__ __forceinline__ uint32_t row_or(uint32_t v) {
    v |= __builtin_amdgcn_mov_dpp(v, 0x124, 0xF, 0xF, true);  // row_ror:4
    v |= __builtin_amdgcn_mov_dpp(v, 0x128, 0xF, 0xF, true);  // row_ror:8
    return v;
}

// Eight entries of a row, as a lane holds them: four pairs of bf16, or eight fp32.
template <int DT>
struct Eight {
    static constexpr int WORDS = DT == kBF16 ? 4 : 8;
    static constexpr int ESZ = DT == kBF16 ? 2 : 4;
    uint32_t w[WORDS];

    __device__ __forceinline__ void load(const char* at) {
#pragma unroll
        for (int i = 0; i < WORDS / 4; ++i) {
            const u32x4 v = reinterpret_cast<const u32x4_any*>(at)[i];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                w[4 * i + j] = v[j];
        }
    }
    // The first n entries of them, zeros behind.
    __device__ __forceinline__ void load_first(const char* at, int n) {
#pragma unroll
        for (int i = 0; i < WORDS; ++i)
            w[i] = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < n) {
                if constexpr (DT == kBF16)
                    w[e >> 1] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(at)[e]) << (16 * (e & 1));
                else
                    w[e] = reinterpret_cast<const uint32_t*>(at)[e];
            }
    }
    // The largest magnitude's bits, as binary32: without a sign the order of floats
    // is that of their bits, and a NaN or infinity comes out on top.
    __device__ __forceinline__ uint32_t largest() const {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < WORDS; ++i) {
            if constexpr (DT == kBF16) {
                const uint32_t hi = w[i] & 0x7FFF0000u, lo = (w[i] << 16) & 0x7FFF0000u;
                m = max(m, max(hi, lo));
            } else {
                m = max(m, w[i] & 0x7FFFFFFFu);
            }
        }
        return m;
    }
    // Their codes over the scale, the first entry lowest: the conversion rounds to
    // nearest, ties to even, and saturates.
    __device__ __forceinline__ uint32_t codes(float scale) const {
        uint32_t r = 0;
        if constexpr (DT == kBF16) {
            r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2, w[0]), scale, 0);
            r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2, w[1]), scale, 1);
            r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2, w[2]), scale, 2);
            r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2, w[3]), scale, 3);
        } else {
            auto f = [&](int i) { return __uint_as_float(w[i]); };
            r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, f(0), f(1), scale, 0);
            r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, f(2), f(3), scale, 1);
            r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, f(4), f(5), scale, 2);
            r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, f(6), f(7), scale, 3);
        }
        return r;
    }
    // What codes stand for.
    __device__ __forceinline__ void values(uint32_t r, float scale) {
        if constexpr (DT == kBF16) {
            w[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(r, scale, 0));
            w[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(r, scale, 1));
            w[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(r, scale, 2));
            w[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(r, scale, 3));
        } else {
            auto put = [&](int i, f32x2 v) {
                w[i] = __float_as_uint(v.x);
                w[i + 1] = __float_as_uint(v.y);
            };
            put(0, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(r, scale, 0));
            put(2, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(r, scale, 1));
            put(4, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(r, scale, 2));
            put(6, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(r, scale, 3));
        }
    }
    __device__ __forceinline__ void fill(uint32_t v) {
#pragma unroll
        for (int i = 0; i < WORDS; ++i)
            w[i] = v;
    }
    __device__ __forceinline__ void store(char* at) const {
#pragma unroll
        for (int i = 0; i < WORDS / 4; ++i)
            reinterpret_cast<u32x4_any*>(at)[i] = u32x4{w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]};
    }
    __device__ __forceinline__ void store_first(char* at, int n) const {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < n) {
                if constexpr (DT == kBF16)
                    reinterpret_cast<uint16_t*>(at)[e] = static_cast<uint16_t>(w[e >> 1] >> (16 * (e & 1)));
                else
                    reinterpret_cast<uint32_t*>(at)[e] = w[e];
            }
    }
};

// A lane takes eight entries, four lanes a block, 16 blocks a wavefront, over all
// rows as one sequence (a padded row is a whole number of lanes' entries, 16 or
// more), so that codes go out as one stream.
template <int DT, bool VALUES>
__global__ __launch_bounds__(kBlock) void mxfp4_quantize_kernel(const void* x, int cols, uint32_t per_row,
                                                                uint32_t total, uint32_t* __restrict__ out_q,
                                                                uint32_t* __restrict__ out_scale, void* out_values) {
    using E = Eight<DT>;
    const uint32_t at = blockIdx.x * kBlock + threadIdx.x;
    if (at >= total)
        return;  // whole groups of 16 lanes: a row is a multiple of them
    const uint32_t row = at / per_row;
    const int k0 = static_cast<int>(at - row * per_row) * 8;
    const size_t offset = (static_cast<size_t>(row) * cols + k0) * E::ESZ;
    const char* src = static_cast<const char*>(x) + offset;
    const int left = cols - k0;  // entries of the row from here on
    E v;
    if (left >= 8)
        v.load(src);
    else
        v.load_first(src, left);
    uint32_t m = v.largest();
    m = quad_max<0xB1>(m);  // lanes 1 0 3 2
    m = quad_max<0x4E>(m);  // lanes 2 3 0 1
    const uint32_t field = m >> 23;  // exponent of the largest magnitude, plus 127
    const bool wild = field == 255;
    const uint32_t byte = wild ? 255u : field > 2 ? field - 2 : 0u;
    const float scale = __uint_as_float(byte << 23);  // its exponent is what the conversions look at
    const uint32_t r = wild ? 0u : v.codes(scale);
    out_q[at] = r;
    const uint32_t word = row_or(byte << (8 * (threadIdx.x >> 2 & 3)));
    if ((threadIdx.x & 15) == 0)
        out_scale[at >> 4] = word;
    if constexpr (VALUES) {
        if (left <= 0)
            return;
        if (wild)
            v.fill(DT == kBF16 ? 0x7FC07FC0u : 0x7FC00000u);
        else
            v.values(r, scale);
        char* to = static_cast<char*>(out_values) + offset;
        if (left >= 8)
            v.store(to);
        else
            v.store_first(to, left);
    }
}

// ----------------------------------------------------------------- product ---

// A workgroup of WV x WN wavefronts forms a TV (vocabulary) x TN (rows) tile of
// the output, each wavefront TV / WV x TN / WN as 32 x 32 tiles of
// v_mfma_scale_f32_32x32x64_f8f6f4, in which a lane holds one block of 32 codes
// (16 bytes) of its row and that block's scale. The vocabulary is the M side: a
// lane then holds runs of four consecutive outputs of one row.
//
// K in stages of BK bytes of codes through a ring of LDS slots, loaded straight
// into LDS RING - 1 stages ahead: one barrier per stage, after which the slot of
// the stage before is refilled. A slot holds TV + TN rows of BK bytes; a row's
// 16-byte chunks sit at positions XORed with the row's number in units of the
// banks' 256 bytes, so that the rows that a phase of a fragment read touches lie
// in different places. Behind them lie the rows' scales, BK / 16 bytes each.
// Which block of K an instruction multiplies is free as long as both sides agree:
// in a stage the lower half of the lanes takes the first half of the blocks, the
// upper half the second, so that a lane's scales of a stage are whole words.
// Rows past the end repeat the last one (their outputs are not stored), chunks
// and scales past the depth come from a page of zeros.
__device__ int4 zero_chunk;  // zero from load on, never written

// SIZE bytes a lane from memory into LDS, behind one another there.
template <int SIZE>
__device__ __forceinline__ void to_lds(const uint8_t* from, uint8_t* to) {
    static_assert(SIZE == 16 || SIZE == 4, "of the sizes that the loads know");
    if constexpr (SIZE == 16)
        __builtin_amdgcn_global_load_lds(reinterpret_cast<const void*>(from), to, 16, 0, 0);
    else
        __builtin_amdgcn_global_load_lds(reinterpret_cast<const void*>(from), to, 4, 0, 0);
}

template <int BYTE>
__device__ __forceinline__ f32x16 multiply_blocks(const i32x4& a, const i32x4& b, const f32x16& c, int sa, int sb) {
    const i32x8 x = __builtin_shufflevector(a, a, 0, 1, 2, 3, -1, -1, -1, -1);
    const i32x8 y = __builtin_shufflevector(b, b, 0, 1, 2, 3, -1, -1, -1, -1);
    // formats 4: e2m1; the scales' byte BYTE
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, y, c, 4, 4, BYTE, sa, BYTE, sb);
}

template <int TV, int TN, int WV, int WN, int BK, int OUT>
__global__ __launch_bounds__(64 * WV * WN, 2) void mxfp4_product_kernel(
    const uint8_t* __restrict__ a, const uint8_t* __restrict__ a_scale, const uint8_t* __restrict__ w,
    const uint8_t* __restrict__ w_scale, int rows, int depth, int cols, int tiles_n, int tiles,
    void* __restrict__ out) {
    constexpr int kWavesHere = WV * WN;
    constexpr int MV = TV / WV / 32, MN = TN / WN / 32;
    constexpr int kRows = TV + TN;
    constexpr int kChunks = BK / 16;                  // of a row in a slot
    constexpr int kRowsPerLoad = 64 / kChunks;        // a load covers 1 KiB
    constexpr int kLoads = kRows / kRowsPerLoad / kWavesHere;  // per wavefront and stage
    constexpr int kLoadsV = TV / kRowsPerLoad / kWavesHere;    // of them of the vocabulary
    constexpr int kWords = BK / 64;                   // of a row's scales of a stage
    constexpr int kPeriod = 4;                        // stages whose scales are loaded together
    constexpr int kRowWords = kWords * kPeriod;       // of a row's scales in LDS
    constexpr int kScaleLoads = kLoads / kPeriod;     // per wavefront and stage
    constexpr int kSlot = kRows * BK;
    constexpr int kScaleSlot = kRows * 4 * kRowWords;
    constexpr int kRing = 2 * kSlot;
    constexpr int kSteps = BK / 32;                   // of two blocks each
    static_assert(TV % (kRowsPerLoad * kWavesHere) == 0 && TN % (kRowsPerLoad * kWavesHere) == 0 &&
                      kLoads % kPeriod == 0, "every wavefront issues the same loads");
    static_assert(kRowWords == kChunks, "a load of scales covers the rows that one of codes does");
    static_assert(kSteps % 4 == 0 && 256 % BK == 0 && kWavesHere * kRowsPerLoad % (256 / BK * kChunks) == 0,
                  "two sets of fragments take turns, and a lane's place in its row is the same in all loads");
    auto swizzle = [](int row) { return row / (256 / BK) % kChunks; };
    // The epilogue turns a wavefront's 32 rows x 32 MV entries through LDS.
    constexpr int ESZ = OUT == kBF16 ? 2 : 4;
    constexpr int kRowBytes = 32 * MV * ESZ + 16;
    constexpr int kTurn = 32 * kRowBytes;
    constexpr int kLds = kRing + 2 * kScaleSlot > kWavesHere * kTurn ? kRing + 2 * kScaleSlot : kWavesHere * kTurn;
    __shared__ __align__(16) uint8_t lds[kLds];
    const int lane = threadIdx.x & 63;
    const int wid = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
    // Workgroups go round the eight XCDs: each XCD takes a contiguous run of
    // tiles, rows fastest, so that the tiles that share weights share an L2.
    const int blk = blockIdx.x, xcd = blk & 7, order = blk >> 3;
    const int per = tiles >> 3, extra = tiles & 7;
    const int tile = xcd * per + (xcd < extra ? xcd : extra) + order;
    const int v0 = tile / tiles_n * TV;
    const int n0 = tile % tiles_n * TN;
    const int bytes = depth / 2, words = depth / 128;  // of a row: codes, words of scales

    // Load i of a wavefront covers rows kRowsPerLoad * (wavefront + kWavesHere * i) and
    // on: of each this lane's row, as an offset from the tile's first (the scales' is
    // a sixteenth), and its chunk and word in it.
    const uint8_t* w_tile = w + static_cast<size_t>(v0) * bytes;
    const uint8_t* a_tile = a + static_cast<size_t>(n0) * bytes;
    const uint8_t* w_scale_tile = w_scale + static_cast<size_t>(v0) * (bytes / 16);
    const uint8_t* a_scale_tile = a_scale + static_cast<size_t>(n0) * (bytes / 16);
    const int first_row = wid * kRowsPerLoad + lane / kChunks;
    const uint32_t chunk = (lane % kChunks ^ swizzle(first_row)) * 16, word = lane % kRowWords;
    uint32_t row_at[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int row = first_row + kRowsPerLoad * kWavesHere * i;
        row_at[i] = static_cast<uint32_t>(i < kLoadsV ? min(row, cols - 1 - v0) : min(row - TV, rows - 1 - n0)) * bytes;
    }
    const int stages = (bytes + BK - 1) / BK;
    const uint8_t* zeros = reinterpret_cast<const uint8_t*>(&zero_chunk);
    asm volatile("" : "+s"(zeros));  // looked up once, not in every stage
    // Stages and periods past the end load zeros into places that nobody reads.
    auto issue = [&](int s, int i) {
        const int k = s * BK;
        const uint8_t* tile = (i < kLoadsV ? w_tile : a_tile) + k;
        uint8_t* to = lds + (s & 1) * kSlot + (wid + kWavesHere * i) * 1024;
        if (k + BK <= bytes)
            to_lds<16>(tile + (row_at[i] + chunk), to);
        else
            to_lds<16>(k + static_cast<int>(chunk) < bytes ? tile + (row_at[i] + chunk) : zeros, to);
    };
    // Load i of a period's scales.
    auto issue_scales = [&](int p, int i) {
        const int k = p * kRowWords;
        const uint8_t* tile = (i < kLoadsV ? w_scale_tile : a_scale_tile) + 4 * k;
        uint8_t* to = lds + kRing + (p & 1) * kScaleSlot + (wid + kWavesHere * i) * 256;
        if (k + kRowWords <= words)
            to_lds<4>(tile + (row_at[i] / 16 + 4 * word), to);
        else
            to_lds<4>(k + static_cast<int>(word) < words ? tile + (row_at[i] / 16 + 4 * word) : zeros, to);
    };
    constexpr int kIssues = kLoads + kScaleLoads;
    f32x16 acc[MV][MN];
#pragma unroll
    for (int i = 0; i < MV; ++i)
#pragma unroll
        for (int j = 0; j < MN; ++j)
            acc[i][j] = f32x16{};
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        issue_scales(0, i);
        issue(0, i);
    }
    const int wv = wid % WV * (TV / WV), wn = wid / WV * (TN / WN);
    const int frag_row = lane & 31, half = lane >> 5;
    const int swz = swizzle(frag_row);  // rows of a tile start at multiples of 32
    // A step (a block of either half) is multiplied while the next one's fragments
    // are read: of stage s - 1 the last step waits in registers over the barrier,
    // with its scales. Reads and loads go between the matrix instructions, in whose
    // shadow they issue.
    constexpr int kReads = MV + MN, kMul = MV * MN;
    constexpr int kHalfWords = kWords / 2;
    i32x4 fw[2][MV], fa[2][MN];
    int sw[2][kHalfWords][MV], sa[2][kHalfWords][MN];  // of this stage, and of the one before
    auto read = [&](int s, int step, int i) {
        const uint8_t* slot = lds + (s & 1) * kSlot;
        const int pos = ((half * kSteps + step) ^ swz) * 16;
        if (i < MN)
            fa[step & 1][i] = *reinterpret_cast<const i32x4*>(slot + (TV + wn + 32 * i + frag_row) * BK + pos);
        else
            fw[step & 1][i - MN] =
                *reinterpret_cast<const i32x4*>(slot + (wv + 32 * (i - MN) + frag_row) * BK + pos);
    };
    auto read_scales = [&](int s, int i) {
        const int* scales = reinterpret_cast<const int*>(lds + kRing + (s / kPeriod & 1) * kScaleSlot);
        const int row = i < MN ? TV + wn + 32 * i + frag_row : wv + 32 * (i - MN) + frag_row;
#pragma unroll
        for (int h = 0; h < kHalfWords; ++h) {
            const int v = scales[row * kRowWords + s % kPeriod * kWords + half * kHalfWords + h];
            if (i < MN)
                sa[0][h][i] = v;
            else
                sw[0][h][i - MN] = v;
        }
    };
    // The last step of stage s - 1 takes the older scales.
    auto multiply = [&](int step, int m, int old) {
        const int i = m / MN, j = m % MN, h = step / 4;
        const i32x4 &x = fw[step & 1][i], &y = fa[step & 1][j];
        const int p = sw[old][h][i], q = sa[old][h][j];
        switch (step & 3) {
            case 0: acc[i][j] = multiply_blocks<0>(x, y, acc[i][j], p, q); break;
            case 1: acc[i][j] = multiply_blocks<1>(x, y, acc[i][j], p, q); break;
            case 2: acc[i][j] = multiply_blocks<2>(x, y, acc[i][j], p, q); break;
            default: acc[i][j] = multiply_blocks<3>(x, y, acc[i][j], p, q); break;
        }
    };
    // Of `work` pieces spread over `steps` steps, the first of step n.
    auto share = [](int n, int steps, int work) { return (n * work + steps - 1) / steps; };
#pragma unroll 1
    for (int s0 = 0; s0 < stages; s0 += kPeriod)
#pragma unroll
    for (int j = 0; j < kPeriod; ++j) {
        const int s = s0 + j;
        if (s >= stages)
            break;
        // Stage s has landed; past the barrier every wavefront has also read all of
        // stage s - 1.
        stage_barrier<0>();
#pragma unroll
        for (int h = 0; h < kHalfWords; ++h) {
#pragma unroll
            for (int i = 0; i < MV; ++i)
                sw[1][h][i] = sw[0][h][i];
#pragma unroll
            for (int j = 0; j < MN; ++j)
                sa[1][h][j] = sa[0][h][j];
        }
#pragma unroll
        for (int h = 0; h < kSteps; ++h) {
            const int pieces = h == 0 ? 2 * kReads + kIssues : kReads;
#pragma unroll
            for (int m = 0; m < kMul; ++m) {
                if (h > 0)
                    multiply(h - 1, m, 0);
                else if (s > 0)
                    multiply(kSteps - 1, m, 1);
#pragma unroll
                for (int p = share(m, kMul, pieces); p < share(m + 1, kMul, pieces); ++p) {
                    if (p < kReads)
                        read(s, h, p);
                    else if (p < 2 * kReads)
                        read_scales(s, p - kReads);
                    else if (p < 2 * kReads + kLoads)
                        issue(s + 1, p - 2 * kReads);
                    else
                        issue_scales(s / kPeriod + 1, p - 2 * kReads - kLoads + kScaleLoads * j);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    }
#pragma unroll
    for (int m = 0; m < kMul; ++m)
        multiply(kSteps - 1, m, 0);
    // No load may still be on its way into LDS when it is used again.
    stage_barrier<0>();

    // Lane l holds entries 8 (e / 4) + 4 (l / 32) + e % 4 of row l % 32 of a
    // 32 x 32 tile. Turned through LDS (each wavefront in its own part), they go
    // out as 16-byte stores along the rows.
    uint8_t* turn = lds + wid * kTurn;
    const bool whole = (static_cast<size_t>(cols) * ESZ) % 16 == 0 &&
                       (reinterpret_cast<uintptr_t>(out) & 15) == 0;
#pragma unroll
    for (int j = 0; j < MN; ++j) {
        const int nb = n0 + wn + 32 * j;
#pragma unroll
        for (int i = 0; i < MV; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int at_v = 32 * i + 8 * e + 4 * half;
                const float z[4] = {acc[i][j][4 * e], acc[i][j][4 * e + 1], acc[i][j][4 * e + 2],
                                    acc[i][j][4 * e + 3]};
                uint8_t* to = turn + (lane & 31) * kRowBytes + at_v * ESZ;
                if constexpr (OUT == kBF16)
                    *reinterpret_cast<uint2*>(to) = make_uint2(
                        __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{z[0], z[1]}, bf16x2)),
                        __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{z[2], z[3]}, bf16x2)));
                else
                    *reinterpret_cast<float4*>(to) = make_float4(z[0], z[1], z[2], z[3]);
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

template <int TV, int TN, int WV, int WN, int BK>
hipError_t launch_tile(int rows, int depth, int cols, const uint8_t* a, const uint8_t* a_scale,
                       const uint8_t* w, const uint8_t* w_scale, int out_dtype, void* out, hipStream_t s) {
    const long tiles_v = (static_cast<long>(cols) + TV - 1) / TV;
    const long tiles_n = (static_cast<long>(rows) + TN - 1) / TN;
    if (tiles_v * tiles_n >= (1L << 32) / (64 * WV * WN))
        return hipErrorInvalidValue;
    const dim3 grid(static_cast<unsigned>(tiles_v * tiles_n)), block(64 * WV * WN);
    if (out_dtype == SPEC_BF16)
        mxfp4_product_kernel<TV, TN, WV, WN, BK, kBF16><<<grid, block, 0, s>>>(
            a, a_scale, w, w_scale, rows, depth, cols, static_cast<int>(tiles_n),
            static_cast<int>(tiles_v * tiles_n), out);
    else
        mxfp4_product_kernel<TV, TN, WV, WN, BK, kF32><<<grid, block, 0, s>>>(
            a, a_scale, w, w_scale, rows, depth, cols, static_cast<int>(tiles_n),
            static_cast<int>(tiles_v * tiles_n), out);
    return hipGetLastError();
}

}  // namespace
}  // namespace specv

using namespace specv;

extern "C" {

int spec_mxfp4_quantize_rows(int rows, int cols, int dtype, const void* x, uint8_t* out_q,
                             uint8_t* out_scale, void* out_values, void* hip_stream) {
    if (rows < 0 || cols < 1 || (dtype != SPEC_F32 && dtype != SPEC_BF16))
        return SPEC_EINVAL;
    if (rows == 0)
        return SPEC_OK;
    const size_t esz = dtype == SPEC_BF16 ? 2 : 4;
    if (!x || !out_q || !out_scale || !aligned(x, esz) || !aligned(out_q, 4) || !aligned(out_scale, 4) ||
        (out_values && !aligned(out_values, esz)))
        return SPEC_EINVAL;
    const long per_row = (static_cast<long>(cols) + 127) / 128 * 16;  // lanes of a row
    if (per_row > ((1L << 32) - kBlock) / rows)
        return SPEC_EINVAL;
    if (out_values && out_values != x) {
        const uintptr_t p = reinterpret_cast<uintptr_t>(x), q = reinterpret_cast<uintptr_t>(out_values);
        const uintptr_t n = static_cast<uintptr_t>(rows) * cols * esz;
        if (p < q + n && q < p + n)
            return SPEC_EINVAL;
    }
    const long total = rows * per_row;
    const dim3 grid(static_cast<unsigned>((total + kBlock - 1) / kBlock)), block(kBlock);
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
#define SPEC_QUANTIZE(DT, VALUES)                                                                       \
    mxfp4_quantize_kernel<DT, VALUES><<<grid, block, 0, s>>>(                                           \
        x, cols, static_cast<uint32_t>(per_row), static_cast<uint32_t>(total),                          \
        reinterpret_cast<uint32_t*>(out_q), reinterpret_cast<uint32_t*>(out_scale), out_values)
    if (dtype == SPEC_BF16) {
        if (out_values)
            SPEC_QUANTIZE(kBF16, true);
        else
            SPEC_QUANTIZE(kBF16, false);
    } else {
        if (out_values)
            SPEC_QUANTIZE(kF32, true);
        else
            SPEC_QUANTIZE(kF32, false);
    }
#undef SPEC_QUANTIZE
    return hipGetLastError() == hipSuccess ? SPEC_OK : SPEC_EHIP;
}

int spec_mxfp4_product(int rows, int depth, int cols, const uint8_t* a, const uint8_t* a_scale,
                       const uint8_t* w, const uint8_t* w_scale, int out_dtype, void* out,
                       void* hip_stream) {
    if (rows < 0 || cols < 1 || depth < 128 || depth % 128 != 0 || depth > SPEC_MXFP4_MAX_DEPTH ||
        (out_dtype != SPEC_F32 && out_dtype != SPEC_BF16))
        return SPEC_EINVAL;
    if (rows == 0)
        return SPEC_OK;
    if (!a || !a_scale || !w || !w_scale || !out || !aligned(a, 16) || !aligned(w, 16) ||
        !aligned(a_scale, 4) || !aligned(w_scale, 4) || !aligned(out, out_dtype == SPEC_BF16 ? 2 : 4))
        return SPEC_EINVAL;
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    auto tiles = [&](long tv, long tn) { return ((cols + tv - 1) / tv) * ((rows + tn - 1) / tn); };
    hipError_t e;
#define SPEC_TILE(...) \
    e = launch_tile<__VA_ARGS__>(rows, depth, cols, a, a_scale, w, w_scale, out_dtype, out, s)
    if (rows > 128 && tiles(256, 256) >= 224)
        SPEC_TILE(256, 256, 2, 4, 128);
    else if (rows > 64 && tiles(128, 128) >= 448)
        SPEC_TILE(128, 128, 2, 2, 128);
    else
        SPEC_TILE(64, 64, 2, 1, 128);
#undef SPEC_TILE
    return e == hipSuccess ? SPEC_OK : e == hipErrorInvalidValue ? SPEC_EINVAL : SPEC_EHIP;
}

}  // extern "C"
