// Quantisation of rows to 4-bit floating point with a scale for every 32
// entries, and the product of two matrices so quantised (spec_mxfp4.h):
//
//   e = floor(log2 max |x|) - 2, code = e2m1(x / 2^e);
//   out[n][v] = sum_b 2^(ea + ew) sum_{k in block b} a[n][k] w[v][k].
#include <hip/hip_runtime.h>

#include <algorithm>
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

// The exponent comes from the largest magnitude's bits; the conversion instructions
// scale, round to nearest even and saturate. Bound by memory: 152064 x 4096 bf16 with
// their values in place take 454 us, 6.2 TB/s, the rate of a large copy, without values
// 256; 2304 x 4001 fp32, whose rows start anywhere, 13.5 us with values, 76032 x 4096
// fp32 252 without.
//
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

// A workgroup of WV x WN wavefronts forms TV (vocabulary) x TN (rows) tiles of
// the output, each wavefront TV / WV x TN / WN as 32 x 32 tiles of
// v_mfma_scale_f32_32x32x64_f8f6f4, in which a lane holds one block of 32 codes
// (16 bytes) of its row and that block's scale. The vocabulary is the M side: a
// lane then holds runs of four consecutive outputs of one row.
//
// K in stages of BK bytes of codes through RING LDS slots, loaded straight into
// LDS RING - 1 stages ahead (a tile has as many at least): one barrier per stage,
// after which the slot of the stage before is filled again. A slot holds TV + TN
// rows of BK bytes; a row's 16-byte chunks sit at positions XORed with the row's
// number, so that the rows that a phase of a fragment read touches lie in different
// banks. Scales come for four stages at a time: a row's 8 bytes of a stage would
// cost as many requests as its 128 bytes of codes. Which block of K an instruction
// multiplies is free as long as both sides agree: in a stage the lower half of the
// lanes takes the first half of the blocks, the upper half the second, so that a
// lane's scales of a stage are a word. Rows past the end repeat the last one (their
// outputs are not stored), scales past the depth come from a page of zeros.
//
// Workgroups stay for several tiles; the first loads of the next one run through
// the epilogue, which turns the outputs in LDS so that stores are whole lines.
//
// With many rows a stage of 256 x 256 is a chain of its loads, a barrier, reads of 192
// KB from LDS (a quarter of the cycles) and the matrix instructions (45 % of them):
// 2304 x 152064 outputs at depth 4096 take 780-815 us, 3.6 PFLOP/s, where a loop of
// nothing but these instructions reaches 6.1 to 6.8 on such data (the clock falls under
// their power) and the kernel without its loads took 557 to 570. Few rows are bound by the read of the weights
// and its latency: 64 x 152064 at depth 4096 take 79 us, 4.4 TB/s, 1 x 152064 60 us,
// 5.5 TB/s, 1 x 32000 14 us, 5 TB/s. Slower: stages of half the length and four
// slots 860 us (then 810), 4 wavefronts of 128 x 128 each, alone on their SIMDs, 885.
// Weights straight into registers, the rows whole in LDS: 85 us for 64 x 152064.
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

template <int TV, int TN, int WV, int WN, int RING, int OUT>
__global__ __launch_bounds__(64 * WV * WN, RING > 2 ? 1 : 2) void mxfp4_product_kernel(
    const uint8_t* __restrict__ a, const uint8_t* __restrict__ a_scale, const uint8_t* __restrict__ w,
    const uint8_t* __restrict__ w_scale, int rows, int depth, int cols, int tiles_n, int tiles,
    void* __restrict__ out) {
    constexpr int kWavesHere = WV * WN;
    constexpr int MV = TV / WV / 32, MN = TN / WN / 32;
    constexpr int kRows = TV + TN;
    constexpr int BK = 128;                           // bytes of a row's codes in a stage
    constexpr int kLoads = kRows / 8 / kWavesHere;    // per wavefront and stage: a load covers 8 rows
    constexpr int kLoadsV = TV / 8 / kWavesHere;      // of them of the vocabulary
    constexpr int kPeriod = 4;                        // stages whose scales are loaded together: a word
    constexpr int kRowWords = 2 * kPeriod;            // of scales for 64 bytes of codes
    constexpr int kAhead = RING - 1;                  // stages that loads run ahead
    // Scales' loads are out by the stage of a period from which on they may not have
    // landed by its end: per wavefront and stage, at most.
    constexpr int kScaleStages = kPeriod + 1 - kAhead;
    constexpr int kScaleLoads = (kLoads + kScaleStages - 1) / kScaleStages;
    constexpr int kSlot = kRows * BK;
    constexpr int kScaleSlot = kRows * 4 * kRowWords;
    constexpr int kSteps = BK / 32;                   // of two blocks each
    static_assert(TV % (8 * kWavesHere) == 0 && TN % (8 * kWavesHere) == 0,
                  "every wavefront issues the same loads");
    static_assert(kWavesHere % 2 == 0, "a lane's chunk is the same in all loads");
    // Loads find a row of a tile by a 24-bit multiplication, in 32 bits.
    constexpr long kMostBytes = SPEC_MXFP4_MAX_DEPTH / 2;
    static_assert(kMostBytes < 1L << 24 && (TV > TN ? TV : TN) * kMostBytes <= 1L << 32,
                  "a tile's offsets stay inside the multiplication and its word");
    // The epilogue turns 32 rows of up to 128 bytes of a wavefront's outputs through LDS
    // at a time, in the slot of the last stage.
    constexpr int ESZ = OUT == kBF16 ? 2 : 4;
    constexpr int kTurnV = MV == 1 ? 1 : 128 / ESZ / 32;  // fragments of the vocabulary at a time
    constexpr int kTurnBytes = 32 * kTurnV * ESZ, kRowBytes = kTurnBytes + 16;
    constexpr int kTurn = 32 * kRowBytes;
    static_assert(MV % kTurnV == 0 && kWavesHere * kTurn <= kSlot, "outputs turn inside a slot");
    // One LDS object: with two the compiler keeps their accesses apart by alias
    // scopes, and then waits for every load into LDS before any read of it.
    __shared__ __align__(16) uint8_t lds[RING * kSlot + 2 * kScaleSlot];
    const int lane = threadIdx.x & 63;
    const int wid = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
    const int bytes = depth / 2, words = depth / 128;  // of a row: codes, words of scales
    const int stages = (bytes + BK - 1) / BK;
    const int wv = wid % WV * (TV / WV), wn = wid / WV * (TN / WN);
    const int frag_row = lane & 31, half = lane >> 5;

    // Workgroups go round the eight XCDs: each XCD takes a contiguous run of tiles,
    // rows fastest, so that the tiles that share weights share an L2; its workgroups
    // go through the run together.
    const int xcd = blockIdx.x & 7;
    const int per = tiles >> 3, extra = tiles & 7;
    const int run_end = (xcd + 1) * per + (xcd + 1 < extra ? xcd + 1 : extra);
    const int stride = (static_cast<int>(gridDim.x) - xcd + 7) >> 3;
    int tile = xcd * per + (xcd < extra ? xcd : extra) + static_cast<int>(blockIdx.x >> 3);

    // Of a tile: its first row and entry, and the last ones' numbers in it.
    struct Tile {
        int v0, n0, last_v, last_n;
    };
    auto tile_at = [&](int t) {
        const int v0 = t / tiles_n * TV, n0 = t % tiles_n * TN;
        return Tile{v0, n0, cols - 1 - v0, rows - 1 - n0};
    };
    // Load i of a wavefront covers rows 8 (wavefront + kWavesHere * i) and on; a row's
    // 16-byte chunks and its words of scales lie at positions XORed with the row's number,
    // so that what the lanes read together lies in different banks.
    const int first_row = wid * 8 + lane / 8;
    const uint32_t chunk = (lane % 8 ^ first_row / 2 % 8) * 16;
    const uint8_t* zeros = reinterpret_cast<const uint8_t*>(&zero_chunk);
    asm volatile("" : "+s"(zeros));  // looked up once, not in every stage
    auto row_of = [&](const Tile& t, int i) {
        const int row = first_row + 8 * kWavesHere * i;
        return static_cast<uint32_t>(i < kLoadsV ? min(row, t.last_v) : min(row - TV, t.last_n));
    };
    // Load i of stage s of tile t, into slot `slot`. Chunks past the depth are the row's
    // last one again: their scales are 2^-127 on either side, and make them nothing.
    auto issue = [&](const Tile& t, int s, int i, int slot) {
        const uint8_t* from = i < kLoadsV ? w + static_cast<size_t>(t.v0) * bytes : a + static_cast<size_t>(t.n0) * bytes;
        const uint32_t at = __umul24(row_of(t, i), bytes) + min(s * BK + static_cast<int>(chunk), bytes - 16);
        to_lds<16>(from + at, lds + slot * kSlot + (wid + kWavesHere * i) * 1024);
    };
    // Load i of the scales of period p of tile t, zeros past the depth.
    auto issue_scales = [&](const Tile& t, int p, int i, int slot) {
        const uint8_t* from = i < kLoadsV ? w_scale + static_cast<size_t>(t.v0) * words * 4
                                          : a_scale + static_cast<size_t>(t.n0) * words * 4;
        const int word = p * kRowWords + static_cast<int>(lane % 8 ^ (wid + kWavesHere * i) % 4 * 2);
        const uint32_t at = __umul24(row_of(t, i), words * 4) + 4 * word;
        to_lds<4>(word < words ? from + at : zeros, lds + RING * kSlot + slot * kScaleSlot + (wid + kWavesHere * i) * 256);
    };
    f32x16 acc[MV][MN];
    // A step (a block of either half) is multiplied while the next one's fragments
    // are read: of stage s - 1 the last step waits in registers over the barrier,
    // with its scales. Reads and loads go between the matrix instructions, in whose
    // shadow they issue.
    constexpr int kReads = MV + MN, kMul = MV * MN;
    i32x4 fw[2][MV], fa[2][MN];
    int sw[2][MV], sa[2][MN];  // scales of this stage, and of the one before
    const int swz = frag_row / 2 % 8;  // rows of a tile start at multiples of 32
    auto read = [&](int slot, int step, int i) {
        const uint8_t* at = lds + slot * kSlot + ((half * kSteps + step) ^ swz) * 16 + frag_row * BK;
        if (i < MN)
            fa[step & 1][i] = *reinterpret_cast<const i32x4*>(at + (TV + wn + 32 * i) * BK);
        else
            fw[step & 1][i - MN] = *reinterpret_cast<const i32x4*>(at + (wv + 32 * (i - MN)) * BK);
    };
    auto read_scales = [&](int slot, int j, int i) {
        const uint8_t* at = lds + RING * kSlot + slot * kScaleSlot + ((2 * j + half) ^ frag_row / 8 * 2) * 4 +
                            frag_row * (4 * kRowWords);
        if (i < MN)
            sa[0][i] = *reinterpret_cast<const int*>(at + (TV + wn + 32 * i) * (4 * kRowWords));
        else
            sw[0][i - MN] = *reinterpret_cast<const int*>(at + (wv + 32 * (i - MN)) * (4 * kRowWords));
    };
    // The last step of stage s - 1 takes the older scales.
    auto multiply = [&](int step, int m, int old) {
        const int i = m / MN, j = m % MN;
        const i32x4 &x = fw[step & 1][i], &y = fa[step & 1][j];
        const int p = sw[old][i], q = sa[old][j];
        switch (step) {
            case 0: acc[i][j] = multiply_blocks<0>(x, y, acc[i][j], p, q); break;
            case 1: acc[i][j] = multiply_blocks<1>(x, y, acc[i][j], p, q); break;
            case 2: acc[i][j] = multiply_blocks<2>(x, y, acc[i][j], p, q); break;
            default: acc[i][j] = multiply_blocks<3>(x, y, acc[i][j], p, q); break;
        }
    };
    // Of `work` pieces spread over `steps` steps, the first of step n.
    auto share = [](int n, int steps, int work) { return (n * work + steps - 1) / steps; };
    constexpr int kPieces = 2 * kReads + kLoads + kScaleLoads;

    Tile cur = tile_at(tile);
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
        issue_scales(cur, 0, i, 0);
#pragma unroll
    for (int s = 0; s < kAhead; ++s)
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            issue(cur, s, i, s);
    constexpr int kYounger = kLoads * (RING - 2);  // loads that may be out when a stage begins
    stage_barrier<kYounger>();
    int slot = 0, scale_slot = 0;  // of the stage and the period at hand
    auto in_ring = [](int s) { return s >= RING ? s - RING : s; };
#pragma unroll 1
    for (;;) {
        tile += stride;
        const bool more = tile < run_end;
        const Tile next = more ? tile_at(tile) : cur;
#pragma unroll
        for (int i = 0; i < MV; ++i)
#pragma unroll
            for (int j = 0; j < MN; ++j)
                acc[i][j] = f32x16{};
#pragma unroll 1
        for (int s0 = 0; s0 < stages; s0 += kPeriod) {
#pragma unroll 1
            for (int j = 0; j < kPeriod; ++j) {
                const int s = s0 + j;
                if (s >= stages)
                    break;
                // Stage s has landed; past the barrier every wavefront has also read all of
                // stage s - 1. (The first one's is the barrier before.)
                if (s > 0) {
                    stage_barrier<kYounger>();
                    slot = in_ring(slot + 1);
                }
                const bool last = s + 1 == stages, over = s + kAhead >= stages;
                const int ahead = over ? s + kAhead - stages : s + kAhead, ahead_slot = in_ring(slot + kAhead);
#pragma unroll
                for (int i = 0; i < MV; ++i)
                    sw[1][i] = sw[0][i];
#pragma unroll
                for (int i = 0; i < MN; ++i)
                    sa[1][i] = sa[0][i];
#pragma unroll
                for (int h = 0; h < kSteps; ++h) {
                    const int pieces = h == 0 ? kPieces : kReads;
#pragma unroll
                    for (int m = 0; m < kMul; ++m) {
                        if (h > 0)
                            multiply(h - 1, m, 0);
                        else if (s > 0)
                            multiply(kSteps - 1, m, 1);
#pragma unroll
                        for (int p = share(m, kMul, pieces); p < share(m + 1, kMul, pieces); ++p) {
                            if (p < kReads)
                                read(slot, h, p);
                            else if (p < 2 * kReads)
                                read_scales(scale_slot, j, p - kReads);
                            else if (p < 2 * kReads + kLoads)
                                issue(over ? next : cur, ahead, p - 2 * kReads, ahead_slot);
                            else if (const int i = p - 2 * kReads - kLoads + kScaleLoads * j;
                                     kLoads == kScaleLoads * kPeriod || i < kLoads)
                                // of the period behind, or the next tile's first
                                issue_scales(s0 + kPeriod < stages ? cur : next, s0 + kPeriod < stages ? s0 / kPeriod + 1 : 0,
                                             i, scale_slot ^ 1);
                        }
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
                if (last && j < kPeriod - 1) {  // the shares of stages that this tile does not have
#pragma unroll 1
                    for (int i = kScaleLoads * (j + 1); i < kLoads; ++i)
                        issue_scales(next, 0, i, scale_slot ^ 1);
                }
            }
            scale_slot ^= 1;
        }
#pragma unroll
        for (int m = 0; m < kMul; ++m)
            multiply(kSteps - 1, m, 0);
        // The next tile's first stage and scales have landed, and the last stage's slot is free.
        if (stages % kPeriod == 0)
            stage_barrier<kYounger>();
        else  // its scales may be what was asked for last
            stage_barrier<0>();

        // Lane l holds entries 8 (e / 4) + 4 (l / 32) + e % 4 of row l % 32 of a
        // 32 x 32 tile. Turned through LDS (each wavefront in its own part), they go
        // out as 16-byte stores along the rows, which nobody waits for before the next
        // tile's second stage.
        uint8_t* turn = lds + slot * kSlot + wid * kTurn;
        const bool whole = (static_cast<size_t>(cols) * ESZ) % 16 == 0 && (reinterpret_cast<uintptr_t>(out) & 15) == 0;
#pragma unroll
        for (int j = 0; j < MN; ++j) {
            const int nb = cur.n0 + wn + 32 * j;
#pragma unroll
            for (int i0 = 0; i0 < MV; i0 += kTurnV) {
#pragma unroll
                for (int i = 0; i < kTurnV; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const f32x16& f = acc[i0 + i][j];
                        const float z[4] = {f[4 * e], f[4 * e + 1], f[4 * e + 2], f[4 * e + 3]};
                        uint8_t* to = turn + frag_row * kRowBytes + (32 * i + 8 * e + 4 * half) * ESZ;
                        if constexpr (OUT == kBF16)
                            *reinterpret_cast<uint2*>(to) = make_uint2(
                                __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{z[0], z[1]}, bf16x2)),
                                __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{z[2], z[3]}, bf16x2)));
                        else
                            *reinterpret_cast<float4*>(to) = make_float4(z[0], z[1], z[2], z[3]);
                    }
                wave_order();
                constexpr int kEntries = 32 * kTurnV;
                const int vb = cur.v0 + wv + 32 * i0;
                if (whole) {
                    constexpr int kPer = 16 / ESZ, kLanes = kTurnBytes / 16;  // entries per store, lanes per row
#pragma unroll
                    for (int t = 0; t < kLanes / 2; ++t) {
                        const int r = t * (64 / kLanes) + lane / kLanes, c = lane % kLanes * kPer;
                        const uint4 x = *reinterpret_cast<const uint4*>(turn + r * kRowBytes + c * ESZ);
                        if (nb + r < rows && vb + c < cols)
                            *reinterpret_cast<uint4*>(static_cast<char*>(out) +
                                                      (static_cast<size_t>(nb + r) * cols + vb + c) * ESZ) = x;
                    }
                } else {
                    using elem_t = typename std::conditional<OUT == kBF16, uint16_t, uint32_t>::type;
                    for (int r = 0; r < 32 && nb + r < rows; ++r)
                        if (lane < kEntries && vb + lane < cols)
                            static_cast<elem_t*>(out)[static_cast<size_t>(nb + r) * cols + vb + lane] =
                                *reinterpret_cast<const elem_t*>(turn + r * kRowBytes + lane * ESZ);
                }
                wave_order();
            }
        }
        if (!more) {
            if constexpr (RING > 2)  // no load into LDS is out when the workgroup ends
                stage_barrier<0>();
            return;
        }
        cur = next;
        slot = in_ring(slot + 1);
        lds_barrier();  // all outputs have left LDS
    }
}

template <int TV, int TN, int WV, int WN, int RING, int PER_CU>
hipError_t launch_tile(int rows, int depth, int cols, const uint8_t* a, const uint8_t* a_scale,
                       const uint8_t* w, const uint8_t* w_scale, int out_dtype, void* out, hipStream_t s) {
    const long tiles_v = (static_cast<long>(cols) + TV - 1) / TV;
    const long tiles_n = (static_cast<long>(rows) + TN - 1) / TN;
    if (tiles_v * tiles_n > (1L << 31) - 4096)  // a workgroup counts on to its next tile
        return hipErrorInvalidValue;
    // Workgroups stay for several tiles: as many as the chip holds at a time.
    const dim3 grid(static_cast<unsigned>(std::min(tiles_v * tiles_n, 256L * PER_CU))), block(64 * WV * WN);
    if (out_dtype == SPEC_BF16)
        mxfp4_product_kernel<TV, TN, WV, WN, RING, kBF16><<<grid, block, 0, s>>>(
            a, a_scale, w, w_scale, rows, depth, cols, static_cast<int>(tiles_n),
            static_cast<int>(tiles_v * tiles_n), out);
    else
        mxfp4_product_kernel<TV, TN, WV, WN, RING, kF32><<<grid, block, 0, s>>>(
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
    // The larger the tile, the less of the codes goes through LDS for a product, but the
    // fewer workgroups there are and the more rows may be empty. Measured at a depth of 4096
    // (us; the rule's side first): 256 against 128 with 196 tiles of 256 (256 rows, 50000
    // entries) 44 : 56, with 158 (512, 20000) 37 : 44; 128 against 256 with 125 (192, 32000)
    // 30 : 36. 128 against 64 with 250 tiles of 128 (128, 32000) 25 : 28; 64 against 128 with
    // 157 (100, 20011, depth 1024) 7.8 : 9.4, and with 64 rows and 152064 entries 83 : 82.
    // 64 against 32 with 33 rows and 32000 entries 21.5 : 23.0, with 64 and 152064 83 : 93;
    // 32 against 64 with 32 rows 20.8 : 21.6, and with 152064 entries 69.8 : 74.7.
    // The small ones at depths that are worth it have four or five slots and half as many
    // workgroups on a compute unit: 64 rows of 20000, 32000, 152064 entries 14.7 : 18.6,
    // 18.8 : 22.0, 79.1 : 83.5, at a depth of 1024 32000 entries 7.5 : 7.4; 1 row of 32000
    // 14.8 : 19.2, of 152064 59.6 : 62.5, 8 rows of 32000 at depths of 3200, 2304, 2048
    // 14.1 : 17.2, 9.6 : 10.2, 9.1 : 9.0. (Of 128, on one workgroup, 128 x 152064 92 : 91.)
    // The rule counts tiles, not the rounds that workgroups go through them, nor rows that
    // a tile leaves empty; with 152064 entries (its side, then the next ones): 96 rows 128
    // 87, 256 110, 64 111; 160 rows 256 116, 128 122; 192 119 : 127; 256 126 : 138; 400
    // 187 : 216; 512 197 : 240; 1024 377 : 463; but 300 rows 177 : 170.
    const bool deep = depth > 2048;
    if (rows > 128 && tiles(256, 256) >= 144)
        SPEC_TILE(256, 256, 2, 4, 2, 1);
    else if (rows > 64 && tiles(128, 128) >= 224)
        SPEC_TILE(128, 128, 2, 2, 2, 2);
    else if (rows > 32)
        deep ? SPEC_TILE(64, 64, 1, 2, 4, 2) : SPEC_TILE(64, 64, 1, 2, 2, 4);
    else
        deep ? SPEC_TILE(64, 32, 2, 1, 5, 2) : SPEC_TILE(64, 32, 2, 1, 2, 5);
#undef SPEC_TILE
    return e == hipSuccess ? SPEC_OK : e == hipErrorInvalidValue ? SPEC_EINVAL : SPEC_EHIP;
}

}  // extern "C"
