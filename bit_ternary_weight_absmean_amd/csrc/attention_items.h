// What the attention kernels share: element types, and the work items that every workgroup derives from the
// sequences' lengths.
#pragma once

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "attention.h"
#include "bt_internal.h"
#include "convert.h"
#include "wave.h"

namespace bt {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef __attribute__((address_space(3))) void lds_void;

constexpr int kUnit = 64;             // keys: granularity of the key slices
constexpr float kLn2 = 0.69314718055994530942f;
constexpr int kBufferWord3 = 0x00020000;
constexpr uint32_t kOutside = 0x7FFFFFF0u;  // a buffer offset past every record

template <typename E>
struct Elem;
template <>
struct Elem<bf16_t> {
    typedef bf16_t v8 __attribute__((ext_vector_type(8)));
    typedef bf16_t v2 __attribute__((ext_vector_type(2)));
    static constexpr uint32_t kExp = 0x7F80u;
    static constexpr float kRise = 8.0f;    // exponent by which a maximum may rise without rescaling
    static constexpr float kRaised = 0.0f;  // exponent of the probabilities at the reference
    static constexpr float kLower = 1.0f;   // 2^-kRaised
    static __device__ f32x16 mma32(v8 a, v8 b, f32x16 c)
    {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
    }
    static __device__ f32x4 mma16(v8 a, v8 b, f32x4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
};
template <>
struct Elem<f16_t> {
    typedef f16_t v8 __attribute__((ext_vector_type(8)));
    typedef f16_t v2 __attribute__((ext_vector_type(2)));
    static constexpr uint32_t kExp = 0x7C00u;
    static constexpr float kRise = 6.0f;
    static constexpr float kRaised = 9.0f;
    static constexpr float kLower = 1.0f / 512.0f;
    static __device__ f32x16 mma32(v8 a, v8 b, f32x16 c)
    {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
    }
    static __device__ f32x4 mma16(v8 a, v8 b, f32x4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
};

typedef float f32x2 __attribute__((ext_vector_type(2)));

// Two values rounded to E, packed.
template <typename E>
__device__ inline uint32_t pack2(float a, float b)
{
    const f32x2 f = {a, b};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, typename Elem<E>::v2));
}
template <typename E>
__device__ inline f32x2 unpack2(uint32_t p)
{
    return __builtin_convertvector(__builtin_bit_cast(typename Elem<E>::v2, p), f32x2);
}

// Does a pair of E values hold an infinity or NaN?
template <typename E>
__device__ inline bool pair_not_finite(uint32_t p)
{
    constexpr uint32_t e = Elem<E>::kExp;
    return (p & e) == e || (p >> 16 & e) == e;
}

// A pair of E values with infinities and NaNs set to 0.
template <typename E>
__device__ inline uint32_t finite_part(uint32_t p)
{
    constexpr uint32_t e = Elem<E>::kExp;
    return ((p & e) == e ? 0u : p & 0xFFFFu) | ((p >> 16 & e) == e ? 0u : p & 0xFFFF0000u);
}

__device__ inline float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

__device__ inline float other_half(float v)  // the value of lane ^ 32
{
    const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float((threadIdx.x & 32) ? p[0] : p[1]);
}

// op over the lanes l % 16 of the wave, in every lane
template <typename Op>
__device__ inline float across_quarters(float v, Op op)
{
    const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = op(__uint_as_float(p[0]), __uint_as_float(p[1]));
    const auto q = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return op(__uint_as_float(q[0]), __uint_as_float(q[1]));
}

// ---------------------------------------------------------------------------- work items

struct Seq {
    int q0, nq, k0, nk;
};

// Sequence b, its rows and keys kept inside the arrays whatever the offsets say. Of keys in pages, k0 is
// the sequence's number (its row of the table) and S what a row of the table can hold.
template <typename Args>
__device__ inline Seq load_seq(const Args &a, int b)
{
    Seq s = {0, 0, 0, 0};
    if (a.shared) {  // the shared prefix: every token's rows over the prefix keys
        s.nq = a.T;
        s.nk = a.P;
        return s;
    }
    s.q0 = min(max(a.q_start[b], 0), a.T);
    s.nq = min(max(a.q_start[b + 1], s.q0), a.T) - s.q0;
    if constexpr (Args::kPaged) {
        s.k0 = b;
        s.nk = min(max(a.k_len[b], 0), a.S);
    } else {
        s.k0 = min(max(a.k_start[b], 0), a.S);
        s.nk = min(max(a.k_len[b], 0), a.S - s.k0);
    }
    return s;
}

struct Item {
    Seq s;
    int tile;           // row tile of the sequence
    int piece, pieces;  // key slice and their number
    int unit;           // units (of kUnit keys) of a slice
    int base;           // first item of the sequence
};

// Inclusive sum over the wave's lanes, without LDS: within rows of 16 by row shifts, then the last
// lane of a row (of two rows) added to the rows behind it.
template <int CTRL, int ROWS>
__device__ inline int shifted_in(int v)
{
    return __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, false);
}
__device__ inline int wave_scan(int v)
{
    v += shifted_in<0x111, 0xF>(v);  // row_shr:1, 2, 4, 8
    v += shifted_in<0x112, 0xF>(v);
    v += shifted_in<0x114, 0xF>(v);
    v += shifted_in<0x118, 0xF>(v);
    v += shifted_in<0x142, 0xA>(v);  // row_bcast:15 into rows 1 and 3
    v += shifted_in<0x143, 0xC>(v);  // row_bcast:31 into rows 2 and 3
    return v;
}

template <typename Args>
__device__ inline int row_tiles(const Args &a, const Seq &s, int bm)
{
    return (int)(((int64_t)s.nq * a.G + bm - 1) / bm);
}

__device__ inline int key_units(const Seq &s) { return (s.nk + kUnit - 1) / kUnit; }

// Units per slice so that the items of all sequences are about `target` per key head.
template <typename Args>
__device__ inline int slice_units(const Args &a, int bm, const Seq &mine, int nseq)
{
    if (a.target == 0)
        return 1 << 30;
    const int lane = threadIdx.x & 63;
    float work = lane < nseq ? (float)row_tiles(a, mine, bm) * (float)key_units(mine) : 0.f;
    for (int c = 64; c < nseq; c += 64)
        if (c + lane < nseq) {
            const Seq s = load_seq(a, c + lane);
            work += (float)row_tiles(a, s, bm) * (float)key_units(s);
        }
    work = __uint_as_float(wave_reduce_bits(__float_as_uint(work), [](uint32_t x, uint32_t y) {
        return __float_as_uint(__uint_as_float(x) + __uint_as_float(y));
    }));
    const float per = ceilf(work / (float)a.target);
    return max(a.min_units, (int)fminf(per, 1e9f));
}

__device__ inline int pieces_of(const Seq &s, int unit) { return max(1, (key_units(s) + unit - 1) / unit); }

// Item `id` (of one key head), or tile `id` when `by_tile`; false: there are fewer.
template <typename Args>
__device__ inline bool find_item(const Args &a, int bm, int id, bool by_tile, Item &it)
{
    const int lane = threadIdx.x & 63;
    const int nseq = a.shared ? 1 : a.B;
    if (nseq == 1) {  // nothing to search
        it.s = load_seq(a, 0);
        it.base = 0;
        const int n = row_tiles(a, it.s, bm);
        const float work = (float)n * (float)key_units(it.s);
        it.unit = a.target ? max(a.min_units, (int)fminf(ceilf(work / (float)a.target), 1e9f)) : 1 << 30;
        it.pieces = pieces_of(it.s, it.unit);
        it.tile = by_tile ? id : n - 1 - id / it.pieces;
        it.piece = by_tile ? 0 : id % it.pieces;
        return it.tile >= 0 && it.tile < n;
    }
    Seq mine = {0, 0, 0, 0};
    if (lane < nseq)
        mine = load_seq(a, lane);
    it.unit = uniform(slice_units(a, bm, mine, nseq));
    int tiles_before = 0, items_before = 0;
    for (int c = 0; c < nseq; c += 64) {
        if (c)
            mine = c + lane < nseq ? load_seq(a, c + lane) : Seq{0, 0, 0, 0};
        const int tiles = row_tiles(a, mine, bm), items = tiles * pieces_of(mine, it.unit);
        const int ti = wave_scan(tiles), ii = wave_scan(items);
        const int key = by_tile ? tiles_before + ti : items_before + ii;
        const uint64_t past = __ballot(key > id);
        if (past) {
            const int l = __builtin_ctzll(past);
            it.s.q0 = __builtin_amdgcn_readlane(mine.q0, l);
            it.s.nq = __builtin_amdgcn_readlane(mine.nq, l);
            it.s.k0 = __builtin_amdgcn_readlane(mine.k0, l);
            it.s.nk = __builtin_amdgcn_readlane(mine.nk, l);
            it.base = items_before + __builtin_amdgcn_readlane(ii - items, l);
            const int tbase = tiles_before + __builtin_amdgcn_readlane(ti - tiles, l);
            it.pieces = uniform(pieces_of(it.s, it.unit));
            const int n = row_tiles(a, it.s, bm);
            if (by_tile) {
                it.tile = id - tbase;
                it.piece = 0;
            } else {
                // later tiles of a prompt see more keys: they come first
                it.tile = n - 1 - (id - it.base) / it.pieces;
                it.piece = (id - it.base) % it.pieces;
            }
            return true;
        }
        tiles_before += __builtin_amdgcn_readlane(ti, 63);
        items_before += __builtin_amdgcn_readlane(ii, 63);
    }
    return false;
}

// The item index of slice 0 of a tile (see find_item).
template <typename Args>
__device__ inline int first_item(const Args &a, const Item &it, int bm)
{
    return it.base + (row_tiles(a, it.s, bm) - 1 - it.tile) * it.pieces;
}

// Keys that row r of a sequence sees: [0, limit).
template <typename Args>
__device__ inline int row_limit(const Args &a, const Seq &s, int token)
{
    return a.causal ? max(0, s.nk - s.nq + token + 1) : s.nk;
}

// 16-byte chunk of a row's chunk c in LDS. Rows of 16 chunks or more: sixteen successive rows put
// their chunk c in sixteen places (the S^T operand reads a column of 32 rows), and four successive
// rows put theirs in different groups of four (the V^T operand reads 64 bytes of four rows at once).
// Rows of eight chunks lie two to a 256-byte line, and do the same with one bit less.
template <int DP>
__device__ inline int swizzle(int row)
{
    return DP >= 128 ? ((row & 3) << 2 | (row >> 2 & 3)) : ((row >> 1 & 1) << 2 | (row >> 2 & 3));
}

}  // namespace
}  // namespace bt
