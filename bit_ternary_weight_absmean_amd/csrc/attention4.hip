// Attention over a cache held in 4 bits, in pages (bt_attention4): single tokens, drafts of a few tokens and
// prompts, whole or continued, whose keys and values lie in the cache (csrc/cache4.h).
//
//   s[r, j] = scale * q_r . K_j over the keys j that row r sees;  out_r = sum_j softmax(s)_j V_j;
//   lse_r = ln sum_j exp(s[r, j])      (no key seen: out 0, lse -inf)
//
// One pass over the keys with a running maximum and sum per row, rows of (token, head of the group), transposed
// products, items, slices and their joining as in csrc/attention.hip.
//
// Types. A code with its scale is exactly a bf16, one conversion for two of them, so both products run on bf16
// operands: K is exact, a bf16 query is exact, an fp16 query is two bf16 (its 11 bits are 8 and 3) and two products.
// Probabilities are carried as a bf16 and its rest (16 bits), and a second rest for fp32 outputs (24 bits), in every form,
// so that a sequence's precision does not depend on what it is batched with. (One bf16 alone would save tiles with bf16
// outputs half of the second product, 14% of a long prompt, and add as much error as the outputs' own rounding: 7B
// prompts behind cached keys 0.0020 of the outputs' size against 64 bits, where rounding alone gives 0.0016, as two do.)
//
// Order of the values. A product's order of summation is free as long as both operands have it. Lane (r, g) of an S^T
// operand takes a key's group g, 16 bytes and one scale in one load each, as its part of the four steps of
// 128 values; the query operands are loaded to match.
//
// NaN. A group of K that holds a NaN makes the scores of its key NaN, which counts in rows that see it only (unseen
// scores are replaced). A group of V that holds one goes into the product as zeros, and rows that see its key get NaN
// in the group's values directly. Finite groups are finite in bf16, so there are no infinities to meet.
#include <stdio.h>

#include "attention_items.h"
#include "cache4.h"

namespace bt {
namespace {

using V8 = bf16x8;

// -------------------------------------------------------------------------- work items
//
// Items are those of csrc/attention_items.h. Where up to sixteen sequences fall to a lane, their lengths are loaded side by
// side and kept, instead of one wave's worth after the other, twice (300 decoding sequences over 300 to 1200 keys: 68.0 us,
// side by side 66.7). The tile's number among all sequences' goes with the item: its first slice notes for the joining
// where the tile's results lie, and the first item of all how many tiles there are.

struct Item4 : Item {
    int number;  // of the tile
};

// The fewest units of a slice by the longest sequence's: no more than about 48 slices of a tile, which the joining
// reads one behind the other (one token over 30000 keys in 118 slices: 29.5 us, in 59: 21.8), and four units where there
// are enough (8000 keys, two: 16.7 us, four: 13.4; 777 keys, two: 9.8, four: 10.7).
__device__ inline int slice_floor(int longest) { return max(longest / 48, min(4, longest / 6)); }

// What the joining needs of a tile: its first slot and slices, and its sequence's queries.
struct TileNote {
    int slot, pieces, tile, q0, nq, pad[3];
};
static_assert(sizeof(TileNote) == kNoteBytes, "room in the workspace");

template <int C>
__device__ inline bool find_among(const Attn4Args &a, int bm, int id, Item4 &it)
{
    const int lane = threadIdx.x & 63;
    Seq s[C];
    float work = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        s[c] = Seq{0, 0, 0, 0};
        if (64 * c + lane < a.B)
            s[c] = load_seq(a, 64 * c + lane);
    }
    it.unit = 1 << 30;
    if (a.target) {
#pragma unroll
        for (int c = 0; c < C; ++c)
            work += (float)row_tiles(a, s[c], bm) * (float)key_units(s[c]);
        work = __uint_as_float(wave_reduce_bits(__float_as_uint(work), [](uint32_t x, uint32_t y) {
            return __float_as_uint(__uint_as_float(x) + __uint_as_float(y));
        }));
        int longest = 0;
#pragma unroll
        for (int c = 0; c < C; ++c)
            longest = max(longest, key_units(s[c]));
        longest = (int)wave_reduce_bits((uint32_t)longest, [](uint32_t x, uint32_t y) { return x > y ? x : y; });
        it.unit = uniform(max(max(a.min_units, slice_floor(longest)), (int)fminf(ceilf(work / (float)a.target), 1e9f)));
    }
    int tiles_before = 0, items_before = 0;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int tiles = row_tiles(a, s[c], bm), items = tiles * pieces_of(s[c], it.unit);
        const int ti = wave_scan(tiles), ii = wave_scan(items);
        const uint64_t past = __ballot(items_before + ii > id);
        if (past) {
            const int l = __builtin_ctzll(past);
            it.s.q0 = __builtin_amdgcn_readlane(s[c].q0, l);
            it.s.nq = __builtin_amdgcn_readlane(s[c].nq, l);
            it.s.k0 = __builtin_amdgcn_readlane(s[c].k0, l);
            it.s.nk = __builtin_amdgcn_readlane(s[c].nk, l);
            it.base = items_before + __builtin_amdgcn_readlane(ii - items, l);
            it.pieces = uniform(pieces_of(it.s, it.unit));
            // later tiles of a prompt see more keys: they come first
            it.tile = row_tiles(a, it.s, bm) - 1 - (id - it.base) / it.pieces;
            it.piece = (id - it.base) % it.pieces;
            it.number = tiles_before + __builtin_amdgcn_readlane(ti - tiles, l) + it.tile;
            return true;
        }
        tiles_before += __builtin_amdgcn_readlane(ti, 63);
        items_before += __builtin_amdgcn_readlane(ii, 63);
    }
    return false;
}

__device__ inline bool find_item4(const Attn4Args &a, int bm, int id, Item4 &it)
{
    if (a.B <= 64)
        return find_among<1>(a, bm, id, it);
    if (a.B <= 256)
        return find_among<4>(a, bm, id, it);
    if (a.B <= 1024)
        return find_among<16>(a, bm, id, it);
    if (!find_item(a, bm, id, false, it))
        return false;
    int before = 0;
    for (int b = threadIdx.x & 63; b < it.s.k0; b += 64)
        before += row_tiles(a, load_seq(a, b), bm);
    it.number = wave_sum_i32(before) + it.tile;
    return true;
}

// Item `id` of key head `head`, and what the joining is told of it; false: there are fewer.
__device__ inline bool take_item(const Attn4Args &a, int bm, int id, int head, Item4 &it)
{
    TileNote *notes = reinterpret_cast<TileNote *>(a.notes);  // the first one: the number of tiles
    const bool found = find_item4(a, bm, id, it);
    if (a.target && head == 0 && threadIdx.x < 64) {
        if (id == 0) {
            int tiles = 0;
            float items = 0.f;
            for (int b = threadIdx.x; b < a.B; b += 64) {
                const Seq s = load_seq(a, b);
                const int n = row_tiles(a, s, bm);
                tiles += n;
                items += (float)n * (float)pieces_of(s, it.unit);
            }
            tiles = wave_sum_i32(tiles);
            items = __uint_as_float(wave_reduce_bits(__float_as_uint(items), [](uint32_t x, uint32_t y) {
                return __float_as_uint(__uint_as_float(x) + __uint_as_float(y));
            }));
            // (sequences that overlap may have more items than were launched: then some notes are not written, and nothing
            // is joined)
            if (threadIdx.x == 0)
                notes[0].pieces = items <= (float)a.items && tiles <= a.tiles ? tiles : 0;
        }
        if (found && it.piece == 0 && (uint32_t)it.number < (uint32_t)a.tiles && threadIdx.x == 0)
            notes[1 + it.number] = TileNote{first_item(a, it, bm), it.pieces, it.tile, it.s.q0, it.s.nq, {0, 0, 0}};
    }
    return found;
}

// A wave's view of a sequence's row of the table: 64 entries of it in the lanes.
struct PageWindow {
    const int *row;
    int used;   // entries that hold keys
    int first, mine;
};

__device__ inline PageWindow page_window(const Attn4Args &a, const Seq &s)
{
    PageWindow w;
    w.row = a.table + (int64_t)s.k0 * a.table_row;
    w.used = (int)(((int64_t)s.nk + (1 << a.page_shift) - 1) >> a.page_shift);
    w.first = -64;
    w.mine = -1;
    return w;
}

// Sixteen keys of one page from `key` (uniform): a buffer over their head's part of the page, of no bytes where there
// is no such page, and the tile's number in it.
struct Tile4 {
    __amdgpu_buffer_rsrc_t from;
    int tile;
    bool there;
};

__device__ inline Tile4 find_tile(const Attn4Args &a, PageWindow &w, int head, int key)
{
    const int p = key >> a.page_shift;
    int page = -1;
    if (p < w.used) {
        if ((uint32_t)(p - w.first) >= 64u) {
            const int at = p + (int)(threadIdx.x & 63);
            w.first = p;
            w.mine = at < w.used ? w.row[at] : -1;
        }
        page = __builtin_amdgcn_readlane(w.mine, p - w.first);
    }
    Tile4 t;
    t.there = page >= 0 && page < a.pages;
    t.tile = (key & ((1 << a.page_shift) - 1)) / kCacheTile;
    const char *base = a.cache + (t.there ? page * a.page_bytes : 0) + (int64_t)head * a.head_bytes;
    t.from = __builtin_amdgcn_make_buffer_rsrc(const_cast<char *>(base), (short)0, t.there ? a.head_bytes : 0,
                                               kBufferWord3);
    return t;
}

// What lane (r, g) holds of sixteen keys: key r's codes of DP / 4 values (from 32 g on; of 16 from 16 g on for
// DP == 64; for DP == 256 also from 128 + 32 g on), and their scale bytes.
template <int DP>
struct Codes4 {
    static constexpr int NB = DP > 128 ? 2 : 1, W = DP == 64 ? 2 : 4;  // pieces, words of a piece
    uint32_t k[NB][W], v[NB][W], ks[NB], vs[NB];
};

template <int DP>
struct Places4 {
    uint32_t code[Codes4<DP>::NB], scale[Codes4<DP>::NB];  // in the tile
};

template <int DP>
__device__ inline Places4<DP> lane_places(const Attn4Args &a)
{
    const int r = threadIdx.x & 15, g = threadIdx.x >> 4 & 3;
    Places4<DP> p;
#pragma unroll
    for (int n = 0; n < Codes4<DP>::NB; ++n) {
        const int group = DP == 64 ? g >> 1 : g + 4 * n;
        const bool in = group < a.groups;
        p.code[n] = in ? (uint32_t)((group * kCacheTile + r) * 16 + (DP == 64 ? 8 * (g & 1) : 0)) : kOutside;
        p.scale[n] = in ? (uint32_t)(group * kCacheTile + r) : kOutside;
    }
    return p;
}

// One piece of codes of a tile, K's or V's.
template <int W>
__device__ inline void load_codes(const __amdgpu_buffer_rsrc_t &from, uint32_t at, uint32_t (&x)[W])
{
    if constexpr (W == 4) {
        const u32x4 y = __builtin_amdgcn_raw_buffer_load_b128(from, at, 0, 0);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            x[j] = y[j];
    } else {
        const u32x2 y = __builtin_amdgcn_raw_buffer_load_b64(from, at, 0, 0);
        x[0] = y[0];
        x[1] = y[1];
    }
}

template <int DP>
__device__ inline void load_keys(const Attn4Args &a, const Places4<DP> &p, const Tile4 &t, Codes4<DP> &x)
{
    const uint32_t plane = (uint32_t)a.groups << a.page_shift, at = (uint32_t)(t.tile * a.groups * kCacheTile);
#pragma unroll
    for (int n = 0; n < Codes4<DP>::NB; ++n) {
        load_codes(t.from, p.code[n] + 16 * at, x.k[n]);
        x.ks[n] = __builtin_amdgcn_raw_buffer_load_b8(t.from, p.scale[n] + 32 * plane + at, 0, 0);
    }
}

template <int DP>
__device__ inline void load_values(const Attn4Args &a, const Places4<DP> &p, const Tile4 &t, Codes4<DP> &x)
{
    const uint32_t plane = (uint32_t)a.groups << a.page_shift, at = (uint32_t)(t.tile * a.groups * kCacheTile);
#pragma unroll
    for (int n = 0; n < Codes4<DP>::NB; ++n) {
        load_codes(t.from, p.code[n] + 16 * (plane + at), x.v[n]);
        x.vs[n] = __builtin_amdgcn_raw_buffer_load_b8(t.from, p.scale[n] + 33 * plane + at, 0, 0);
    }
}

// First value of step st of lane group g in the order of the S^T operands (see Codes4).
template <int DP>
__device__ inline int step_value(int g, int st)
{
    return DP == 64 ? 16 * g + 8 * st : 128 * (st / 4) + 32 * g + 8 * (st % 4);
}

// Eight query values as bf16, or as bf16 and their rests.
template <typename E>
__device__ inline void split_query(u32x4 x, V8 &hi, V8 &lo)
{
    if constexpr (sizeof(E) == 2 && Elem<E>::kRaised == 0.0f) {  // bf16
        hi = __builtin_bit_cast(V8, x);
        lo = hi;
    } else {
        const typename Elem<E>::v8 h = __builtin_bit_cast(typename Elem<E>::v8, x);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            hi[j] = (bf16_t)(float)h[j];
            lo[j] = (bf16_t)((float)h[j] - (float)hi[j]);
        }
    }
}

template <typename E>
constexpr bool kSplitQuery = sizeof(typename Elem<E>::v8) == 16 && Elem<E>::kRaised != 0.0f;

// The keys r < n of sixteen, as bits.
__device__ inline uint32_t first_bits(int n) { return n >= 16 ? 0xFFFFu : n <= 0 ? 0u : (1u << n) - 1; }

// ------------------------------------------------------------------------- prompt kernel
//
// attn4_tile: 32 rows per wave (32x32x16 MFMA) against a slice of the tile's keys, 64 at a time, as attn_tile of
// csrc/attention.hip has it: a vector phase from scores to probabilities, then a matrix phase of this block's product with
// V and the next block's scores; two buffers of K and of V in LDS, K one block ahead. A block's codes are loaded
// into registers (each wave 16 of its keys) while the one before them is used, and go to LDS as bf16, once for
// all of the tile's rows, beside that one's matrix phase.
//
// HALVES == 2, for calls whose tiles of 128 rows would not fill the CUs: 64 rows, and the waves of a pair take the two
// halves of every block's keys and are joined at the end.
//
// Bound by the matrix cores and the vector phase in turn, two waves a SIMD: a prompt of 8192 tokens of 32 heads of 128, bf16,
// 754 to 787 us (0.70 to 0.73 PFLOP/s of the formula's operations, 1.05 to 1.09 of the matrix cores', whose second product
// runs twice; a matrix product of 8192^3 reaches 1.39 on this card), fp16, where the first does too, 999 to 1029; 512 and
// 300 tokens of 32 heads over 4608 and 300 keys 76 to 78 us and 8 for the joining; 256 tokens of 20 heads of five groups
// over 8192 keys 43 to 48 and 8. Codes are converted once for 128 rows instead of once for 16, and a block is two
// barriers: with each wave converting the codes for its own rows the conversion took longer than both products.

constexpr int kTileRows = 128, kSmallRows = 64, kTileKeys = 64;

// Of the blocks in LDS: which 16-key tiles name no page (those of four blocks on end: K's are written two ahead of their
// use), and which keys have NaN groups (V's).
template <int DP>
struct BlockNotes {
    uint32_t gone[4][4];
    unsigned short nan[2][DP / 32][4];
};

template <typename E, int DP, bool WIDE, int HALVES>
__device__ __forceinline__ void attn4_tile(const Attn4Args &a, int block, char *kbuf0, char *kbuf1, char *vbuf0,
                                           char *vbuf1, BlockNotes<DP> *notes)
{
    constexpr int ROWS = kTileRows / HALVES, KB = 2 / HALVES;  // rows of the tile, 32-key parts per wave
    constexpr int NS = DP / 16, ND = DP / 32;                  // MFMA steps over D, 32-wide tiles of D
    constexpr int PARTS = WIDE ? 3 : 2;                        // of a probability
    using Codes = Codes4<DP>;
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int col = lane & 31, h = lane >> 5, r16 = lane & 15, g = lane >> 4;
    const int rg = HALVES == 2 ? wave & 1 : wave;        // the wave's 32 rows
    const int part0 = HALVES == 2 ? wave >> 1 : 0;       // its first 32-key part of a block
    const int id = block / a.Hkv, head = block % a.Hkv;
    Item4 it;
    if (!take_item(a, ROWS, id, head, it))
        return;
    const Seq s = it.s;

    // this lane's row
    const int rows = s.nq * a.G;
    const int row = it.tile * ROWS + 32 * rg + col;
    const int token = row / a.G, qh = head * a.G + row % a.G;
    const bool live = row < rows;
    const int limit = live ? row_limit(a, s, token) : 0;
    // the keys of the tile, and those that every live row of the wave sees
    const int last = min(rows, (it.tile + 1) * ROWS) - 1;
    const int lo = (int)min((int64_t)it.piece * it.unit * kUnit, (int64_t)s.nk);
    const int hi = min((int)min((int64_t)(it.piece + 1) * it.unit * kUnit, (int64_t)s.nk), row_limit(a, s, last / a.G));
    const int first = it.tile * ROWS + 32 * rg;
    const int wfull = first < rows ? row_limit(a, s, first / a.G) : 0;
    const int wmost = first < rows ? row_limit(a, s, min(rows - 1, first + 31) / a.G) : 0;

    // Q^T operands: lane (col, h) holds values 16 st + 8 h .. + 7 of its row
    V8 qf[NS], ql[NS];
    {
        const char *p = static_cast<const char *>(a.q) + 2 * ((int64_t)(s.q0 + token) * a.q_row + (int64_t)qh * a.q_head);
#pragma unroll
        for (int st = 0; st < NS; ++st) {
            u32x4 x = {0, 0, 0, 0};
            if (live && 16 * st + 8 * h < a.D)
                x = *reinterpret_cast<const u32x4 *>(p + 2 * (16 * st + 8 * h));
            split_query<E>(x, qf[st], ql[st]);
        }
    }
    const Places4<DP> places = lane_places<DP>(a);
    PageWindow kwindow = page_window(a, s), vwindow = kwindow;
    // the codes of this wave's 16 keys of a block of K and one of V, on their way
    Codes x;
    bool there = false;
    auto load_k = [&](int key) __attribute__((always_inline)) {
        if (key >= hi)
            return;
        const Tile4 t = find_tile(a, kwindow, head, key + 16 * wave);
        there = t.there;
        load_keys<DP>(a, places, t, x);
    };
    auto load_v = [&](int key) __attribute__((always_inline)) {
        if (key >= hi)
            return;
        load_values<DP>(a, places, find_tile(a, vwindow, head, key + 16 * wave), x);
    };
    // Their values to LDS as [key][D]: lane (r, g) has key r of the wave's tile, 32 values from chunk 4 g (16 from 2 g).
    auto store_k = [&](int key, char *kb) __attribute__((always_inline)) {
        if (key >= hi)
            return;
        const int r = 16 * wave + r16;
#pragma unroll
        for (int n = 0; n < Codes::NB; ++n)
#pragma unroll
            for (int w = 0; w < Codes::W; ++w) {
                const int c = Codes::W * (g + 4 * n) + w;
                *reinterpret_cast<u32x4 *>(kb + r * (DP * 2) + ((c ^ swizzle<DP>(r)) << 4)) =
                    __builtin_bit_cast(u32x4, cache_values(x.k[n][w], cache_scale(x.ks[n])));
            }
        if (lane == 0)
            notes->gone[key / kTileKeys & 3][wave] = !there;
    };
    // V: keys past the sequence's end hold anything: zeros; groups with NaNs: zeros, and noted
    auto store_v = [&](int key, char *vb) __attribute__((always_inline)) {
        if (key >= hi)
            return;
        const int r = 16 * wave + r16;
        const bool past = key + r >= s.nk;
#pragma unroll
        for (int n = 0; n < Codes::NB; ++n) {
            const bool bad = x.vs[n] > kCacheNaN, none = past || bad;
            const uint64_t nan = __ballot(bad && !past);
            const float f = cache_scale(none ? 0u : x.vs[n]);
#pragma unroll
            for (int w = 0; w < Codes::W; ++w) {
                const int c = Codes::W * (g + 4 * n) + w;
                *reinterpret_cast<u32x4 *>(vb + r * (DP * 2) + ((c ^ swizzle<DP>(r)) << 4)) =
                    __builtin_bit_cast(u32x4, cache_values(none ? 0u : x.v[n][w], f));
            }
            if (r16 == 0)
                notes->nan[key / kTileKeys & 1][DP == 64 ? g >> 1 : g + 4 * n][wave] = (unsigned short)(nan >> (16 * g));
        }
    };

    f32x16 o[ND];
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i)
            o[d][i] = 0.f;
    float m = -INFINITY, l = 0.f;  // l: this lane's keys only until the end
    const float c2 = a.scale_log2;

    // S^T of a block; register i of half b: key + 32 b + 8 (i / 4) + 4 h + i % 4
    f32x16 sc[KB];
    const int kbase = col * (DP * 2) + ((h ^ swizzle<DP>(col)) << 4);
    auto scores = [&](const char *kb) __attribute__((always_inline)) {
        kb += part0 * 32 * DP * 2;
#pragma unroll
        for (int b = 0; b < KB; ++b) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                sc[b][i] = 0.f;
#pragma unroll
            for (int st = 0; st < NS; ++st) {
                const char *at = kb + (kbase ^ (st << 5)) + b * 32 * DP * 2;
                const V8 k = __builtin_bit_cast(V8, *reinterpret_cast<const u32x4 *>(at));
                sc[b] = Elem<bf16_t>::mma32(k, qf[st], sc[b]);
                if constexpr (kSplitQuery<E>)
                    sc[b] = Elem<bf16_t>::mma32(k, ql[st], sc[b]);
            }
        }
    };
    // The vector phase: probabilities of the block, as P^T operands (slot j of step t is register
    // 8 (t % 2) + j of half t / 2).
    u32x4 pf[PARTS][2 * KB];
    auto soften = [&](int key) __attribute__((always_inline)) {
        const u32x4 gone = *reinterpret_cast<const u32x4 *>(notes->gone[key / kTileKeys & 3]);
        if (uniform(gone[0] | gone[1] | gone[2] | gone[3]) || key + kTileKeys > wfull) {
#pragma unroll
            for (int b = 0; b < KB; ++b)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (key + 32 * (part0 + b) + 8 * (i / 4) + 4 * h + i % 4 >= limit ||
                        (part0 ? gone[2 + i / 8] : gone[2 * b + i / 8]))
                        sc[b][i] = -INFINITY;
        }
        float mx = sc[0][0];
#pragma unroll
        for (int b = 0; b < KB; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                mx = fmaxf(mx, sc[b][i]);
        mx = fmaxf(mx, other_half(mx));
        if (__any((mx - m) * c2 > Elem<bf16_t>::kRise || (m == -INFINITY && mx > -INFINITY))) {
            const float mn = fmaxf(m, mx);
            const float f = mn == -INFINITY ? 1.f : exp2_fast((m - mn) * c2);
            l *= f;
#pragma unroll
            for (int d = 0; d < ND; ++d)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    o[d][i] *= f;
            m = mn;
        }
        const float ref = m == -INFINITY ? 0.f : m * c2;
        float lb = 0.f;
#pragma unroll
        for (int t = 0; t < 2 * KB; ++t)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float p[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    p[e] = exp2_fast(__builtin_fmaf(sc[t / 2][8 * (t % 2) + 2 * j + e], c2, -ref));
                    lb += p[e];
                }
#pragma unroll
                for (int q = 0; q < PARTS; ++q) {
                    pf[q][t][j] = pack2<bf16_t>(p[0], p[1]);
                    const f32x2 back = unpack2<bf16_t>(pf[q][t][j]);
                    p[0] -= back[0];
                    p[1] -= back[1];
                }
            }
        l += lb;
        // done here, not where they are used
        asm volatile("" : "+v"(l));
#pragma unroll
        for (int q = 0; q < PARTS; ++q)
#pragma unroll
            for (int t = 0; t < 2 * KB; ++t)
                asm volatile("" : "+v"(pf[q][t]));
    };
    // The matrix phase. V^T operands: lane i of 16 reads 8 bytes of row i / 4 of its 4 x 16 block of V. Row
    // 16 t + 8 j + tr_row is swizzled by that of tr_row, with bit 1 flipped by j.
    const int tr_row = 4 * h + (lane & 15) / 4, tr_col = (lane >> 4 & 1) * 32 + (lane & 3) * 8;  // bytes
    const int vbase = tr_row * (DP * 2) + (((tr_col >> 4) ^ swizzle<DP>(tr_row)) << 4) + (tr_col & 15);
    auto weigh = [&](int key, const char *vb) __attribute__((always_inline)) {
        vb += part0 * 32 * DP * 2;
        uint64_t any = 0;
#pragma unroll
        for (int d = 0; d < ND; ++d) {
            any |= *reinterpret_cast<const uint64_t *>(notes->nan[key / kTileKeys & 1][d]);
#pragma unroll
            for (int t = 0; t < 2 * KB; ++t) {
                u32x4 y;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const char *p = vb + (vbase ^ (d << 6) ^ (j << 5)) + (16 * t + 8 * j) * DP * 2;
                    const u32x2 half =
                        __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)p));
                    y[2 * j] = half[0];
                    y[2 * j + 1] = half[1];
                }
#pragma unroll
                for (int q = 0; q < PARTS; ++q)
                    o[d] = Elem<bf16_t>::mma32(__builtin_bit_cast(V8, y), __builtin_bit_cast(V8, pf[q][t]), o[d]);
            }
        }
        if (__builtin_expect(uniform((uint32_t)(any | any >> 32)), 0)) {
            const int n = limit - key;
            const uint64_t sees = n >= 64 ? ~0ull : n <= 0 ? 0ull : (1ull << n) - 1;
#pragma unroll
            for (int d = 0; d < ND; ++d)
                if (*reinterpret_cast<const uint64_t *>(notes->nan[key / kTileKeys & 1][d]) & sees)
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        o[d][i] = NAN;
        }
    };

    // End of a block: this wave's LDS operations are done; then all waves'.
    auto sync = [] {
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    };
    if (lo < hi) {
        load_k(lo);
        load_v(lo);
        store_k(lo, kbuf0);
        load_k(lo + kTileKeys);
        sync();
        scores(kbuf0);
        store_v(lo, vbuf0);
        store_k(lo + kTileKeys, kbuf1);
        load_k(lo + 2 * kTileKeys);
        load_v(lo + kTileKeys);
        sync();
        // K runs one block ahead of V; the last block's matrix phase forms scores from whatever the
        // other buffer holds, and they are not used.
        auto one = [&](int key, char *vb, char *kb, char *vnext, char *knext) __attribute__((always_inline)) {
            if (key < wmost)
                soften(key);
            store_k(key + 2 * kTileKeys, knext);
            store_v(key + kTileKeys, vnext);
            load_k(key + 3 * kTileKeys);
            load_v(key + 2 * kTileKeys);
            if (key < wmost) {
                scores(kb);
                weigh(key, vb);
            }
            sync();
        };
        for (int key = lo; key < hi; key += 2 * kTileKeys) {
            one(key, vbuf0, kbuf1, vbuf1, kbuf0);
            if (key + kTileKeys < hi)
                one(key + kTileKeys, vbuf1, kbuf0, vbuf0, kbuf1);
        }
    }
    l += other_half(l);
    __syncthreads();
    if constexpr (HALVES == 2) {
        // the second half's sums to the first half's waves
        float *sums = reinterpret_cast<float *>(rg ? kbuf1 : kbuf0), *stat = reinterpret_cast<float *>(vbuf0) + 64 * rg;
        if (part0) {
#pragma unroll
            for (int d = 0; d < ND; ++d)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    sums[(d * 16 + i) * 64 + lane] = o[d][i];
            stat[col] = m;
            stat[32 + col] = l;
        }
        __syncthreads();
        if (part0)
            return;
        const float m1 = stat[col], mn = fmaxf(m, m1);
        const float f0 = m == mn ? 1.f : exp2_fast((m - mn) * c2), f1 = m1 == mn ? 1.f : exp2_fast((m1 - mn) * c2);
        l = l * f0 + stat[32 + col] * f1;
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                o[d][i] = o[d][i] * f0 + sums[(d * 16 + i) * 64 + lane] * f1;
        m = mn;
    }
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);  // l NaN: NaN
    const float lse = l == 0.f ? -INFINITY : m * c2 * kLn2 + logf(l);
    if (!live)
        return;
    const bool part = it.pieces > 1;
    if (part) {
        const int64_t slot = block;
        const int r = 32 * rg + col;
        float *dst = a.ws_o + (slot * ROWS + r) * a.D;
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const int e = 32 * d + 8 * b + 4 * h;
                if (e < a.D) {
                    const float x[4] = {o[d][4 * b] * inv, o[d][4 * b + 1] * inv, o[d][4 * b + 2] * inv,
                                        o[d][4 * b + 3] * inv};
                    store4(dst + e, x);
                }
            }
        if (h == 0)
            a.ws_l[slot * ROWS + r] = lse;
        return;
    }
    const int64_t at = (int64_t)(s.q0 + token) * a.o_row + (int64_t)qh * a.o_head;
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const int e = 32 * d + 8 * b + 4 * h;
            if (e < a.D) {
                const float x[4] = {o[d][4 * b] * inv, o[d][4 * b + 1] * inv, o[d][4 * b + 2] * inv,
                                    o[d][4 * b + 3] * inv};
                if constexpr (WIDE)
                    store4(static_cast<float *>(a.out) + at + e, x);
                else
                    store4(static_cast<E *>(a.out) + at + e, x);
            }
        }
    if (a.lse && h == 0)
        a.lse[(int64_t)(s.q0 + token) * a.Hq + qh] = lse;
}

// -------------------------------------------------------------------- few-rows kernel
//
// attn4_few: 16 rows (a decode step's heads of one group, a short draft) against a slice of their keys; bound by
// the cache's bytes. Each of four waves takes every fourth block of 32 keys on its own. K's codes become S^T operands
// in their registers; V's go as bf16 through a private piece of LDS for the transposing read. The next block's
// loads are issued before this block is used; the four partial results are joined at the end.
//
// 64 tokens of 20 heads of 128 in five groups over 253 thousand keys (172 MB): 51 us, 3.4 TB/s, with nothing but its loads
// 47; pages of 16 tokens, whose numbers a wave has to read four times as often, take no longer (49). Part of it is the end,
// where not all CUs have work: 1140 workgroups of one length where 768 fit at once. Three blocks on their way, blocks of
// 64 keys, loads past the caches or more waves a CU: no gain. One token over 777 keys: 6.2 us, of which finding
// the item and the page are about three, and 3.7 for the joining.

constexpr int kFewRows = 16, kFewKeys = 32, kFewWaves = 4;

template <typename E, int DP, bool WIDE>
__device__ __forceinline__ void attn4_few(const Attn4Args &a, int block, char *buf,
                                          float (&stat)[kFewWaves][3][kFewRows])
{
    constexpr int NS = DP / 32, ND = DP / 16;
    constexpr int kVBytes = kFewKeys * DP * 2;
    using Codes = Codes4<DP>;
    static_assert(kVBytes >= kFewRows * DP * 4, "the waves' partial outputs reuse the V blocks");

    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int col = lane & 15, g = lane >> 4;
    const int id = block / a.Hkv, head = block % a.Hkv;
    Item4 it;
    if (!take_item(a, kFewRows, id, head, it))
        return;
    const Seq s = it.s;
    const int rows = s.nq * a.G;
    const int row = it.tile * kFewRows + col;
    const int token = row / a.G, qh = head * a.G + row % a.G;
    const bool live = row < rows;
    const int limit = live ? row_limit(a, s, token) : 0;
    const int first = it.tile * kFewRows, last = min(rows, first + kFewRows) - 1;
    const int lo = (int)min((int64_t)it.piece * it.unit * kUnit, (int64_t)s.nk);
    const int hi = min((int)min((int64_t)(it.piece + 1) * it.unit * kUnit, (int64_t)s.nk), row_limit(a, s, last / a.G));
    const int wfull = row_limit(a, s, first / a.G);

    V8 qf[NS], ql[NS];
    {
        const char *p = static_cast<const char *>(a.q) + 2 * ((int64_t)(s.q0 + token) * a.q_row + (int64_t)qh * a.q_head);
#pragma unroll
        for (int st = 0; st < NS; ++st) {
            u32x4 x = {0, 0, 0, 0};
            const int d = step_value<DP>(g, st);
            if (live && d < a.D)
                x = *reinterpret_cast<const u32x4 *>(p + 2 * d);
            split_query<E>(x, qf[st], ql[st]);
        }
    }
    const Places4<DP> places = lane_places<DP>(a);
    PageWindow window = page_window(a, s);
    struct Block {
        Codes t[2];
        bool there[2];
    };
    auto fetch = [&](int key, Block &x) __attribute__((always_inline)) {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const Tile4 t = find_tile(a, window, head, key + 16 * b);
            x.there[b] = t.there;
            load_keys<DP>(a, places, t, x.t[b]);
            load_values<DP>(a, places, t, x.t[b]);
        }
    };

    f32x4 o[ND];
#pragma unroll
    for (int d = 0; d < ND; ++d)
        o[d] = f32x4{0.f, 0.f, 0.f, 0.f};
    float m = -INFINITY, l = 0.f;
    const float c2 = a.scale_log2;
    char *vb = buf + wave * kVBytes;
    const int tr_row = 4 * g + (lane & 15) / 4, tr_col = (lane & 3) * 8;
    auto v_frag = [&](int dt) {
        u32x4 x;
#pragma unroll
        for (int jj = 0; jj < 2; ++jj) {
            const int r = 16 * jj + tr_row;
            const int byte = dt * 32 + tr_col;
            const char *p = vb + r * (DP * 2) + (((byte >> 4) ^ swizzle<DP>(r)) << 4) + (byte & 15);
            const u32x2 half = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)p));
            x[2 * jj] = half[0];
            x[2 * jj + 1] = half[1];
        }
        return __builtin_bit_cast(V8, x);
    };
    auto step = [&](int key, Block &x) __attribute__((always_inline)) {
        f32x4 sc[2];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            sc[b] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int st = 0; st < NS; ++st) {
                const int n = st / Codes::W;
                const V8 k = cache_values(x.t[b].k[n][st % Codes::W], cache_scale(x.t[b].ks[n]));
                sc[b] = Elem<bf16_t>::mma16(k, qf[st], sc[b]);
                if constexpr (kSplitQuery<E>)
                    sc[b] = Elem<bf16_t>::mma16(k, ql[st], sc[b]);
            }
        }
        // register i of block b: key + 16 b + 4 g + i
        if (key + kFewKeys > wfull || !x.there[0] || !x.there[1]) {
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (key + 16 * b + 4 * g + i >= limit || !x.there[b])
                        sc[b][i] = -INFINITY;
        }
        // V to LDS. Keys past the sequence's end hold anything: zeros. Groups with NaNs: zeros, and remembered.
        uint64_t nan[2][Codes::NB], any = 0;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const bool past = key + 16 * b + col >= s.nk;
            const int r = 16 * b + col;
#pragma unroll
            for (int n = 0; n < Codes::NB; ++n) {
                const bool bad = x.t[b].vs[n] > kCacheNaN;
                nan[b][n] = __ballot(bad && !past);
                any |= nan[b][n];
                const bool none = past || bad;
                const float f = cache_scale(none ? 0u : x.t[b].vs[n]);
#pragma unroll
                for (int w = 0; w < Codes::W; ++w) {
                    const int c = Codes::W * (g + 4 * n) + w;
                    const V8 y = cache_values(none ? 0u : x.t[b].v[n][w], f);
                    *reinterpret_cast<u32x4 *>(vb + r * (DP * 2) + ((c ^ swizzle<DP>(r)) << 4)) =
                        __builtin_bit_cast(u32x4, y);
                }
            }
        }
        float mx = fmaxf(fmaxf(fmaxf(sc[0][0], sc[0][1]), fmaxf(sc[0][2], sc[0][3])),
                         fmaxf(fmaxf(sc[1][0], sc[1][1]), fmaxf(sc[1][2], sc[1][3])));
        mx = across_quarters(mx, [](float x, float y) { return fmaxf(x, y); });
        if (__any((mx - m) * c2 > Elem<bf16_t>::kRise || (m == -INFINITY && mx > -INFINITY))) {
            const float mn = fmaxf(m, mx);
            const float f = mn == -INFINITY ? 1.f : exp2_fast((m - mn) * c2);
            l *= f;
#pragma unroll
            for (int d = 0; d < ND; ++d)
                o[d] *= f;
            m = mn;
        }
        const float ref = m == -INFINITY ? 0.f : m * c2;
        constexpr int PARTS = WIDE ? 3 : 2;
        u32x4 pf[PARTS];
        float lb = 0.f;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                sc[b][i] = exp2_fast(__builtin_fmaf(sc[b][i], c2, -ref));
                lb += sc[b][i];
            }
#pragma unroll
            for (int p = 0; p < PARTS; ++p)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    pf[p][2 * b + j] = pack2<bf16_t>(sc[b][2 * j], sc[b][2 * j + 1]);
                    const f32x2 back = unpack2<bf16_t>(pf[p][2 * b + j]);
                    sc[b][2 * j] -= back[0];
                    sc[b][2 * j + 1] -= back[1];
                }
        }
        l += lb;
        // This wave's LDS writes before its reads: LDS operations of a wave complete in order, so
        // only the compiler has to keep them so.
        asm volatile("" ::: "memory");
#pragma unroll
        for (int d = 0; d < ND; ++d) {
            const V8 v = v_frag(d);
#pragma unroll
            for (int p = 0; p < PARTS; ++p)
                o[d] = Elem<bf16_t>::mma16(v, __builtin_bit_cast(V8, pf[p]), o[d]);
        }
        asm volatile("" ::: "memory");
        if (__builtin_expect(any != 0, 0)) {
#pragma unroll
            for (int d = 0; d < ND; ++d) {
                // 16 values of group d / 2, in piece n of the lanes of quarter q
                const int n = DP > 128 ? d / 8 : 0, q = DP == 64 ? d & 2 : d / 2 % 4;
                uint32_t seen = 0;
#pragma unroll
                for (int b = 0; b < 2; ++b)
                    if (x.there[b])
                        seen |= (uint32_t)(nan[b][n] >> (16 * q)) & first_bits(limit - key - 16 * b);
                if (seen)
                    o[d] = f32x4{NAN, NAN, NAN, NAN};
            }
        }
    };

    constexpr int kStride = kFewWaves * kFewKeys;
    const int k0 = lo + wave * kFewKeys;
    if (k0 < hi) {
        Block x, y;
        fetch(k0, x);
        for (int key = k0; key < hi; key += 2 * kStride) {
            fetch(key + kStride, y);
            step(key, x);
            if (key + kStride >= hi)
                break;
            fetch(key + 2 * kStride, x);
            step(key + kStride, y);
        }
    }
    // join the four waves: common maximum, then the sums
    l = across_quarters(l, [](float x, float y) { return x + y; });
    if (g == 0) {
        stat[wave][0][col] = m;
        stat[wave][1][col] = l;
    }
    __syncthreads();
    float mall = stat[0][0][col];
#pragma unroll
    for (int w = 1; w < kFewWaves; ++w)
        mall = fmaxf(mall, stat[w][0][col]);
    float lall = 0.f;
#pragma unroll
    for (int w = 0; w < kFewWaves; ++w) {
        const float mw = stat[w][0][col];
        lall += mw == -INFINITY ? stat[w][1][col] : stat[w][1][col] * exp2_fast((mw - mall) * c2);  // 0, or NaN scores
    }
    const float inv = lall > 0.f ? 1.f / lall : (lall == 0.f ? 0.f : lall);
    const float f = m == -INFINITY ? inv : exp2_fast((m - mall) * c2) * inv;
    const float lse = lall == 0.f ? -INFINITY : mall * c2 * kLn2 + logf(lall);
    // wave's O^T to LDS as [row][D]: 4 values of row col per register group
    float *mine = reinterpret_cast<float *>(vb);
#pragma unroll
    for (int d = 0; d < ND; ++d) {
        const f32x4 x = l == 0.f ? f32x4{0.f, 0.f, 0.f, 0.f} : o[d] * f;
        *reinterpret_cast<f32x4 *>(mine + col * DP + ((4 * d + g) ^ (col & 7)) * 4) = x;
    }
    __syncthreads();
    const bool part = it.pieces > 1;
    for (int e = threadIdx.x; e < kFewRows * (DP / 4); e += 256) {
        const int r = e / (DP / 4), c = e % (DP / 4);
        const int rr = it.tile * kFewRows + r;
        if (rr >= rows || c * 4 >= a.D)
            continue;
        f32x4 sum = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < kFewWaves; ++w)
            sum += *reinterpret_cast<const f32x4 *>(reinterpret_cast<const float *>(buf + w * kVBytes) + r * DP +
                                                    (c ^ (r & 7)) * 4);
        const float x[4] = {sum[0], sum[1], sum[2], sum[3]};
        if (part) {
            store4(a.ws_o + ((int64_t)block * kFewRows + r) * a.D + 4 * c, x);
        } else {
            const int64_t at = (int64_t)(s.q0 + rr / a.G) * a.o_row + (int64_t)(head * a.G + rr % a.G) * a.o_head + 4 * c;
            if constexpr (WIDE)
                store4(static_cast<float *>(a.out) + at, x);
            else
                store4(static_cast<E *>(a.out) + at, x);
        }
    }
    if (wave == 0 && g == 0 && live) {
        if (part)
            a.ws_l[(int64_t)block * kFewRows + col] = lse;
        else if (a.lse)
            a.lse[(int64_t)(s.q0 + token) * a.Hq + qh] = lse;
    }
}

template <typename E, int DP, bool WIDE>
__global__ __launch_bounds__(256, DP > 128 ? 1 : 2) void k_attn4_few(Attn4Args a)
{
    __shared__ __attribute__((aligned(1024))) char buf[kFewWaves * kFewKeys * DP * 2];
    __shared__ float stat[kFewWaves][3][kFewRows];
    attn4_few<E, DP, WIDE>(a, blockIdx.x, buf, stat);
}

template <typename E, int DP, bool WIDE, int HALVES>
__global__ __launch_bounds__(256, DP > 128 ? 1 : 2) void k_attn4_tile(Attn4Args a)
{
    constexpr int bytes = kTileKeys * DP * 2;
    __shared__ __attribute__((aligned(1024))) char kbuf0[bytes], kbuf1[bytes], vbuf0[bytes], vbuf1[bytes];
    __shared__ __attribute__((aligned(16))) BlockNotes<DP> notes;
    attn4_tile<E, DP, WIDE, HALVES>(a, blockIdx.x, kbuf0, kbuf1, vbuf0, vbuf1, &notes);
}

// ------------------------------------------------------------------------------- joining
//
// k_attn4_join: a row's slices joined by their lse, out = sum_i w_i out_i / sum_i w_i with w_i = exp(lse_i - max), as
// k_attn_combine of csrc/attention.hip does, from the notes that the items left. Up to eight rows of a tile to a workgroup;
// fewer share its groups of lanes, four slices of each on their way at once. 3.7 us for one token's slices, 4.8 for those
// of 64 tokens, 8.5 for 812 tokens of 32 heads.

constexpr int kJoinGroups = 8;  // and the largest number of rows of a workgroup

template <typename TO>
__global__ __launch_bounds__(32 * kJoinGroups) void k_attn4_join(Attn4Args a, int bm)
{
    __shared__ f32x4 sums[kJoinGroups][2][32];
    __shared__ float stat[kJoinGroups][2];
    const int l32 = threadIdx.x & 31, group = threadIdx.x >> 5;
    const int id = blockIdx.x / a.Hkv, head = blockIdx.x % a.Hkv;
    const TileNote *notes = reinterpret_cast<const TileNote *>(a.notes);
    if (id >= notes[0].pieces)
        return;
    const TileNote tile = notes[1 + id];
    const int pieces = tile.pieces, slot = tile.slot;
    if (pieces == 1)
        return;  // written by its one item
    const int rows = tile.nq * a.G;
    const int r0 = blockIdx.y * kJoinGroups;
    const int here = min(min(bm - r0, kJoinGroups), rows - tile.tile * bm - r0);  // rows of this workgroup
    if (here <= 0)
        return;
    const int ways = 32 - __builtin_clz(2 * here - 1) - 1;  // log2 of here rounded up to a power of two
    const int gp = kJoinGroups >> ways;                              // groups of a row
    const int r = r0 + (group & ((1 << ways) - 1)), part = group >> ways;
    const int row = tile.tile * bm + r;
    const bool live = r < r0 + here;
    const int n = pieces;
    float m = -INFINITY, total = 0.f;
    f32x4 s0 = {0.f, 0.f, 0.f, 0.f}, s1 = s0;
    const int c0 = 4 * l32 < a.D ? 4 * l32 : 0, c1 = 128 + 4 * l32 < a.D ? 128 + 4 * l32 : 0;
    if (live)
        for (int i = part; i < n; i += 4 * gp) {
            float v[4];
            f32x4 x0[4], x1[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int j = min(i + u * gp, n - 1);
                const int64_t at = ((int64_t)(slot + j) * a.Hkv + head) * bm + r;
                const float *o = a.ws_o + at * a.D;
                v[u] = a.ws_l[at];
                x0[u] = *reinterpret_cast<const f32x4 *>(o + c0);
                if (a.D > 128)
                    x1[u] = *reinterpret_cast<const f32x4 *>(o + c1);
            }
            float mx = m;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                if (i + u * gp >= n) {  // the last slice again: not taken (0 * inf would be NaN)
                    v[u] = -INFINITY;
                    x0[u] = x1[u] = f32x4{0.f, 0.f, 0.f, 0.f};
                }
                mx = fmaxf(mx, v[u]);
            }
            const float ref = mx == -INFINITY ? 0.f : mx, f = expf(m - ref);
            total *= f;
            s0 *= f;
            s1 *= f;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const float w = expf(v[u] - ref);
                total += w;
                s0 += x0[u] * w;
                if (a.D > 128)
                    s1 += x1[u] * w;
            }
            m = mx;
        }
    if (gp > 1) {
        sums[group][0][l32] = s0;
        sums[group][1][l32] = s1;
        if (l32 == 0) {
            stat[group][0] = m;
            stat[group][1] = total;
        }
        __syncthreads();
        if (part)
            return;
        float mx = m;
        for (int q = 1; q < gp; ++q)
            mx = fmaxf(mx, stat[group + (q << ways)][0]);
        const float ref = mx == -INFINITY ? 0.f : mx, f = expf(m - ref);
        total *= f;
        s0 *= f;
        s1 *= f;
        for (int q = 1; q < gp; ++q) {
            const int g = group + (q << ways);
            const float w = expf(stat[g][0] - ref);
            total += stat[g][1] * w;
            s0 += sums[g][0][l32] * w;
            s1 += sums[g][1][l32] * w;
        }
        m = mx;
    }
    if (!live)
        return;
    const int token = row / a.G, qh = head * a.G + row % a.G;
    const int64_t at = (int64_t)(tile.q0 + token) * a.o_row + (int64_t)qh * a.o_head;
    const float inv = total == 0.f ? 0.f : 1.f / total;
    TO *dst = static_cast<TO *>(a.out) + at;
    if (4 * l32 < a.D) {
        const float y[4] = {s0[0] * inv, s0[1] * inv, s0[2] * inv, s0[3] * inv};
        store4(dst + 4 * l32, y);
    }
    if (128 + 4 * l32 < a.D) {
        const float y[4] = {s1[0] * inv, s1[1] * inv, s1[2] * inv, s1[3] * inv};
        store4(dst + 128 + 4 * l32, y);
    }
    if (a.lse && l32 == 0)
        a.lse[(int64_t)(tile.q0 + token) * a.Hq + qh] = total == 0.f ? -INFINITY : m + logf(total);
}

// --------------------------------------------------------------------------------- plans

template <typename E, int DP, bool WIDE>
hipError_t run_kind4(const Attn4Args &a, const Attn4Plan &p, hipStream_t s)
{
    const unsigned grid = (unsigned)(p.main.items * a.Hkv);
    if (p.main.bm == kFewRows)
        k_attn4_few<E, DP, WIDE><<<grid, 256, 0, s>>>(a);
    else if (p.main.bm == kSmallRows)
        k_attn4_tile<E, DP, WIDE, 2><<<grid, 256, 0, s>>>(a);
    else
        k_attn4_tile<E, DP, WIDE, 1><<<grid, 256, 0, s>>>(a);
    return hipGetLastError();
}

template <typename E, bool WIDE>
hipError_t run_dim4(const Attn4Args &a, const Attn4Plan &p, hipStream_t s)
{
    if (a.D <= 64)
        return run_kind4<E, 64, WIDE>(a, p, s);
    if (a.D <= 128)
        return run_kind4<E, 128, WIDE>(a, p, s);
    return run_kind4<E, 256, WIDE>(a, p, s);
}

template <typename TO>
hipError_t run_join4(const Attn4Args &a, const Attn4Plan &p, hipStream_t s)
{
    const dim3 grid((unsigned)(p.main.tiles * a.Hkv), (unsigned)((p.main.bm + kJoinGroups - 1) / kJoinGroups));
    k_attn4_join<TO><<<grid, 32 * kJoinGroups, 0, s>>>(a, p.main.bm);
    return hipGetLastError();
}

}  // namespace

Attn4Plan attn4_plan(int64_t T, int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t most_keys)
{
    Attn4Plan plan{};
    AttnPart &p = plan.main;
    const int64_t rows = T * (Hq / Hkv), seqs = B < T ? B : T;  // no more than these have rows
    // Rows of a tile, by the mean rows of such a sequence (idle ones of the table count, too): up to 16, one small tile
    // each; up to 64, one of 64. Longer ones take tiles of 128, or of 64 where those would not fill the CUs and there are no
    // long caches to cut instead (capacity of twice the call's tokens or more; 7B prompts of 813 tokens behind 4096 keys:
    // 86 us cut, 137 uncut with 64 rows; packed 2B prompts of 2048 tokens 49 and 39). Lengths are on the device, so that the
    // capacity, what a row of the table can hold, is what there is to go by: new prompts in a wide table count as cached
    // (those packed ones in a table of 128 pages of 64: 52 us; one prompt of 2048 82 where a table cut to size takes 66).
    const bool few = rows <= kFewRows * seqs;
    const int64_t tiles128 = rows / kTileRows + seqs;
    const bool fills = tiles128 * Hkv >= 512, cached = most_keys > 2 * T;
    p.bm = few ? kFewRows : rows <= kSmallRows * seqs || !(fills || cached) ? kSmallRows : kTileRows;
    p.tiles = seqs == 1 ? (rows + p.bm - 1) / p.bm : rows / p.bm + seqs;  // at least sum of ceil(rows_b / bm)
    // Keys are cut into slices where the tiles alone leave CUs idle: into about four workgroups of few rows a CU, or a
    // little under the two of many that a CU holds, since the tiles' last slices come on top (256 tokens over 8192 keys, five
    // key heads: 72 us aiming at 512, 55 at 480, 62 at 384). Few rows: 64 tokens over slabs of up to 8192 keys, five key
    // heads, 104 us uncut, 55 cut; 300 tokens over 300 to 1200 keys, eight key heads, 66 and 76. Tiles of 64: 48 drafts of 8
    // over 2000 keys, five key heads, 60 and 47; 64 of them 65 and 78; 100 of them 75 and 73.
    const int64_t target = ((few ? 1024 : 480) + Hkv - 1) / Hkv;
    const bool cut = few ? p.tiles * Hkv < 768 : p.bm == kSmallRows ? cached && p.tiles * Hkv < 448 : !fills;
    p.target = cut && most_keys > 512 ? target : 0;
    p.min_units = few ? 2 : 4;
    const int64_t most = ((most_keys + kUnit - 1) / kUnit + p.min_units - 1) / p.min_units;
    p.items = p.tiles + (p.target ? p.target + 8 : 0);
    if (p.target && p.tiles * (most > 1 ? most : 1) < p.items)
        p.items = p.tiles * (most > 1 ? most : 1);
    const int64_t slots = p.target ? p.items * Hkv * p.bm : 0;
    p.l_off = round_up(slots * D * 4, 256);
    plan.notes_off = p.l_off + round_up(slots * 4, 256);
    plan.bytes = (size_t)(plan.notes_off + (p.target ? round_up((1 + p.tiles) * kNoteBytes, 256) : 0));
    return plan;
}

// The kernels of launch_attention4, in order (bt_attention4_plan).
void attention4_plan_text(const Attn4Plan &p, int D, int type, int out_type, char *buf, size_t len)
{
    auto name = [](int t) { return t == kF32 ? "fp32" : t == kBF16 ? "bf16" : "fp16"; };
    const int dp = D <= 64 ? 64 : D <= 128 ? 128 : 256;
    char tile[32] = "", join[64] = "";
    if (p.main.bm != kFewRows)
        snprintf(tile, sizeof(tile), ",%d", p.main.bm);
    if (p.main.target)
        snprintf(join, sizeof(join), " + k_attn4_join<%s>", name(out_type));
    snprintf(buf, len, "k_attn4_%s<%s,%d,%s%s>%s", p.main.bm == kFewRows ? "few" : "tile", name(type), dp, name(out_type),
             tile, join);
}

hipError_t launch_attention4(const Attn4Args &args, const Attn4Plan &p, int type, int out_type, hipStream_t s)
{
    Attn4Args a = args;
    char *ws = reinterpret_cast<char *>(args.ws_o);
    a.target = (int)p.main.target;
    a.items = (int)p.main.items;
    a.min_units = p.main.min_units;
    a.ws_o = reinterpret_cast<float *>(ws);
    a.ws_l = reinterpret_cast<float *>(ws + p.main.l_off);
    a.notes = ws + p.notes_off;
    a.tiles = (int)p.main.tiles;
    const bool wide = out_type == kF32;
    hipError_t e = type == kBF16 ? (wide ? run_dim4<bf16_t, true>(a, p, s) : run_dim4<bf16_t, false>(a, p, s))
                                 : (wide ? run_dim4<f16_t, true>(a, p, s) : run_dim4<f16_t, false>(a, p, s));
    if (e != hipSuccess || !p.main.target)
        return e;
    return wide            ? run_join4<float>(a, p, s)
           : type == kBF16 ? run_join4<bf16_t>(a, p, s)
                           : run_join4<f16_t>(a, p, s);
}

}  // namespace bt
