// Low-rank adapters of many requests beside one shared projection (bt_lora_apply):
//
//   Y[m, n] = Y0[m, n] + scale[a] * sum_{r < rank[a]} H[m, g(n), r] * B[a, n, r]
//   H[m, g, r] = sum_k X[m, k] * A[a, g R + r, k]          a = adapter[m], g(n) = row group of n
//
// Two launches: a shrink kernel forms H (times the scale) in the workspace, as one partial per
// slice of K; an expand kernel adds the partials in their order, multiplies by B and adds Y0. No
// atomics: the same call gives the same bits.
//
// The tokens of a tile (16) are worked off adapter by adapter, each adapter's weights being read
// once for all of the tile's tokens that use it (once per two of them in the few-tokens form). The
// other tokens of the tile take no part in it: an adapter's weights, whatever they hold, never reach
// a token that does not use it.
//  * Few tokens (k_lora_shrink_few, k_lora_expand_few; see lora_plan): a workgroup per (tile,
//    first token of an adapter), so that a decode batch's adapters are read side by side; bound by
//    the bytes of A and B. fp32 FMA where at most four of the tile's tokens share the adapter (the matrix
//    cores would mostly multiply columns that are not wanted, and cutting operands for them costs more
//    than the FMAs), else the many-tokens form's products for that adapter.
//  * Many tokens (k_lora_shrink, k_lora_expand): a workgroup walks its tile's adapters (one or two
//    where prompts are runs) on the matrix cores; bound by the bytes of X, Y0 and Y.
//
// Precision: X, H and Y are fp32 and so is the sum. On the matrix cores the products run in bf16
// without rounding any operand: an fp32 value is cut (by truncation) into three bf16 pieces of eight
// significant bits each that add up to it exactly, a bf16 weight is one piece, an fp16 weight
// two and an fp32 weight three, and the piece products are summed in fp32: 3, 6 or 8 MFMAs for
// one (of fp32 weights' nine, the last is left out: below 2^-30 of the whole). fp32 MFMA would
// take 5.3 times the bf16 form's cycles.
//
// Infinities. Cut into pieces an infinity becomes inf and inf - inf, and the zero rows and columns that
// fill up a matrix product (unused ranks, outputs of another row group) make NaNs of infinite H. Where a
// matrix product's sum comes out infinite or NaN, it is therefore formed again in fp32 FMAs over what belongs
// to it, which gives what the formula gives; unused ranks of H are stored as 0.
#include "bt_internal.h"
#include "convert.h"
#include "wave.h"

namespace bt {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kTile = 16;        // tokens of a tile
constexpr int kWaves = 4;            // of a workgroup of k_lora_shrink_few
constexpr int kDeepWaves = 8;        // of a workgroup of k_lora_shrink
constexpr int kStepK = 32 * kDeepWaves;  // k of one workgroup step of k_lora_shrink
constexpr int kMaxRank = 256;
constexpr int kFewTokens = 128;      // M up to which the few-tokens kernels are taken for any adapters,
constexpr int kFewMixed = 1024, kFewPer = 8;  // and up to which where there are at most so many per adapter
constexpr int kChunkK = 512;         // k of one wave step of k_lora_shrink_few: 8 per lane
constexpr int kFewShare = 4;         // tokens of a tile sharing an adapter above which it goes to the matrix cores
constexpr int kGroupTok = 2;         // tokens that share one reading of an adapter there

struct LoraArgs {
    const void *A, *B;
    const float *scale;
    const int *ranks, *adapter;
    const float *X, *Y0;
    float *Y, *ws;
    int64_t M, N, K;
    int L, R, Rp;  // Rp: R rounded up to 16
    int slices, kslice, tiles;
    int quads;  // N is a multiple of 4: outputs move four at a time
    RowGroups groups;
};

// Number of bf16 pieces that an element type is cut into without rounding.
template <typename W>
struct Terms {
    static constexpr int n = 1;
};
template <>
struct Terms<f16_t> {
    static constexpr int n = 2;
};
template <>
struct Terms<float> {
    static constexpr int n = 3;
};

// Memory is read through buffers whose range check gives 0 outside: a lane that wants nothing asks for
// kOutside, and no load sits in a branch of its own (loads in divergent branches wait for each other).
constexpr uint32_t kOutside = 0x7FFFFFF0u;

__device__ inline __amdgpu_buffer_rsrc_t buffer_of(const void *p, int64_t bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), (short)0, (int)min(bytes, (int64_t)0x7FFFFF00),
                                             0x00020000);
}

// Eight consecutive values as they are in memory.
template <typename W>
struct Raw8 {
    u32x4 q[sizeof(W) / 2];
};

// Elements 0 .. n - 1 (n <= 8, none if <= 0) from byte offset `at`; the others are 0. VEC: 16-byte
// reads; n is then 8 or <= 0.
template <typename W, bool VEC>
__device__ inline Raw8<W> fetch8(__amdgpu_buffer_rsrc_t from, uint32_t at, int n)
{
    Raw8<W> out;
    if constexpr (VEC) {
        const uint32_t off = n > 0 ? at : kOutside;
#pragma unroll
        for (int i = 0; i < (int)sizeof(W) / 2; ++i)
            out.q[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(from, off, 16 * i, 0));
    } else if constexpr (sizeof(W) == 4) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            out.q[j / 4][j % 4] = __builtin_amdgcn_raw_buffer_load_b32(from, j < n ? at + 4 * j : kOutside, 0, 0);
    } else {
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            const uint32_t lo = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(from, j < n ? at + 2 * j : kOutside, 0, 0);
            const uint32_t hi =
                (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(from, j + 1 < n ? at + 2 * j + 2 : kOutside, 0, 0);
            out.q[0][j / 2] = lo | hi << 16;
        }
    }
    return out;
}

// Elements from n on set to 0, whatever they hold.
template <typename W>
__device__ inline void keep(Raw8<W> &r, int n)
{
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if constexpr (sizeof(W) == 4)
            r.q[j / 4][j % 4] = j < n ? r.q[j / 4][j % 4] : 0u;
        else
            r.q[0][j / 2] = j < n ? r.q[0][j / 2] : r.q[0][j / 2] & (j & 1 ? 0x0000FFFFu : 0xFFFF0000u);
    }
}

template <typename W>
__device__ inline float raw_value(const Raw8<W> &r, int j)  // j: a constant once unrolled
{
    if constexpr (Terms<W>::n == 3) {
        return __uint_as_float(r.q[j / 4][j % 4]);
    } else {
        const uint32_t u = r.q[0][j / 2];
        if constexpr (Terms<W>::n == 1)
            return __uint_as_float(j & 1 ? u & 0xFFFF0000u : u << 16);
        else
            return (float)__builtin_bit_cast(f16_t, (uint16_t)(u >> (16 * (j & 1))));
    }
}

// Eight values as up to three bf16 operands whose sum is exact.
template <int TERMS>
struct Pieces {
    u32x4 p[TERMS];
};

template <int TERMS>
__device__ inline Pieces<TERMS> cut(const float (&x)[8])
{
    Pieces<TERMS> out;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float a = x[2 * j], b = x[2 * j + 1];
#pragma unroll
        for (int t = 0; t < TERMS; ++t) {
            const uint32_t ua = __float_as_uint(a), ub = __float_as_uint(b);
            out.p[t][j] = __builtin_amdgcn_perm(ub, ua, 0x07060302u);  // the two high halves
            a -= __uint_as_float(ua & 0xFFFF0000u);
            b -= __uint_as_float(ub & 0xFFFF0000u);
        }
    }
    return out;
}

template <typename W>
__device__ inline Pieces<Terms<W>::n> pieces(const Raw8<W> &r)
{
    if constexpr (Terms<W>::n == 1) {
        return Pieces<1>{{r.q[0]}};
    } else {
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            x[j] = raw_value(r, j);
        return cut<Terms<W>::n>(x);
    }
}

// acc + w^T x over the 32 k (or r) of the operands, the small piece products first. Piece i is
// below 2^(1 - 8 i) of the value.
template <int TW>
__device__ inline f32x4 mma(const Pieces<TW> &w, const Pieces<3> &x, f32x4 acc)
{
#pragma unroll
    for (int d = TW == 1 ? 2 : 3; d >= 0; --d)
#pragma unroll
        for (int i = 0; i < TW; ++i)
            if (d - i >= 0 && d - i < 3)
                acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w.p[i]),
                                                              __builtin_bit_cast(bf16x8, x.p[d - i]), acc, 0, 0, 0);
    return acc;
}

// The adapter of this lane's token (lane % 16 of the tile), -1 for none or no such token.
__device__ inline int lane_adapter(const LoraArgs &a, int64_t m0, int t)
{
    if (m0 + t >= a.M)
        return -2;
    const int ad = a.adapter[m0 + t];
    return ad >= 0 && ad < a.L ? ad : -1;
}

__device__ inline int adapter_rank(const LoraArgs &a, int ad)
{
    return a.ranks ? max(0, min(a.ranks[ad], a.R)) : a.R;
}

// sum_k x[k] w[k] over k0 .. k1 - 1 in FMAs: for sums that are infinite or NaN on the matrix cores.
template <typename W>
__device__ inline float plain_dot(const float *x, const W *w, int k0, int k1)
{
    float s = 0.f;
#pragma unroll 1
    for (int k = k0; k < k1; ++k)
        s = __builtin_fmaf(x[k], (float)w[k], s);
    return s;
}

// Four sums (rows r .. r + 3 of group grp of adapter ad's A with token m over k0 .. k1 - 1) as they are
// stored in H, but for the scale: unused ranks 0, and infinite or NaN ones formed again.
template <typename W>
__device__ inline f32x4 checked_sums(const LoraArgs &a, f32x4 s, int ad, int grp, int r, int rank, int64_t m, int k0,
                                     int k1)
{
    // (four that overflow together cost a look that changes little)
    if (__builtin_expect(not_finite((s[0] + s[1]) + (s[2] + s[3])), 0)) {
        const float *x = a.X + m * a.K;
        const W *w = static_cast<const W *>(a.A) + (((int64_t)ad * a.groups.n + grp) * a.R + r) * a.K;
#pragma unroll 1
        for (int j = 0; j < 4; ++j, w += a.K) {
            float v = s[0];  // the four in turn
            if (r + j >= rank)
                v = 0.f;
            else if (not_finite(v))
                v = plain_dot(x, w, k0, k1);
            s = f32x4{s[1], s[2], s[3], v};
        }
    }
    return s;
}

// k_lora_shrink: 16 tokens against RT rank tiles of 16; eight waves take every eighth step of 32 k.
template <typename W, int RT, bool VEC>
__global__ __launch_bounds__(64 * kDeepWaves) void k_lora_shrink(LoraArgs a)
{
    __shared__ f32x4 part[kDeepWaves][RT][64];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int t = lane & 15, g = lane >> 4;
    const int64_t m0 = (int64_t)blockIdx.x * kTile;
    const int mine = lane_adapter(a, m0, t);
    uint32_t todo = (uint32_t)__ballot(mine >= 0) & 0xFFFFu;
    const int tpg = a.Rp / 16, tiles = tpg * a.groups.n;
    const int k0 = (int)blockIdx.y * a.kslice, k1 = (int)min((int64_t)k0 + a.kslice, a.K);
    const int row_x = (int)a.K * 4, row_w = (int)(a.K * sizeof(W));
    const __amdgpu_buffer_rsrc_t xs = buffer_of(a.X + m0 * a.K, min((int64_t)kTile, a.M - m0) * row_x);

    while (todo) {
        const int lead = __builtin_ctz(todo);
        const int ad = __builtin_amdgcn_readlane(mine, lead);
        const uint32_t same = (uint32_t)__ballot(mine == ad) & 0xFFFFu;
        todo &= ~same;
        const int rank = adapter_rank(a, ad);
        // an adapter's A (all groups, at most 8 * 256 rows) is below 2^31 bytes
        const __amdgpu_buffer_rsrc_t ws =
            buffer_of(static_cast<const W *>(a.A) + (int64_t)ad * a.groups.n * a.R * a.K, (int64_t)a.groups.n * a.R * row_w);
        uint32_t at[RT];
        bool in[RT];
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            const int tile = blockIdx.z * RT + i, r = (tile % tpg) * 16 + t;
            in[i] = tile < tiles && r < rank;
            at[i] = (uint32_t)((tile / tpg) * a.R + r) * (uint32_t)row_w;
        }
        f32x4 acc[RT];
#pragma unroll
        for (int i = 0; i < RT; ++i)
            acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 2
        for (int kk = k0 + 32 * wave; kk < k1; kk += kStepK) {
            const int k = kk + 8 * g, n = min(8, k1 - k);
            const Raw8<float> xr = fetch8<float, VEC>(xs, (uint32_t)t * row_x + 4u * k, n);
            Raw8<W> wr[RT];
#pragma unroll
            for (int i = 0; i < RT; ++i)
                wr[i] = fetch8<W, VEC>(ws, at[i] + (uint32_t)sizeof(W) * k, in[i] ? n : 0);
            const Pieces<3> x = pieces(xr);
#pragma unroll
            for (int i = 0; i < RT; ++i)
                acc[i] = mma(pieces(wr[i]), x, acc[i]);
        }
#pragma unroll
        for (int i = 0; i < RT; ++i)
            part[wave][i][lane] = acc[i];
        __syncthreads();
        for (int e = threadIdx.x; e < RT * 64; e += 64 * kDeepWaves) {
            const int i = e >> 6, l = e & 63;
            const int tile = blockIdx.z * RT + i;
            if (tile < tiles && (same >> (l & 15) & 1)) {
                f32x4 s = part[0][i][l];
#pragma unroll
                for (int w = 1; w < kDeepWaves; ++w)
                    s += part[w][i][l];
                const int64_t m = m0 + (l & 15);
                s = checked_sums<W>(a, s, ad, tile / tpg, (tile % tpg) * 16 + (l >> 4) * 4, rank, m, k0, k1);
                s *= a.scale[ad];
                float *dst = a.ws + (((int64_t)blockIdx.y * a.M + m) * a.groups.n + tile / tpg) * a.Rp +
                             (tile % tpg) * 16 + (l >> 4) * 4;
                *reinterpret_cast<f32x4 *>(dst) = s;
            }
        }
        if (todo)
            __syncthreads();
    }
}

// k_lora_expand: each wave on its own takes 16 tokens and 64 outputs. H and the weights go from
// memory straight into the MFMA operands (no barrier), and Y0 is requested before either, so that a wave
// waits twice: for its tokens' adapters, and for what depends on them. Y0 and Y move as 256-byte pieces of
// four rows, past the caches, the sums through LDS into that order: 2048 tokens of 2B gate+up, both kernels,
// 61 us (4.2 TB/s; a large copy reaches 4.9), against 67.9 us through the caches, 71.6 us with the MFMA's own
// order (64-byte pieces of sixteen rows), 82 us with H read again from every slice of K. Between the product
// that wrote Y0 and a launch that reads Y, past / through the caches: 2048 tokens of 2B QKV with the product
// and the head norms 70.5 / 66.8 us, 4096 of 7B QKV 330 / 337, 2048 of 2B gate+up with the product 125.5 / 127.
constexpr int kStream = 2;  // buffer loads and stores: non-temporal
constexpr int kExpandN = 64, kExpandT = kExpandN / 16;

struct Slab {
    float row[kTile][kExpandN + 4];
};

// Adapter ad's part of output n of token m in FMAs: for those that are infinite or NaN on the matrix cores.
template <typename W>
__device__ inline float plain_output(const LoraArgs &a, int64_t m, int ad, int64_t n)
{
    int grp = 0;
    while (n >= a.groups.end[grp])
        ++grp;
    const W *b = static_cast<const W *>(a.B) + ((int64_t)ad * a.N + n) * a.R;
    const float *h = a.ws + (m * a.groups.n + grp) * a.Rp;
    const int64_t step = a.M * a.groups.n * a.Rp;
    const int rank = adapter_rank(a, ad);
    float sum = 0.f;
#pragma unroll 1
    for (int r = 0; r < rank; ++r) {
        float x = 0.f;
#pragma unroll 1
        for (int s = 0; s < a.slices; ++s)
            x += h[r + s * step];
        sum = __builtin_fmaf(x, (float)b[r], sum);
    }
    return sum;
}

// The wave's 64 outputs from n0 on of the tokens in `stored`; `mine`: the adapter of token lane % 16.
template <typename W, bool VEC>
__device__ __forceinline__ void expand_tile(const LoraArgs &a, int64_t m0, int64_t n0, int mine, uint32_t stored,
                                            Slab &slab)
{
    static_assert(kExpandN == 64 && kExpandT == 4, "sixteen lanes move a row of four values each");
    const int lane = threadIdx.x & 63, t = lane & 15, g = lane >> 4;
    const int cols = (int)min((int64_t)kExpandN, a.N - n0);
    // this lane's outputs: tokens 4 i + g, columns 4 t .. + 3 of the wave's
    const int64_t corner = m0 * a.N + n0;
    const int64_t span = ((min((int64_t)kTile, a.M - m0) - 1) * a.N + cols) * 4;
    uint32_t yoff[kExpandT];
#pragma unroll
    for (int i = 0; i < kExpandT; ++i)
        yoff[i] = (stored >> (4 * i + g) & 1) && 4 * t < cols ? (uint32_t)((4 * i + g) * a.N + 4 * t) * 4u : kOutside;
    const __amdgpu_buffer_rsrc_t ys = buffer_of(a.Y0 ? a.Y0 + corner : nullptr, a.Y0 ? span : 0);
    f32x4 y[kExpandT], acc[kExpandT];
    if (a.quads) {
#pragma unroll
        for (int i = 0; i < kExpandT; ++i)
            y[i] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(ys, yoff[i], 0, kStream));
    } else {
#pragma unroll
        for (int i = 0; i < kExpandT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                y[i][j] = __builtin_bit_cast(
                    float, __builtin_amdgcn_raw_buffer_load_b32(ys, 4 * t + j < cols ? yoff[i] + 4 * j : kOutside, 0, 0));
    }
#pragma unroll
    for (int i = 0; i < kExpandT; ++i)
        acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};  // token t, columns 16 i + 4 g .. + 3
    uint32_t todo = (uint32_t)__ballot(mine >= 0) & stored;
    const int64_t hrow = min(m0 + t, a.M - 1) * a.groups.n, hstep = a.M * a.groups.n * a.Rp;
    while (todo) {
        const int lead = __builtin_ctz(todo);
        const int ad = __builtin_amdgcn_readlane(mine, lead);
        const uint32_t same = (uint32_t)__ballot(mine == ad) & 0xFFFFu;
        todo &= ~same;
        const int rank = adapter_rank(a, ad);
        const __amdgpu_buffer_rsrc_t bs = buffer_of(static_cast<const W *>(a.B) + ((int64_t)ad * a.N + n0) * a.R,
                                                    (int64_t)cols * a.R * sizeof(W));
        for (int grp = 0; grp < a.groups.n; ++grp) {
            const int64_t lo = grp ? a.groups.end[grp - 1] : 0, hi = a.groups.end[grp];
            if (hi <= n0 || lo >= n0 + cols)
                continue;
            f32x4 sum[kExpandT];
#pragma unroll
            for (int i = 0; i < kExpandT; ++i)
                sum[i] = f32x4{0.f, 0.f, 0.f, 0.f};
            for (int rr = 0; rr < a.Rp; rr += 32) {
                const int r = rr + 8 * g;
                Raw8<W> wr[kExpandT];
#pragma unroll
                for (int i = 0; i < kExpandT; ++i) {
                    const int c = 16 * i + t;
                    const bool in = n0 + c >= lo && n0 + c < hi;
                    wr[i] = fetch8<W, VEC>(bs, (uint32_t)(c * a.R + r) * (uint32_t)sizeof(W), in ? min(8, rank - r) : 0);
                }
                // this token's H (other tokens' columns are computed from theirs and not taken)
                const float *src = a.ws + (hrow + grp) * a.Rp + min(r, a.Rp - 8);
                f32x4 h0 = {0.f, 0.f, 0.f, 0.f}, h1 = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
                for (int s = 0; s < a.slices; ++s) {
                    h0 += *reinterpret_cast<const f32x4 *>(src + s * hstep);
                    h1 += *reinterpret_cast<const f32x4 *>(src + s * hstep + 4);
                }
                float h[8];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    h[j] = r < a.Rp ? h0[j] : 0.f;
                    h[4 + j] = r < a.Rp ? h1[j] : 0.f;
                }
                const Pieces<3> x = cut<3>(h);
                if (VEC && (rank & 7) && rr + 32 > rank)
#pragma unroll
                    for (int i = 0; i < kExpandT; ++i)
                        keep(wr[i], rank - r);
#pragma unroll
                for (int i = 0; i < kExpandT; ++i)
                    sum[i] = mma(pieces(wr[i]), x, sum[i]);
            }
            if (same >> t & 1)
#pragma unroll
                for (int i = 0; i < kExpandT; ++i)
                    acc[i] += sum[i];
        }
    }
    // from the MFMA's order to rows, through the wave's own piece of LDS (a wave's LDS operations
    // complete in order)
#pragma unroll
    for (int i = 0; i < kExpandT; ++i)
        *reinterpret_cast<f32x4 *>(&slab.row[t][16 * i + 4 * g]) = acc[i];
    asm volatile("" ::: "memory");
    const f32x4 all = (acc[0] + acc[1]) + (acc[2] + acc[3]);
    if (__builtin_expect(not_finite((all[0] + all[1]) + (all[2] + all[3])), 0))
#pragma unroll 1
        for (int e = 0; e < 4 * kExpandT; ++e) {
            const int c = 16 * (e / 4) + 4 * g + e % 4;
            if (not_finite(slab.row[t][c]))
                slab.row[t][c] = c < cols ? plain_output<W>(a, m0 + t, mine, n0 + c) : 0.f;
        }
    asm volatile("" ::: "memory");
#pragma unroll
    for (int i = 0; i < kExpandT; ++i)
        y[i] += *reinterpret_cast<const f32x4 *>(&slab.row[4 * i + g][4 * t]);
    const __amdgpu_buffer_rsrc_t out = buffer_of(a.Y + corner, span);
    if (a.quads) {
#pragma unroll
        for (int i = 0; i < kExpandT; ++i)
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, y[i]), out, yoff[i], 0, kStream);
    } else {
#pragma unroll
        for (int i = 0; i < kExpandT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(y[i][j]), out,
                                                      4 * t + j < cols ? yoff[i] + 4 * j : kOutside, 0, 0);
    }
}

template <typename W, bool VEC>
__global__ __launch_bounds__(256, 3) void k_lora_expand(LoraArgs a)
{
    __shared__ __attribute__((aligned(16))) Slab slab[4];
    const int wave = uniform(threadIdx.x >> 6);
    // outputs vary fastest, over a workgroup's waves and over workgroups
    const int64_t blocks = (a.N + 4 * kExpandN - 1) / (4 * kExpandN);
    const int64_t m0 = (int64_t)(blockIdx.x / blocks) * kTile;
    const int64_t n0 = ((int64_t)(blockIdx.x % blocks) * 4 + wave) * kExpandN;
    if (n0 >= a.N)
        return;
    const int mine = lane_adapter(a, m0, threadIdx.x & 15);
    expand_tile<W, VEC>(a, m0, n0, mine, (uint32_t)__ballot(mine > -2) & 0xFFFFu, slab[wave]);
}

// The leader token of this workgroup of a few-tokens kernel and the tokens that share its adapter;
// false: the token is not the first one of its adapter, or does not exist. (Workgroups go to the eight
// dies in turn. Tiles vary fastest over them: with leaders fastest, where a tile has one adapter, all
// the workgroups that have work would be on one die.)
__device__ inline bool lead_tokens(const LoraArgs &a, int64_t m0, int lead, int &mine, int &ad, uint32_t &same)
{
    mine = lane_adapter(a, m0, threadIdx.x & 15);
    ad = __builtin_amdgcn_readlane(mine, lead);
    same = (uint32_t)__ballot(mine == ad) & 0xFFFFu;
    return ad > -2 && __builtin_ctz(same) == lead;
}

// The lowest kGroupTok set bits of `todo` as token numbers (the last one repeated), taken out of it.
__device__ inline int take_tokens(uint32_t &todo, int (&tok)[kGroupTok])
{
    int n = 0;
#pragma unroll
    for (int i = 0; i < kGroupTok; ++i) {
        if (todo) {
            tok[i] = __builtin_ctz(todo);
            todo &= todo - 1;
            n = i + 1;
        } else {
            tok[i] = tok[i ? i - 1 : 0];
        }
    }
    return n;
}

// k_lora_shrink_few: 16 rows of one adapter's A against up to two of its tokens at a time. A lane
// keeps eight k of the tokens in registers; every row is then one contiguous 1 KiB read of the wave,
// all sixteen in flight together. The sixteen rows' partial sums are added over the lanes by swaps
// that halve the number of values each time.
template <typename W, bool VEC>
__global__ __launch_bounds__(256, 3) void k_lora_shrink_few(LoraArgs a)
{
    __shared__ float part[kWaves][kGroupTok][16];
    __shared__ f32x4 tile[kWaves][64];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int64_t m0 = (int64_t)(blockIdx.x % a.tiles) * kTile;
    int mine, ad;
    uint32_t same;
    if (!lead_tokens(a, m0, blockIdx.x / a.tiles, mine, ad, same) || ad < 0)
        return;
    const int tpg = a.Rp / 16, grp = blockIdx.z / tpg, r0 = (blockIdx.z % tpg) * 16;
    const int rank = adapter_rank(a, ad);
    const int rows = min(16, rank - r0);  // may be <= 0: H is 0 there
    const int row_w = (int)(a.K * sizeof(W));
    const __amdgpu_buffer_rsrc_t ws =
        buffer_of(static_cast<const W *>(a.A) + (((int64_t)ad * a.groups.n + grp) * a.R + r0) * a.K,
                  (int64_t)max(rows, 0) * row_w);
    const __amdgpu_buffer_rsrc_t xs = buffer_of(a.X + m0 * a.K, min((int64_t)kTile, a.M - m0) * a.K * 4);
    const float scale = a.scale[ad];
    const int k0 = (int)blockIdx.y * a.kslice, k1 = (int)min((int64_t)k0 + a.kslice, a.K);
    if (__builtin_popcount(same) > kFewShare) {
        // the whole tile on the matrix cores; the four waves take every fourth step of 32 k
        const int t = lane & 15, g = lane >> 4;
        f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
        for (int kk = k0 + 32 * wave; kk < k1; kk += 32 * kWaves) {
            const int k = kk + 8 * g, n = min(8, k1 - k);
            const Raw8<float> xr = fetch8<float, VEC>(xs, (uint32_t)(t * (int)a.K + k) * 4u, n);
            const Raw8<W> wr = fetch8<W, VEC>(ws, (uint32_t)t * (uint32_t)row_w + (uint32_t)sizeof(W) * k, n);
            acc = mma(pieces(wr), pieces(xr), acc);
        }
        tile[wave][lane] = acc;
        __syncthreads();
        if (wave == 0 && (same >> t & 1)) {
            f32x4 s = tile[0][lane];
#pragma unroll
            for (int q = 1; q < kWaves; ++q)
                s += tile[q][lane];
            s = checked_sums<W>(a, s, ad, grp, r0 + 4 * g, rank, m0 + t, k0, k1);
            *reinterpret_cast<f32x4 *>(a.ws + (((int64_t)blockIdx.y * a.M + m0 + t) * a.groups.n + grp) * a.Rp + r0 +
                                       4 * g) = s * scale;
        }
        return;
    }
    while (same) {
        int tok[kGroupTok];
        const int nt = take_tokens(same, tok);
        float acc[kGroupTok][16];
#pragma unroll
        for (int i = 0; i < kGroupTok; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r)
                acc[i][r] = 0.f;
        for (int kk = k0 + kChunkK * wave; kk < k1; kk += kChunkK * kWaves) {
            const int k = kk + 8 * lane, n = min(8, k1 - k);
            Raw8<W> raw[16];
#pragma unroll
            for (int r = 0; r < 16; ++r)  // rows from `rows` on are outside the buffer
                raw[r] = fetch8<W, VEC>(ws, (uint32_t)r * (uint32_t)row_w + (uint32_t)sizeof(W) * k, n);
            float x[kGroupTok][8];  // a token that is not there: the last one again
#pragma unroll
            for (int i = 0; i < kGroupTok; ++i) {
                const Raw8<float> xr = fetch8<float, VEC>(xs, (uint32_t)(tok[i] * (int)a.K + k) * 4u, n);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    x[i][j] = raw_value(xr, j);
            }
#pragma unroll
            for (int r = 0; r < 16; ++r)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float v = raw_value(raw[r], j);
#pragma unroll
                    for (int i = 0; i < kGroupTok; ++i)
                        acc[i][r] = __builtin_fmaf(v, x[i][j], acc[i][r]);
                }
        }
#pragma unroll
        for (int i = 0; i < kGroupTok; ++i) {
            if (i >= nt)
                break;
            // rows r and r + 8: lanes 0 .. 31 keep row r, lanes 32 .. 63 row r + 8; and so on, until
            // each 16 lanes hold four rows, which are then added within them
            float v[8], u[4];
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(acc[i][r]),
                                                                __float_as_uint(acc[i][r + 8]), false, false);
                v[r] = __uint_as_float(p[0]) + __uint_as_float(p[1]);
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v[r]), __float_as_uint(v[r + 4]), false,
                                                                false);
                u[r] = __uint_as_float(p[0]) + __uint_as_float(p[1]);
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                u[r] += __int_as_float(dpp_i<kDppQuadXor1>(__float_as_int(u[r])));
                u[r] += __int_as_float(dpp_i<kDppQuadXor2>(__float_as_int(u[r])));
                u[r] += __int_as_float(dpp_i<kDppRowHalfMirror>(__float_as_int(u[r])));
                u[r] += __int_as_float(dpp_i<kDppRowMirror>(__float_as_int(u[r])));
            }
            // lanes 16 q .. 16 q + 15 hold rows 8 (q / 2) + 4 (q % 2) + 0 .. 3
            if ((lane & 15) == 0)
                *reinterpret_cast<f32x4 *>(&part[wave][i][4 * (lane >> 4)]) = f32x4{u[0], u[1], u[2], u[3]};
        }
        __syncthreads();
        if (threadIdx.x < nt * 16) {
            const int i = threadIdx.x / 16, r = threadIdx.x % 16;
            float s = part[0][i][r];
#pragma unroll
            for (int q = 1; q < kWaves; ++q)
                s += part[q][i][r];
            int m = tok[0];
#pragma unroll
            for (int q = 1; q < kGroupTok; ++q)
                m = i == q ? tok[q] : m;
            a.ws[(((int64_t)blockIdx.y * a.M + m0 + m) * a.groups.n + grp) * a.Rp + r0 + r] = r < rows ? s * scale : 0.f;
        }
        if (same)
            __syncthreads();
    }
}

// k_lora_expand_few: 256 outputs of one adapter's tokens. A lane has one output, i.e. one row of B,
// whose first 64 values are requested before H is waited for; H is the same for all lanes (LDS
// broadcasts). Tokens without an adapter are one more group, which only copies Y0.
constexpr int kFewN = 256, kFewR = 64;

template <typename W, bool VEC>
__global__ __launch_bounds__(256) void k_lora_expand_few(LoraArgs a)
{
    __shared__ __attribute__((aligned(16))) float hs[kGroupTok][kMaxRank];
    __shared__ __attribute__((aligned(16))) Slab slab[4];
    const int64_t m0 = (int64_t)(blockIdx.x % a.tiles) * kTile;
    const int64_t nb = (int64_t)blockIdx.y * kFewN, n = nb + threadIdx.x;
    int mine, ad;
    uint32_t same;
    if (!lead_tokens(a, m0, blockIdx.x / a.tiles, mine, ad, same))
        return;
    if (ad >= 0 && __builtin_popcount(same) > kFewShare) {
        const int wave = uniform(threadIdx.x >> 6);
        if (nb + kExpandN * wave < a.N)
            expand_tile<W, VEC>(a, m0, nb + kExpandN * wave, mine, same, slab[wave]);
        return;
    }
    if (ad < 0) {
        if (a.Y0 != a.Y)
            for (; same; same &= same - 1)
                if (n < a.N) {
                    const int64_t at = (m0 + __builtin_ctz(same)) * a.N + n;
                    a.Y[at] = a.Y0 ? a.Y0[at] : 0.f;
                }
        return;
    }
    const int rank = adapter_rank(a, ad);
    // rows past N are outside the buffer
    const __amdgpu_buffer_rsrc_t bs = buffer_of(static_cast<const W *>(a.B) + ((int64_t)ad * a.N + nb) * a.R,
                                                min((int64_t)kFewN, a.N - nb) * a.R * sizeof(W));
    const uint32_t brow = threadIdx.x * (uint32_t)(a.R * sizeof(W));
    auto row8 = [&](int r) __attribute__((always_inline)) {
        Raw8<W> x = fetch8<W, VEC>(bs, brow + (uint32_t)sizeof(W) * r, min(8, rank - r));
        if (VEC && rank - r < 8)
            keep(x, rank - r);
        return x;
    };
    Raw8<W> raw[kFewR / 8];
#pragma unroll
    for (int c = 0; c < kFewR / 8; ++c)
        raw[c] = row8(8 * c);
    while (same) {
        int tok[kGroupTok];
        const int nt = take_tokens(same, tok);
        float y[kGroupTok], acc[kGroupTok];
#pragma unroll
        for (int i = 0; i < kGroupTok; ++i) {
            acc[i] = 0.f;
            y[i] = i < nt && a.Y0 && n < a.N ? a.Y0[(m0 + tok[i]) * a.N + n] : 0.f;
        }
        for (int grp = 0; grp < a.groups.n; ++grp) {
            const int64_t lo = grp ? a.groups.end[grp - 1] : 0, hi = a.groups.end[grp];
            if (hi <= nb || lo >= nb + kFewN)
                continue;
            __syncthreads();  // the last reads of hs are done
            for (int e = threadIdx.x; e < nt * (a.Rp / 4); e += 256) {
                const int i = e / (a.Rp / 4), r = e % (a.Rp / 4) * 4;
                int m = tok[0];
#pragma unroll
                for (int q = 1; q < kGroupTok; ++q)
                    m = i == q ? tok[q] : m;
                const float *src = a.ws + ((m0 + m) * a.groups.n + grp) * a.Rp + r;
                const int64_t step = a.M * a.groups.n * a.Rp;
                f32x4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
                for (int q = 0; q < a.slices; ++q)
                    s += *reinterpret_cast<const f32x4 *>(src + q * step);
                *reinterpret_cast<f32x4 *>(&hs[i][r]) = s;
            }
            __syncthreads();
            if (n < lo || n >= hi)
                continue;
            for (int r0 = 0; r0 < rank; r0 += kFewR) {
                Raw8<W> v[kFewR / 8];
#pragma unroll
                for (int c = 0; c < kFewR / 8; ++c)
                    v[c] = r0 ? row8(r0 + 8 * c) : raw[c];
#pragma unroll
                for (int c = 0; c < kFewR / 8; ++c) {
                    if (r0 + 8 * c >= rank)
                        break;
#pragma unroll
                    for (int i = 0; i < kGroupTok; ++i) {
                        if (i >= nt)
                            break;
                        const f32x4 h0 = *reinterpret_cast<const f32x4 *>(&hs[i][r0 + 8 * c]);
                        const f32x4 h1 = *reinterpret_cast<const f32x4 *>(&hs[i][r0 + 8 * c + 4]);
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            acc[i] = __builtin_fmaf(raw_value(v[c], j), h0[j], acc[i]);
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            acc[i] = __builtin_fmaf(raw_value(v[c], 4 + j), h1[j], acc[i]);
                    }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kGroupTok; ++i)
            if (i < nt && n < a.N)
                a.Y[(m0 + tok[i]) * a.N + n] = y[i] + acc[i];
    }
}

struct LoraPlan {
    bool few;
    int rt, slices, leads;
    int64_t kslice, tiles, ztiles;
};

// The few-tokens form costs a workgroup per token, most of them idle where tokens come in runs; the other
// form walks a tile's adapters one after the other. 256 tokens in random order over 64 adapters of 7B O,
// few / many: 32 / 72 us; 512: 54 / 78; 1024 (sixteen tokens for each adapter): 91 / 108 in random order and
// 33 / 18 in runs; in runs over 4 adapters of 2B QKV, 256 tokens: 20 / 12 us; of 7B QKV (rank 64), 512: 66 / 40
// us. Which one it will be is device data; adapters that tokens hardly share (kFewPer) are taken for the first.
LoraPlan lora_plan(int64_t M, int64_t K, int64_t R, int64_t groups, bool few)
{
    LoraPlan p;
    const int64_t rank_tiles = round_up(R, 16) / 16 * groups;
    p.few = few;
    p.rt = p.few ? 1 : rank_tiles >= 3 ? 4 : (int)rank_tiles;
    p.ztiles = (rank_tiles + p.rt - 1) / p.rt;
    p.tiles = (M + kTile - 1) / kTile;
    p.leads = (int)(M < kTile ? M : kTile);
    // K in as many slices as give four workgroups per CU (eight waves each, one is enough), each at least
    // one step, and few: the expand kernels read every slice's partial sums, and with many tokens they do
    // so for every 64 outputs.
    const int64_t wgs = (p.few ? p.tiles * p.leads : p.tiles) * p.ztiles;
    const int64_t unit = p.few ? kChunkK : kStepK;             // smallest slice
    const int64_t whole = p.few ? kChunkK * kWaves : kStepK;   // k of a workgroup step
    const int64_t steps = K > 0 ? (K + whole - 1) / whole : 1;
    const int64_t want = p.few ? 1024 : 256, most = p.few ? 8 : 4;
    int64_t slices = (want + wgs - 1) / wgs;
    slices = slices < steps ? slices : steps;
    slices = slices < most ? slices : most;
    const int64_t k = K > 0 ? K : 1;
    p.kslice = round_up((k + slices - 1) / slices, unit);
    p.slices = (int)((k + p.kslice - 1) / p.kslice);
    return p;
}

template <typename W, bool VEC>
hipError_t launch_shrink(const LoraArgs &a, const LoraPlan &p, hipStream_t s)
{
    const dim3 grid((unsigned)(p.tiles * (p.few ? p.leads : 1)), (unsigned)p.slices, (unsigned)p.ztiles);
    if (p.few)
        k_lora_shrink_few<W, VEC><<<grid, 64 * kWaves, 0, s>>>(a);
    else if (p.rt == 1)
        k_lora_shrink<W, 1, VEC><<<grid, 64 * kDeepWaves, 0, s>>>(a);
    else if (p.rt == 2)
        k_lora_shrink<W, 2, VEC><<<grid, 64 * kDeepWaves, 0, s>>>(a);
    else
        k_lora_shrink<W, 4, VEC><<<grid, 64 * kDeepWaves, 0, s>>>(a);
    return hipGetLastError();
}

template <typename W, bool VEC>
hipError_t launch_expand(const LoraArgs &a, const LoraPlan &p, hipStream_t s)
{
    if (p.few) {
        const dim3 grid((unsigned)(p.tiles * p.leads), (unsigned)((a.N + kFewN - 1) / kFewN));
        k_lora_expand_few<W, VEC><<<grid, 256, 0, s>>>(a);
    } else {
        const int64_t blocks = p.tiles * ((a.N + 4 * kExpandN - 1) / (4 * kExpandN));
        k_lora_expand<W, VEC><<<(unsigned)blocks, 256, 0, s>>>(a);
    }
    return hipGetLastError();
}

// 16-byte reads where rows are whole eights of values and start on 4 bytes (a buffer load's alignment).
template <typename W>
hipError_t launch_weights(const LoraArgs &a, const LoraPlan &p, hipStream_t s)
{
    const bool vec_a = a.K % 8 == 0 && (reinterpret_cast<uintptr_t>(a.A) & 3) == 0;
    const bool vec_b = a.R % 8 == 0 && (reinterpret_cast<uintptr_t>(a.B) & 3) == 0;
    if (hipError_t e = vec_a ? launch_shrink<W, true>(a, p, s) : launch_shrink<W, false>(a, p, s))
        return e;
    return vec_b ? launch_expand<W, true>(a, p, s) : launch_expand<W, false>(a, p, s);
}

}  // namespace

size_t lora_workspace_bytes(int64_t M, int64_t K, int64_t R, int64_t groups)
{
    // for either form: which one is taken depends on the number of adapters
    const int few = lora_plan(M, K, R, groups, true).slices, many = lora_plan(M, K, R, groups, false).slices;
    const int slices = M <= kFewTokens ? few : M > kFewMixed ? many : few > many ? few : many;
    return (size_t)slices * M * groups * round_up(R, 16) * 4;
}

hipError_t launch_lora(const void *A, const void *B, int w_type, const float *scale, const int32_t *ranks, int64_t L,
                       int64_t R, const RowGroups &groups, const int32_t *adapter, const float *X, const float *Y0,
                       int64_t M, int64_t N, int64_t K, float *Y, void *workspace, hipStream_t s)
{
    const bool few = M <= kFewTokens || (M <= kFewMixed && M <= kFewPer * L);
    const LoraPlan p = lora_plan(M, K, R, groups.n, few);
    LoraArgs a;
    a.A = A;
    a.B = B;
    a.scale = scale;
    a.ranks = ranks;
    a.adapter = adapter;
    a.X = X;
    a.Y0 = Y0;
    a.Y = Y;
    a.ws = static_cast<float *>(workspace);
    a.M = M;
    a.N = N;
    a.K = K;
    a.L = (int)L;
    a.R = (int)R;
    a.Rp = (int)round_up(R, 16);
    a.tiles = (int)p.tiles;
    a.slices = p.slices;
    a.kslice = (int)p.kslice;
    a.quads = N % 4 == 0;
    a.groups = groups;
    switch (w_type) {
    case kBF16: return launch_weights<bf16_t>(a, p, s);
    case kF16: return launch_weights<f16_t>(a, p, s);
    default: return launch_weights<float>(a, p, s);
    }
}

}  // namespace bt
