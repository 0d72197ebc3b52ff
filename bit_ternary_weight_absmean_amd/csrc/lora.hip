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
// once for all of the tile's tokens that use it (once per four of them in the few-tokens form). The
// other tokens of the tile take no part in it: an adapter's weights, whatever they hold, never reach
// a token that does not use it.
//  * Few tokens (k_lora_shrink_few, k_lora_expand_few; up to kFewTokens): a workgroup per (tile,
//    first token of an adapter), so that a decode batch's adapters are read side by side; bound by
//    the bytes of A and B. fp32 FMA: with a token or two per adapter the matrix cores would mostly
//    multiply columns that are not wanted, and cutting operands for them costs more than the FMAs.
//  * Many tokens (k_lora_shrink, k_lora_expand): a workgroup walks its tile's adapters (one or two
//    where prompts are runs) on the matrix cores; bound by the bytes of X, Y0 and Y.
//
// Precision: X, H and Y are fp32 and so is the sum. On the matrix cores the products run in bf16
// without rounding any operand: an fp32 value is cut (by truncation) into three bf16 pieces of eight
// significant bits each that add up to it exactly, a bf16 weight is one piece, an fp16 weight
// two and an fp32 weight three, and the piece products are summed in fp32: 3, 6 or 8 MFMAs for
// one (of fp32 weights' nine, the last is left out: below 2^-30 of the whole). fp32 MFMA would
// take 5.3 times the bf16 form's cycles.
#include "bt_internal.h"
#include "convert.h"
#include "wave.h"

namespace bt {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kTile = 16;        // tokens of a tile
constexpr int kWaves = 4;
constexpr int kStepK = 32 * kWaves;  // k of one workgroup step of k_lora_shrink
constexpr int kMaxRank = 256;
constexpr int kFewTokens = 128;      // largest M of the few-tokens kernels
constexpr int kChunkK = 512;         // k of one wave step of k_lora_shrink_few: 8 per lane
constexpr int kGroupTok = 4;         // tokens that share one reading of an adapter there

struct LoraArgs {
    const void *A, *B;
    const float *scale;
    const int *ranks, *adapter;
    const float *X, *Y0;
    float *Y, *ws;
    int64_t M, N, K;
    int L, R, Rp;  // Rp: R rounded up to 16
    int slices, kslice, leads;  // leads: workgroups per tile of the few-tokens kernels
    int vec_x, vec_a, vec_b, vec_y;
    RowGroups groups;
};

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

// Values p[0 .. min(n, 8)) as pieces, zeros behind them (n <= 0: nothing is read). vec: p is
// 16-byte aligned (32 bytes are then read as 16-byte pieces wherever n >= 8).
template <typename W>
__device__ inline Pieces<Terms<W>::n> load_pieces(const W *p, int64_t n, bool vec)
{
    if constexpr (Terms<W>::n == 1) {
        Pieces<1> out;
        out.p[0] = u32x4{0, 0, 0, 0};
        if (vec && n >= 8) {
            out.p[0] = *reinterpret_cast<const u32x4 *>(p);
        } else {
            const uint16_t *h = reinterpret_cast<const uint16_t *>(p);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < n)
                    out.p[0][j / 2] |= (uint32_t)h[j] << (16 * (j & 1));
        }
        return out;
    } else {
        float x[8] = {};
        if (vec && n >= 8) {
            float lo[4], hi[4];
            load4(p, lo);
            load4(p + 4, hi);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[j] = lo[j];
                x[4 + j] = hi[j];
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < n)
                    x[j] = (float)p[j];
        }
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

template <typename W, int RT>
__global__ __launch_bounds__(256) void k_lora_shrink(LoraArgs a)
{
    __shared__ f32x4 part[kWaves][RT][64];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int t = lane & 15, g = lane >> 4;
    const int64_t m0 = (int64_t)blockIdx.x * kTile;
    const int mine = lane_adapter(a, m0, t);
    uint32_t todo = (uint32_t)__ballot(mine >= 0) & 0xFFFFu;
    const int tpg = a.Rp / 16, tiles = tpg * a.groups.n;
    const int64_t k0 = (int64_t)blockIdx.y * a.kslice;
    const int64_t k1 = min(k0 + a.kslice, a.K);
    const float *xrow = a.X + min(m0 + t, a.M - 1) * a.K;

    while (todo) {
        const int lead = __builtin_ctz(todo);
        const int ad = __builtin_amdgcn_readlane(mine, lead);
        const uint32_t same = (uint32_t)__ballot(mine == ad) & 0xFFFFu;
        todo &= ~same;
        const int rank = adapter_rank(a, ad);
        const W *wrow[RT];
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            const int tile = blockIdx.z * RT + i;
            const int r = (tile % tpg) * 16 + t;
            wrow[i] = nullptr;
            if (tile < tiles && r < rank)
                wrow[i] = static_cast<const W *>(a.A) + ((int64_t)ad * a.groups.n * a.R + (tile / tpg) * a.R + r) * a.K;
        }
        f32x4 acc[RT];
#pragma unroll
        for (int i = 0; i < RT; ++i)
            acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 2
        for (int64_t kk = k0 + 32 * wave; kk < k1; kk += kStepK) {
            const int64_t k = kk + 8 * g;
            const Pieces<3> x = load_pieces<float>(xrow + k, k1 - k, a.vec_x);
#pragma unroll
            for (int i = 0; i < RT; ++i)
                acc[i] = mma(load_pieces<W>(wrow[i] + k, wrow[i] ? k1 - k : 0, a.vec_a), x, acc[i]);
        }
#pragma unroll
        for (int i = 0; i < RT; ++i)
            part[wave][i][lane] = acc[i];
        __syncthreads();
        for (int e = threadIdx.x; e < RT * 64; e += 256) {
            const int i = e >> 6, l = e & 63;
            const int tile = blockIdx.z * RT + i;
            if (tile < tiles && (same >> (l & 15) & 1)) {
                f32x4 s = part[0][i][l];
#pragma unroll
                for (int w = 1; w < kWaves; ++w)
                    s += part[w][i][l];
                s *= a.scale[ad];
                const int64_t m = m0 + (l & 15);
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
// memory straight into the MFMA operands (no LDS, no barrier), and Y0 is requested before either, so
// that a wave waits twice: for its tokens' adapters, and for what depends on them.
constexpr int kExpandN = 64, kExpandT = kExpandN / 16;

template <typename W>
__global__ __launch_bounds__(256, 4) void k_lora_expand(LoraArgs a)
{
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int t = lane & 15, g = lane >> 4;
    // token tiles vary fastest over workgroups, outputs over a workgroup's waves
    const int64_t m0 = (int64_t)blockIdx.x * kTile, n0 = ((int64_t)blockIdx.y * 4 + wave) * kExpandN;
    if (n0 >= a.N)
        return;
    const int mine = lane_adapter(a, m0, t);
    f32x4 y[kExpandT];
#pragma unroll
    for (int i = 0; i < kExpandT; ++i) {
        y[i] = f32x4{0.f, 0.f, 0.f, 0.f};
        const int64_t n = n0 + 16 * i + 4 * g;
        if (a.Y0 && m0 + t < a.M) {
            const float *p = a.Y0 + (m0 + t) * a.N + n;
            if (a.vec_y) {
                if (n < a.N)
                    y[i] = *reinterpret_cast<const f32x4 *>(p);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (n + j < a.N)
                        y[i][j] = p[j];
            }
        }
    }
    uint32_t todo = (uint32_t)__ballot(mine >= 0) & 0xFFFFu;
    const int64_t hrow = min(m0 + t, a.M - 1) * a.groups.n, hstep = a.M * a.groups.n * a.Rp;
    while (todo) {
        const int lead = __builtin_ctz(todo);
        const int ad = __builtin_amdgcn_readlane(mine, lead);
        const uint32_t same = (uint32_t)__ballot(mine == ad) & 0xFFFFu;
        todo &= ~same;
        const int rank = adapter_rank(a, ad);
        for (int grp = 0; grp < a.groups.n; ++grp) {
            const int64_t lo = grp ? a.groups.end[grp - 1] : 0, hi = a.groups.end[grp];
            if (hi <= n0 || lo >= n0 + kExpandN)
                continue;
            f32x4 sum[kExpandT];
#pragma unroll
            for (int i = 0; i < kExpandT; ++i)
                sum[i] = f32x4{0.f, 0.f, 0.f, 0.f};
            for (int rr = 0; rr < a.Rp; rr += 32) {
                const int r = rr + 8 * g;
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
#pragma unroll
                for (int i = 0; i < kExpandT; ++i) {
                    const int64_t n = n0 + 16 * i + t;
                    const bool in = n >= lo && n < hi;
                    const W *w = static_cast<const W *>(a.B) + ((int64_t)ad * a.N + (in ? n : lo)) * a.R + r;
                    sum[i] = mma(load_pieces<W>(w, in ? rank - r : 0, a.vec_b), x, sum[i]);
                }
            }
            if (same >> t & 1)
#pragma unroll
                for (int i = 0; i < kExpandT; ++i)
                    y[i] += sum[i];
        }
    }
    if (m0 + t >= a.M)
        return;
#pragma unroll
    for (int i = 0; i < kExpandT; ++i) {
        const int64_t n = n0 + 16 * i + 4 * g;
        float *p = a.Y + (m0 + t) * a.N + n;
        if (a.vec_y) {
            if (n < a.N)
                *reinterpret_cast<f32x4 *>(p) = y[i];
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (n + j < a.N)
                    p[j] = y[i][j];
        }
    }
}

// Eight weights p[0 .. min(n, 8)) as fp32, zeros behind them (n <= 0: nothing is read).
template <typename W>
struct Raw8 {
    u32x4 q[Terms<W>::n == 3 ? 2 : 1];
};
template <typename W>
__device__ inline Raw8<W> load_raw(const W *p, int64_t n, bool vec)
{
    Raw8<W> out;
    if (vec && n >= 8) {
        out.q[0] = *reinterpret_cast<const u32x4 *>(p);
        if constexpr (Terms<W>::n == 3)
            out.q[1] = *reinterpret_cast<const u32x4 *>(p + 4);
        return out;
    }
    out.q[0] = u32x4{0, 0, 0, 0};
    if constexpr (Terms<W>::n == 3) {
        out.q[1] = u32x4{0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < n)
                out.q[j / 4][j % 4] = __float_as_uint(p[j]);
    } else {
        const uint16_t *h = reinterpret_cast<const uint16_t *>(p);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < n)
                out.q[0][j / 2] |= (uint32_t)h[j] << (16 * (j & 1));
    }
    return out;
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

// The leader token of this workgroup of a few-tokens kernel and the tokens that share its adapter;
// false: the token is not the first one of its adapter, or does not exist.
__device__ inline bool lead_tokens(const LoraArgs &a, int64_t m0, int lead, int &ad, uint32_t &same)
{
    const int mine = lane_adapter(a, m0, threadIdx.x & 15);
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

// k_lora_shrink_few: 16 rows of one adapter's A against up to four of its tokens at a time. A lane
// keeps eight k of the tokens in registers; every row is then one contiguous 1 KiB read of the wave,
// all sixteen in flight together. The sixteen rows' partial sums are added over the lanes by swaps
// that halve the number of values each time.
template <typename W>
__global__ __launch_bounds__(256) void k_lora_shrink_few(LoraArgs a)
{
    __shared__ float part[kWaves][kGroupTok][16];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int64_t m0 = (int64_t)(blockIdx.x / a.leads) * kTile;
    int ad;
    uint32_t same;
    if (!lead_tokens(a, m0, blockIdx.x % a.leads, ad, same) || ad < 0)
        return;
    const int tpg = a.Rp / 16, grp = blockIdx.z / tpg, r0 = (blockIdx.z % tpg) * 16;
    const int rank = adapter_rank(a, ad);
    const int rows = min(16, rank - r0);  // may be <= 0: H is 0 there
    const W *w = static_cast<const W *>(a.A) + (((int64_t)ad * a.groups.n + grp) * a.R + r0) * a.K;
    const float scale = a.scale[ad];
    const int64_t k0 = (int64_t)blockIdx.y * a.kslice, k1 = min(k0 + a.kslice, a.K);
    while (same) {
        int tok[kGroupTok];
        const int nt = take_tokens(same, tok);
        float acc[kGroupTok][16];
#pragma unroll
        for (int i = 0; i < kGroupTok; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r)
                acc[i][r] = 0.f;
        for (int64_t kk = k0 + kChunkK * wave; kk < k1; kk += kChunkK * kWaves) {
            const int64_t k = kk + 8 * lane;
            Raw8<W> raw[16];
#pragma unroll
            for (int r = 0; r < 16; ++r)
                raw[r] = load_raw(w + r * a.K + k, r < rows ? k1 - k : 0, a.vec_a);
#pragma unroll
            for (int i = 0; i < kGroupTok; ++i) {
                if (i >= nt)
                    break;
                const Raw8<float> xr = load_raw(a.X + (m0 + tok[i]) * a.K + k, k1 - k, a.vec_x);
                float x[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    x[j] = raw_value(xr, j);
#pragma unroll
                for (int r = 0; r < 16; ++r)
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        acc[i][r] = __builtin_fmaf(raw_value(raw[r], j), x[j], acc[i][r]);
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
            a.ws[(((int64_t)blockIdx.y * a.M + m0 + m) * a.groups.n + grp) * a.Rp + r0 + r] = s * scale;
        }
        if (same)
            __syncthreads();
    }
}

// k_lora_expand_few: 256 outputs of one adapter's tokens. A lane has one output, i.e. one row of B,
// whose first 64 values are requested before H is waited for; H is the same for all lanes (LDS
// broadcasts). Tokens without an adapter are one more group, which only copies Y0.
constexpr int kFewN = 256, kFewR = 64;

template <typename W>
__global__ __launch_bounds__(256) void k_lora_expand_few(LoraArgs a)
{
    __shared__ __attribute__((aligned(16))) float hs[kGroupTok][kMaxRank];
    const int64_t m0 = (int64_t)(blockIdx.x / a.leads) * kTile;
    const int64_t nb = (int64_t)blockIdx.y * kFewN, n = nb + threadIdx.x;
    int ad;
    uint32_t same;
    if (!lead_tokens(a, m0, blockIdx.x % a.leads, ad, same))
        return;
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
    const W *w = static_cast<const W *>(a.B) + ((int64_t)ad * a.N + min(n, a.N - 1)) * a.R;
    Raw8<W> raw[kFewR / 8];
#pragma unroll
    for (int c = 0; c < kFewR / 8; ++c)
        raw[c] = load_raw(w + 8 * c, rank - 8 * c, a.vec_b);
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
                    v[c] = r0 ? load_raw(w + r0 + 8 * c, rank - r0 - 8 * c, a.vec_b) : raw[c];
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

LoraPlan lora_plan(int64_t M, int64_t K, int64_t R, int64_t groups)
{
    LoraPlan p;
    const int64_t rank_tiles = round_up(R, 16) / 16 * groups;
    p.few = M <= kFewTokens;
    p.rt = p.few ? 1 : rank_tiles >= 3 ? 4 : (int)rank_tiles;
    p.ztiles = (rank_tiles + p.rt - 1) / p.rt;
    p.tiles = (M + kTile - 1) / kTile;
    p.leads = (int)(M < kTile ? M : kTile);
    // K in as many slices as give about four workgroups per CU, each at least one wave step, and no
    // more than eight (the expand kernels read every slice's partial sums).
    const int64_t wgs = (p.few ? p.tiles * p.leads : p.tiles) * p.ztiles;
    const int64_t unit = p.few ? kChunkK : kStepK;             // smallest slice
    const int64_t whole = p.few ? kChunkK * kWaves : kStepK;   // k of a workgroup step
    const int64_t steps = K > 0 ? (K + whole - 1) / whole : 1;
    int64_t slices = (1024 + wgs - 1) / wgs;
    slices = slices < steps ? slices : steps;
    slices = slices < 8 ? slices : 8;
    const int64_t k = K > 0 ? K : 1;
    p.kslice = round_up((k + slices - 1) / slices, unit);
    p.slices = (int)((k + p.kslice - 1) / p.kslice);
    return p;
}

bool al16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

template <typename W>
hipError_t launch_weights(const LoraArgs &a, const LoraPlan &p, hipStream_t s)
{
    if (p.few) {
        const unsigned gx = (unsigned)(p.tiles * p.leads);
        k_lora_shrink_few<W><<<dim3(gx, (unsigned)p.slices, (unsigned)p.ztiles), 256, 0, s>>>(a);
        if (hipError_t e = hipGetLastError())
            return e;
        k_lora_expand_few<W><<<dim3(gx, (unsigned)((a.N + kFewN - 1) / kFewN)), 256, 0, s>>>(a);
        return hipGetLastError();
    }
    const dim3 shrink((unsigned)p.tiles, (unsigned)p.slices, (unsigned)p.ztiles);
    if (p.rt == 1)
        k_lora_shrink<W, 1><<<shrink, 256, 0, s>>>(a);
    else if (p.rt == 2)
        k_lora_shrink<W, 2><<<shrink, 256, 0, s>>>(a);
    else
        k_lora_shrink<W, 4><<<shrink, 256, 0, s>>>(a);
    if (hipError_t e = hipGetLastError())
        return e;
    const dim3 expand((unsigned)p.tiles, (unsigned)((a.N + 4 * kExpandN - 1) / (4 * kExpandN)));
    k_lora_expand<W><<<expand, 256, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

size_t lora_workspace_bytes(int64_t M, int64_t K, int64_t R, int64_t groups)
{
    return (size_t)lora_plan(M, K, R, groups).slices * M * groups * round_up(R, 16) * 4;
}

hipError_t launch_lora(const void *A, const void *B, int w_type, const float *scale, const int32_t *ranks, int64_t L,
                       int64_t R, const RowGroups &groups, const int32_t *adapter, const float *X, const float *Y0,
                       int64_t M, int64_t N, int64_t K, float *Y, void *workspace, hipStream_t s)
{
    const LoraPlan p = lora_plan(M, K, R, groups.n);
    const int wb = type_bytes(w_type);
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
    a.leads = p.leads;
    a.slices = p.slices;
    a.kslice = (int)p.kslice;
    a.vec_x = al16(X) && K % 4 == 0;
    a.vec_a = al16(A) && K * wb % 16 == 0;
    a.vec_b = al16(B) && R * wb % 16 == 0;
    a.vec_y = al16(Y) && (!Y0 || al16(Y0)) && N % 4 == 0;
    a.groups = groups;
    switch (w_type) {
    case kBF16: return launch_weights<bf16_t>(a, p, s);
    case kF16: return launch_weights<f16_t>(a, p, s);
    default: return launch_weights<float>(a, p, s);
    }
}

}  // namespace bt
