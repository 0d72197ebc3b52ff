// Low-rank adapters of many requests beside one shared projection (bt_lora_apply):
//
//   Y[m, n] = Y0[m, n] + scale[a] * sum_{r < rank[a]} H[m, g(n), r] * B[a, n, r]
//   H[m, g, r] = sum_k X[m, k] * A[a, g R + r, k]          a = adapter[m], g(n) = row group of n
//
// Two launches: k_lora_shrink forms H (times the scale) into the workspace, as one partial per
// slice of K; k_lora_expand adds the partials in their order, multiplies by B and adds Y0. No
// atomics: results do not depend on the order in which workgroups run.
//
// Precision: X, H and Y are fp32 and so is the sum. The products run on bf16 MFMA without
// rounding any operand: an fp32 value is cut (by truncation) into three bf16 pieces of eight
// significant bits each that add up to it exactly, a bf16 weight is one piece, an fp16 weight
// two and an fp32 weight three, and the piece products are summed in fp32: 3, 6 or 8 MFMAs for
// one (of fp32 weights' nine, the last is left out: below 2^-30 of the whole). fp32 MFMA would
// take 5.3 times the bf16 form's cycles.
//
// Adapters of a tile of 16 tokens: the tile is worked off adapter by adapter, each adapter's
// weights being read once for all of the tile's tokens that use it. A token is a column of the
// MFMA's result, so the other tokens' columns of a pass are simply not taken: an adapter's
// weights, whatever they hold, never reach a token that does not use it.
//  * few tokens (`par`): a workgroup per (tile, first token of an adapter), so that a decode
//    batch's adapters are read side by side;
//  * many tokens: one workgroup walks its tile's adapters (one or two where prompts are runs).
#include "bt_internal.h"
#include "convert.h"

namespace bt {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kTile = 16;        // tokens of a tile
constexpr int kWaves = 4;
constexpr int kStepK = 32 * kWaves;  // k of one workgroup step of k_lora_shrink
constexpr int kMaxRank = 256;

struct LoraArgs {
    const void *A, *B;
    const float *scale;
    const int *ranks, *adapter;
    const float *X, *Y0;
    float *Y, *ws;
    int64_t M, N, K;
    int L, R, Rp;  // Rp: R rounded up to 16
    int par, slices, kslice;
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
    const int64_t m0 = (int64_t)(a.par ? blockIdx.x / kTile : blockIdx.x) * kTile;
    const int mine = lane_adapter(a, m0, t);
    uint32_t todo = (uint32_t)__ballot(mine >= 0) & 0xFFFFu;
    if (a.par)
        todo &= 1u << (blockIdx.x % kTile);
    const int tpg = a.Rp / 16, tiles = tpg * a.groups.n;
    const int64_t k0 = (int64_t)blockIdx.y * a.kslice;
    const int64_t k1 = min(k0 + a.kslice, a.K);
    const float *xrow = a.X + min(m0 + t, a.M - 1) * a.K;

    while (todo) {
        const int lead = __builtin_ctz(todo);
        const int ad = __builtin_amdgcn_readlane(mine, lead);
        const uint32_t same = (uint32_t)__ballot(mine == ad) & 0xFFFFu;
        if (a.par && __builtin_ctz(same) != lead)
            return;
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

constexpr int kExpandN = 256;  // output columns of a workgroup: 64 per wave

template <typename W>
__global__ __launch_bounds__(256) void k_lora_expand(LoraArgs a)
{
    __shared__ __attribute__((aligned(16))) float hs[kTile][kMaxRank + 4];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int t = lane & 15, g = lane >> 4;
    const int64_t m0 = (int64_t)(a.par ? blockIdx.x / kTile : blockIdx.x) * kTile;
    const int mine = lane_adapter(a, m0, t);
    const uint32_t real = (uint32_t)__ballot(mine >= -1) & 0xFFFFu;
    uint32_t todo = real;
    const int64_t nb = (int64_t)blockIdx.y * kExpandN, n0 = nb + 64 * wave;
    if (a.par) {
        const int lead = blockIdx.x % kTile;
        if (!(todo >> lead & 1))
            return;
        const int ad = __builtin_amdgcn_readlane(mine, lead);
        const uint32_t same = (uint32_t)__ballot(mine == ad) & 0xFFFFu;
        if (__builtin_ctz(same) != lead)
            return;
        todo = same;
    }
    const uint32_t stored = todo;
    f32x4 acc[4], base[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        acc[i] = base[i] = f32x4{0.f, 0.f, 0.f, 0.f};
        const int64_t n = n0 + 16 * i + 4 * g;
        if (a.Y0 && (stored >> t & 1)) {
            const float *p = a.Y0 + (m0 + t) * a.N + n;
            if (a.vec_y) {
                if (n < a.N)
                    base[i] = *reinterpret_cast<const f32x4 *>(p);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (n + j < a.N)
                        base[i][j] = p[j];
            }
        }
    }
    todo &= (uint32_t)__ballot(mine >= 0);
    while (todo) {
        const int lead = __builtin_ctz(todo);
        const int ad = __builtin_amdgcn_readlane(mine, lead);
        const uint32_t same = (uint32_t)__ballot(mine == ad) & 0xFFFFu;
        todo &= ~same;
        const int rank = adapter_rank(a, ad);
        for (int grp = 0; grp < a.groups.n; ++grp) {
            const int64_t lo = grp ? a.groups.end[grp - 1] : 0, hi = a.groups.end[grp];
            if (hi <= nb || lo >= nb + kExpandN)
                continue;
            __syncthreads();  // the last group's reads of hs are done
            for (int e = threadIdx.x; e < kTile * (a.Rp / 4); e += 256) {
                const int tt = e / (a.Rp / 4), r = e % (a.Rp / 4) * 4;
                f32x4 s = f32x4{0.f, 0.f, 0.f, 0.f};
                if (same >> tt & 1) {
                    const float *src = a.ws + ((m0 + tt) * a.groups.n + grp) * a.Rp + r;
                    const int64_t step = a.M * a.groups.n * a.Rp;
                    for (int i = 0; i < a.slices; ++i)
                        s += *reinterpret_cast<const f32x4 *>(src + i * step);
                }
                *reinterpret_cast<f32x4 *>(&hs[tt][r]) = s;
            }
            __syncthreads();
            f32x4 sum[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                sum[i] = f32x4{0.f, 0.f, 0.f, 0.f};
            for (int rr = 0; rr < a.Rp; rr += 32) {
                const int r = rr + 8 * g;
                float h[8] = {};
                if (r < a.Rp) {
                    const f32x4 h0 = *reinterpret_cast<const f32x4 *>(&hs[t][r]);
                    const f32x4 h1 = *reinterpret_cast<const f32x4 *>(&hs[t][r + 4]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        h[j] = h0[j];
                        h[4 + j] = h1[j];
                    }
                }
                const Pieces<3> x = cut<3>(h);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int64_t n = n0 + 16 * i + t;
                    const bool in = n >= lo && n < hi;
                    const W *w = static_cast<const W *>(a.B) + ((int64_t)ad * a.N + (in ? n : lo)) * a.R + r;
                    sum[i] = mma(load_pieces<W>(w, in ? rank - r : 0, a.vec_b), x, sum[i]);
                }
            }
            if (same >> t & 1)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    acc[i] += sum[i];
        }
    }
    if (!(stored >> t & 1))
        return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t n = n0 + 16 * i + 4 * g;
        const f32x4 y = base[i] + acc[i];
        float *p = a.Y + (m0 + t) * a.N + n;
        if (a.vec_y) {
            if (n < a.N)
                *reinterpret_cast<f32x4 *>(p) = y;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (n + j < a.N)
                    p[j] = y[j];
        }
    }
}

struct LoraPlan {
    int par, rt, slices;
    int64_t kslice, tiles, ztiles;
};

LoraPlan lora_plan(int64_t M, int64_t K, int64_t R, int64_t groups)
{
    LoraPlan p;
    const int64_t rank_tiles = round_up(R, 16) / 16 * groups;
    p.par = M <= 128;
    p.rt = p.par ? 1 : rank_tiles >= 3 ? 4 : (int)rank_tiles;
    p.ztiles = (rank_tiles + p.rt - 1) / p.rt;
    p.tiles = (M + kTile - 1) / kTile;
    // K in as many slices as give about four workgroups per CU, each at least one step.
    const int64_t wgs = p.par ? M * p.ztiles : p.tiles * p.ztiles;
    const int64_t steps = K > 0 ? (K + kStepK - 1) / kStepK : 1;
    int64_t slices = (1024 + wgs - 1) / wgs;
    slices = slices < steps ? slices : steps;
    slices = slices < 32 ? slices : 32;
    p.kslice = (steps + slices - 1) / slices * kStepK;
    p.slices = (int)((steps * kStepK + p.kslice - 1) / p.kslice);
    return p;
}

bool al16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

template <typename W>
hipError_t launch_weights(const LoraArgs &a, const LoraPlan &p, hipStream_t s)
{
    const unsigned gx = (unsigned)(p.tiles * (p.par ? kTile : 1));
    const dim3 shrink(gx, (unsigned)p.slices, (unsigned)p.ztiles);
    if (p.rt == 1)
        k_lora_shrink<W, 1><<<shrink, 256, 0, s>>>(a);
    else if (p.rt == 2)
        k_lora_shrink<W, 2><<<shrink, 256, 0, s>>>(a);
    else
        k_lora_shrink<W, 4><<<shrink, 256, 0, s>>>(a);
    if (hipError_t e = hipGetLastError())
        return e;
    const dim3 expand(gx, (unsigned)((a.N + kExpandN - 1) / kExpandN));
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
    a.par = p.par;
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
