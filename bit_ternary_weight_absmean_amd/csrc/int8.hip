// Products of int8 tokens and int8 weights (bt_int8_gemm): acc[m,n] = sum_k W[n,k] X[m,k] in int32, exact, and
// Y[m,n] = fp32(acc) * (x_scale[m] * w_scale[n]) + bias[n].
//
// Weights are packed once (bt_int8_pack) into blocks of 16 rows x 64 k, 1 KB each, byte 16 * (r + 16 g) + e of a
// block holding row r, k = 16 g + e: the operand of v_mfma_i32_16x16x64_i8 as its 64 lanes take it, so that a wave
// reads a block as one contiguous KB, from memory and from LDS. Rows of the product are weight rows, columns tokens:
// a lane then holds four outputs of one token that lie side by side.
//
// Up to 64 tokens go to k_int8_few, which streams the weights past the matrix cores without LDS; more to k_int8_tile.
#include <type_traits>

#include "bt_internal.h"
#include "convert.h"

namespace bt {
namespace {

typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(1))) const void global_void;

__global__ __launch_bounds__(256) void k_int8_pack(const int8_t *W, int64_t ld, int64_t N, int64_t K, int64_t pieces,
                                                   int64_t KC, char *Wp)
{
    const int64_t step = (int64_t)gridDim.x * 256;
    for (int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x; id < pieces; id += step) {  // 16 bytes of Wp
        const int64_t block = id >> 6;
        const int lane = (int)(id & 63);
        const int64_t n = block / KC * 16 + (lane & 15), k = block % KC * 64 + 16 * (lane >> 4);
        v4i x = {0, 0, 0, 0};
        if (n < N && k + 16 <= K) {
            typedef int unaligned __attribute__((ext_vector_type(4), aligned(1)));
            x = *reinterpret_cast<const unaligned *>(W + n * ld + k);
        } else if (n < N) {
            for (int e = 0; e < 16 && k + e < K; ++e)
                x[e / 4] |= (int)((uint32_t)(uint8_t)W[n * ld + k + e] << 8 * (e % 4));
        }
        *reinterpret_cast<v4i *>(Wp + id * 16) = x;
    }
}

struct Int8Args {
    const char *Wp;
    const float *w_scale, *x_scale, *bias;
    const int8_t *X;
    void *Y;
    int *acc;
    int64_t M, N, ldx;
    int KC, NB;       // 64-k blocks of a row, 16-row blocks
    int wide;         // four outputs side by side can be stored at once
    int pieces;       // rows of Y are whole 16-byte pieces, 16-byte aligned
    int tiles_m, tiles_n;
};

// Four outputs of token m from column n on.
template <typename TY>
__device__ inline void store_outputs(const Int8Args &a, int64_t m, int64_t n, v4i c, float xs, const float (&ws)[4],
                                     const float (&bias)[4], bool with_y)
{
    float y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        y[i] = (float)c[i] * (xs * ws[i]);
        if (a.bias)
            y[i] = y[i] + bias[i];
    }
    const int64_t at = m * a.N + n;
    if (a.wide && n + 4 <= a.N) {
        if (a.acc)
            *reinterpret_cast<v4i *>(a.acc + at) = c;
        if (a.Y && with_y)
            store4(static_cast<TY *>(a.Y) + at, y);
        return;
    }
    for (int i = 0; i < 4 && n + i < a.N; ++i) {
        if (a.acc)
            a.acc[at + i] = c[i];
        if (a.Y && with_y)
            static_cast<TY *>(a.Y)[at + i] = (TY)y[i];
    }
}

__device__ inline void load_scales(const Int8Args &a, int64_t n, float (&ws)[4], float (&bias)[4])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t at = min(n + i, a.N - 1);
        ws[i] = a.w_scale[at];
        bias[i] = a.bias ? a.bias[at] : 0.f;
    }
}

// At most VM of the wave's direct loads are on their way, its LDS reads are done.
// (The wait is the builtin, which the compiler counts as its own: an asm one it does not see, and adds others.)
template <int VM>
__device__ inline void landed()
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt((VM & 0xF) | (VM >> 4) << 14 | 0x7 << 4);
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
}

// A read of 16 bytes by 64 lanes goes in groups of sixteen, lanes 0-3, 12-15, 20-27 and their like: with r = lane % 16
// and g = lane / 16, quarters 0 and 3 of r at one g, 1 and 2 at its neighbour. A block of sixteen tokens x 64 k lies in
// LDS as rows of 64 bytes, whose 16-byte piece p is at place p ^ piece_place(row): g ^ piece_place is different in the four
// quarters of a group, so that its pieces lie in different places of a 256-byte line. (With the quarter's own
// number: 40% of the LDS cycles were conflicts.)
__device__ inline int piece_place(int row) { return (row >> 1 & 2) ^ (row >> 3 & 1) * 3; }

// ------------------------------------------------------------------------------ few tokens
//
// k_int8_few: 16 RT weight rows against 16 MT tokens by W waves, which take every W-th 64-k block each (side by side, so
// that the workgroup streams whole rows of blocks) and are joined through LDS. Weights go from memory straight into
// registers, RING blocks ahead. So do tokens where weights are what there is to read (DIRECT; with RING == 2 more
// workgroups fit a CU); in few workgroups they take a direct way into a piece of LDS of the wave's own, since a lane's
// 16 bytes of 16 rows cost the load path more than 64 bytes side by side do.
// Bound by the weights' bytes: 1 x 32000 x 2560 in 12.1 us (6.8 TB/s, more than from memory alone: part of the 82 MB is
// still in the last cache from the call before), 40 x 28672 x 8192 48.2 us (4.9 TB/s; a large copy 5.2).

template <typename TY, int RT, int MT, int RING, int W, bool DIRECT>
__global__ __launch_bounds__(64 * W) void k_int8_few(Int8Args a)
{
    static_assert(DIRECT || RING == 4, "four stages in LDS");
    constexpr int kStagesUsed = DIRECT ? 1 : 4;
    constexpr int kEach = DIRECT ? RT * MT : MT > RT * MT / 4 ? MT : RT * MT / 4;  // KB of a wave in a stage
    constexpr int kPart = kEach * 1024;
    static_assert(kEach * kStagesUsed >= RT * MT, "room for the waves' results");
    __shared__ __attribute__((aligned(1024))) char ring0[W * kPart], ring1[DIRECT ? 16 : W * kPart],
        ring2[DIRECT ? 16 : W * kPart], ring3[DIRECT ? 16 : W * kPart];
    auto stage = [&](auto sc) -> char * {
        constexpr int S = decltype(sc)::value;
        if constexpr (S == 0)
            return ring0;
        else if constexpr (S == 1)
            return ring1;
        else if constexpr (S == 2)
            return ring2;
        else
            return ring3;
    };
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int r = lane & 15, g = lane >> 4;
    const int rb0 = blockIdx.x * RT;
    const int64_t m0 = (int64_t)blockIdx.y * (16 * MT);

    const char *w[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i)
        w[i] = a.Wp + (int64_t)min(rb0 + i, a.NB - 1) * a.KC * 1024 + lane * 16;
    const int8_t *x[MT];
#pragma unroll
    for (int j = 0; j < MT; ++j) {
        const int row = DIRECT ? r : lane >> 2, p = DIRECT ? g : (lane & 3) ^ piece_place(row);
        x[j] = a.X + min(m0 + 16 * j + row, a.M - 1) * a.ldx + 16 * p;
    }
    const int x_off = wave * kPart + r * 64 + ((g ^ piece_place(r)) << 4);

    v4i c[RT][MT];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < MT; ++j)
            c[i][j] = v4i{0, 0, 0, 0};
    const int n = (a.KC - wave + W - 1) / W;  // blocks of this wave (none: <= 0)
    v4i wf[RING][RT], xf[DIRECT ? RING : 1][MT];
    auto fetch = [&](auto sc, int k) __attribute__((always_inline)) {
        constexpr int S = decltype(sc)::value;
        const int64_t at = wave + (int64_t)min(k, n - 1) * W;  // past the end: the last one again, not used
#pragma unroll
        for (int j = 0; j < MT; ++j)
            if constexpr (DIRECT)
                xf[S][j] = *reinterpret_cast<const v4i *>(x[j] + at * 64);
            else
                __builtin_amdgcn_global_load_lds((global_void *)(x[j] + at * 64),
                                                 (lds_void *)(stage(sc) + wave * kPart + j * 1024), 16, 0, 0);
#pragma unroll
        for (int i = 0; i < RT; ++i)
            wf[S][i] = __builtin_nontemporal_load(reinterpret_cast<const v4i *>(w[i] + at * 1024));
    };
    auto multiply = [&](const v4i (&wv)[RT], const v4i (&xv)[MT]) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int j = 0; j < MT; ++j)
                c[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wv[i], xv[j], c[i][j], 0, 0, 0);
    };
    // MORE: loads of three further steps are on their way, and this one's places are filled again
    auto step = [&](auto sc, int k, auto more) __attribute__((always_inline)) {
        constexpr int S = decltype(sc)::value;
        constexpr bool MORE = decltype(more)::value;
        if constexpr (DIRECT) {
            multiply(wf[S], xf[S]);
        } else {
            landed<MORE ? (RING - 1) * (RT + MT) : 0>();
#pragma unroll
            for (int j = 0; j < MT; ++j)
                xf[0][j] = *reinterpret_cast<const v4i *>(stage(sc) + x_off + j * 1024);
            multiply(wf[S], xf[0]);
            if constexpr (MORE)
                landed<(RING - 1) * (RT + MT)>();  // the reads, before the stage is filled again
        }
        if constexpr (MORE)
            fetch(sc, k + RING);
    };
    using More = std::true_type;
    using NoMore = std::false_type;
    using I0 = std::integral_constant<int, 0>;
    using I1 = std::integral_constant<int, 1>;
    using I2 = std::integral_constant<int, 2>;
    using I3 = std::integral_constant<int, 3>;
    if (n > 0) {
        fetch(I0{}, 0);
        fetch(I1{}, 1);
        if constexpr (RING > 2) {
            fetch(I2{}, 2);
            fetch(I3{}, 3);
        }
        int k = 0;
        for (; k + RING <= n; k += RING) {
            step(I0{}, k, More{});
            step(I1{}, k + 1, More{});
            if constexpr (RING > 2) {
                step(I2{}, k + 2, More{});
                step(I3{}, k + 3, More{});
            }
        }
        if (k < n)
            step(I0{}, k, NoMore{});
        if constexpr (RING > 2) {
            if (k + 1 < n)
                step(I1{}, k + 1, NoMore{});
            if (k + 2 < n)
                step(I2{}, k + 2, NoMore{});
        }
        landed<0>();
    }
    __syncthreads();  // no load is on its way to LDS
    // the results take the stages' room: kEach tiles of a wave in each
    auto place = [&](int v, int t) -> v4i * {
        const int s = t / kEach;
        char *p = s == 0 ? ring0 : s == 1 ? ring1 : s == 2 ? ring2 : ring3;
        return reinterpret_cast<v4i *>(p + v * kPart + t % kEach * 1024);
    };
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < MT; ++j)
            place(wave, i * MT + j)[lane] = c[i][j];
    __syncthreads();
    // four outputs of a token each; threads side by side along the row
    for (int q = threadIdx.x; q < RT * MT * 64; q += 64 * W) {
        const int t = q / (4 * RT), rest = q % (4 * RT), i = rest / 4, quad = rest % 4;
        const int64_t m = m0 + t, row = (int64_t)(rb0 + i) * 16 + 4 * quad;
        if (m >= a.M || row >= a.N)
            continue;
        v4i sum = {0, 0, 0, 0};
#pragma unroll
        for (int v = 0; v < W; ++v)
            sum += place(v, i * MT + t / 16)[16 * quad + t % 16];
        float ws[4], bias[4];
        load_scales(a, row, ws, bias);
        store_outputs<TY>(a, m, row, sum, a.x_scale[m], ws, bias, true);
    }
}

// ------------------------------------------------------------------------------- many tokens
//
// k_int8_tile: BM tokens x BN weight rows by WM x WN waves; 64 k a step through a ring of four LDS stages filled by
// direct loads. A stage holds the weights' blocks as they are and the tokens as rows of 64 bytes, whose 16-byte piece p
// lies at place p ^ piece_place(row); four lanes of a load read 64 neighbouring bytes.
//
// A step is two halves of the wave's tokens. While the first one's MFMAs run, the second's operands are read; then one
// barrier publishes the next stage and frees this one for the load four steps ahead; while the second half's MFMAs run,
// the next step's weights and first tokens are read.
// Bound by the matrix cores at the clock that the power leaves them: 4096 x 28672 x 8192 in 727 us (2.65 POP/s where the
// library's product has 2.17; median of 40 under the tracer 765, least 730; in bursts of five, which the power limit
// hardly reaches, 622), at 1.6 to 1.9 GHz. Steps of 128 k, matrix instructions of 32 x 32 x 32, four waves of
// 128 x 128 or a ring of eight stages: slower or no gain.


// The same for all waves of the workgroup.
template <int VM>
__device__ inline void meet()
{
    landed<VM>();
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
}

// The order of a half step: READS reads of LDS, then LOADS direct loads, each behind one of the first of its MMAS matrix
// instructions, so that the reads are back when the next half needs them.
template <int READS, int LOADS, int MMAS>
__device__ __forceinline__ void interleave()
{
    if constexpr (MMAS > 0) {
        __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
        if constexpr (READS > 0)
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        else if constexpr (LOADS > 0)
            __builtin_amdgcn_sched_group_barrier(0x20, 1, 0);
        interleave<(READS > 0 ? READS - 1 : 0), (READS > 0 || LOADS == 0 ? LOADS : LOADS - 1), MMAS - 1>();
    }
}

constexpr int kStages = 4;

template <typename TY, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN, 2) void k_int8_tile(Int8Args a)
{
    constexpr int WAVES = WM * WN, TM = BM / WM / 16, TN = BN / WN / 16;  // 16 x 16 tiles of a wave
    constexpr int XB = BM / 16, WB = BN / 16;                            // 1 KB blocks of a stage
    constexpr int LX = XB / WAVES, LW = WB / WAVES;                      // of them, by a wave
    constexpr int HALF = TM / 2;
    constexpr int kBytes = (XB + WB) * 1024;
    static_assert(XB % WAVES == 0 && WB % WAVES == 0 && TM % 2 == 0, "blocks split evenly over waves");
    __shared__ __attribute__((aligned(1024))) char lds0[kBytes], lds1[kBytes], lds2[kBytes], lds3[kBytes];
    __shared__ __attribute__((aligned(16))) float s_w[BN], s_bias[BN], s_x[BM];
    auto stage = [&](auto sc) -> char * {
        constexpr int S = decltype(sc)::value % kStages;
        if constexpr (S == 0)
            return lds0;
        else if constexpr (S == 1)
            return lds1;
        else if constexpr (S == 2)
            return lds2;
        else
            return lds3;
    };
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int r = lane & 15, g = lane >> 4;
    const int wm = wave % WM, wn = wave / WM;

    // Workgroup b runs on XCD b % 8: every XCD takes a contiguous run of a tile order that goes through groups of
    // kGroup token tiles column by column, so that what runs on it at a time shares its operands in its L2.
    constexpr int kGroup = 8, kXcd = 8;
    const int total = a.tiles_m * a.tiles_n, run = (total + kXcd - 1) / kXcd;
    const int t = blockIdx.x % kXcd * run + blockIdx.x / kXcd;
    if (blockIdx.x / kXcd >= run || t >= total)
        return;
    const int gid = t / (kGroup * a.tiles_n), in = t - gid * kGroup * a.tiles_n;
    const int rows = min(kGroup, a.tiles_m - gid * kGroup);
    const int64_t m0 = (int64_t)(gid * kGroup + in % rows) * BM;
    const int tn = in / rows, rb0 = tn * WB;

    // scales, for the end
    for (int i = threadIdx.x; i < BN; i += 64 * WAVES) {
        const int64_t n = min((int64_t)rb0 * 16 + i, a.N - 1);
        s_w[i] = a.w_scale[n];
        s_bias[i] = a.bias ? a.bias[n] : 0.f;
    }
    for (int i = threadIdx.x; i < BM; i += 64 * WAVES)
        s_x[i] = a.x_scale[min(m0 + i, a.M - 1)];

    // this wave's direct loads; rows past the last read the last
    const int8_t *xp[LX];
    const char *wp[LW];
#pragma unroll
    for (int i = 0; i < LX; ++i) {
        const int row = lane >> 2, p = (lane & 3) ^ piece_place(row);
        xp[i] = a.X + min(m0 + (wave * LX + i) * 16 + row, a.M - 1) * a.ldx + 16 * p;
    }
#pragma unroll
    for (int i = 0; i < LW; ++i)
        wp[i] = a.Wp + (int64_t)min(rb0 + wave * LW + i, a.NB - 1) * a.KC * 1024 + lane * 16;
    const int last = a.KC - 1;
    auto issue = [&](int k, char *dst) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < LX; ++i)
            __builtin_amdgcn_global_load_lds((global_void *)(xp[i] + (int64_t)k * 64),
                                             (lds_void *)(dst + (wave * LX + i) * 1024), 16, 0, 0);
#pragma unroll
        for (int i = 0; i < LW; ++i)
            __builtin_amdgcn_global_load_lds((global_void *)(wp[i] + (int64_t)k * 1024),
                                             (lds_void *)(dst + (XB + wave * LW + i) * 1024), 16, 0, 0);
    };
    const int x_off = wm * TM * 1024 + r * 64 + ((g ^ piece_place(r)) << 4);
    const int w_off = (XB + wn * TN) * 1024 + lane * 16;
    v4i acc[TN][TM];
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int j = 0; j < TM; ++j)
            acc[i][j] = v4i{0, 0, 0, 0};
    v4i wf[2][TN], xf[2][HALF];
    auto read_w = [&](const char *s, v4i (&f)[TN]) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < TN; ++i)
            f[i] = *reinterpret_cast<const v4i *>(s + w_off + i * 1024);
    };
    auto read_x = [&](const char *s, int half, v4i (&f)[HALF]) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < HALF; ++j)
            f[j] = *reinterpret_cast<const v4i *>(s + x_off + (half * HALF + j) * 1024);
    };
    auto multiply = [&](const v4i (&w)[TN], const v4i (&x)[HALF], int half) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < HALF; ++j)
#pragma unroll
            for (int i = 0; i < TN; ++i)
                acc[i][half * HALF + j] =
                    __builtin_amdgcn_mfma_i32_16x16x64_i8(w[i], x[j], acc[i][half * HALF + j], 0, 0, 0);
    };
    auto step = [&](auto sc, int k) __attribute__((always_inline)) {
        constexpr int S = decltype(sc)::value;
        char *now = stage(sc);
        const char *next = stage(std::integral_constant<int, S + 1>{});
        read_x(now, 1, xf[1]);
        multiply(wf[S % 2], xf[0], 0);
        interleave<HALF, 0, TN * HALF>();
        // the next stage has landed (two more may be on their way), this one's operands are read
        meet<(kStages - 2) * (LX + LW)>();
        issue(min(k + kStages, last), now);  // past the end: the last one again, not used
        read_w(next, wf[(S + 1) % 2]);
        read_x(next, 0, xf[0]);
        multiply(wf[S % 2], xf[1], 1);
        interleave<TN + HALF, LX + LW, TN * HALF>();
        __builtin_amdgcn_sched_barrier(0);
    };
    using I0 = std::integral_constant<int, 0>;
    using I1 = std::integral_constant<int, 1>;
    using I2 = std::integral_constant<int, 2>;
    using I3 = std::integral_constant<int, 3>;
    issue(0, lds0);
    issue(min(1, last), lds1);
    issue(min(2, last), lds2);
    issue(min(3, last), lds3);
    meet<(kStages - 1) * (LX + LW)>();
    read_w(lds0, wf[0]);
    read_x(lds0, 0, xf[0]);
    int k = 0;
    for (; k + kStages <= a.KC; k += kStages) {
        step(I0{}, k);
        step(I1{}, k + 1);
        step(I2{}, k + 2);
        step(I3{}, k + 3);
    }
    if (k <= last)
        step(I0{}, k);
    if (k + 1 <= last)
        step(I1{}, k + 1);
    if (k + 2 <= last)
        step(I2{}, k + 2);
    meet<0>();  // no load is on its way to LDS, all reads are done: the stages are free

    // Outputs. A lane has four of a token side by side, and storing those writes 32 bytes of 16 rows at a time (7 rounds of
    // tiles of a 4096 x 28672 product: 190 us). Rows of whole 16-byte pieces go through the wave's part of the stages
    // instead, and leave as 128 or 256 bytes of a row.
    const int64_t mw = m0 + wm * TM * 16, nw = (int64_t)(rb0 + wn * TN) * 16;
    const bool pieces = a.Y && a.pieces;
    if (pieces) {
        constexpr int ROW = 16 * TN * (int)sizeof(TY), PIECES = ROW / 16;  // bytes and pieces of a wave's row
        constexpr int PART = 16384, TOKENS = PART / ROW < 16 * TM ? PART / ROW : 16 * TM;
        static_assert(PART * WAVES == kStages * kBytes && kBytes % PART == 0, "a part each");
        static_assert(TOKENS % 16 == 0 && 16 * TM % TOKENS == 0, "whole tiles at a time");
        const int at = wave * PART / kBytes;
        char *mine = (at == 0 ? lds0 : at == 1 ? lds1 : at == 2 ? lds2 : lds3) + wave * PART % kBytes;
#pragma unroll
        for (int j0 = 0; j0 < TM; j0 += TOKENS / 16) {
#pragma unroll
            for (int i = 0; i < TN; ++i) {
                const float4 ws = *reinterpret_cast<const float4 *>(s_w + (wn * TN + i) * 16 + 4 * g);
                const float4 bias = *reinterpret_cast<const float4 *>(s_bias + (wn * TN + i) * 16 + 4 * g);
#pragma unroll
                for (int j = 0; j < TOKENS / 16; ++j) {
                    const v4i c = acc[i][j0 + j];
                    const float xs = s_x[(wm * TM + j0 + j) * 16 + r];
                    float y[4] = {(float)c[0] * (xs * ws.x), (float)c[1] * (xs * ws.y), (float)c[2] * (xs * ws.z),
                                  (float)c[3] * (xs * ws.w)};
                    if (a.bias) {
                        y[0] = y[0] + bias.x;
                        y[1] = y[1] + bias.y;
                        y[2] = y[2] + bias.z;
                        y[3] = y[3] + bias.w;
                    }
                    const int byte = (16 * i + 4 * g) * (int)sizeof(TY), row = 16 * j + r;
                    char *at = mine + row * ROW + ((byte >> 4 ^ (row & (PIECES - 1))) << 4) + (byte & 15);
                    store4(reinterpret_cast<TY *>(at), y);
                }
            }
            // LDS operations of a wave complete in order: only the compiler has to keep them so
            asm volatile("" ::: "memory");
#pragma unroll
            for (int q = 0; q < TOKENS * PIECES / 64; ++q) {
                const int row = (q * 64 + lane) / PIECES, piece = lane % PIECES;
                const char *at = mine + row * ROW + ((piece ^ (row & (PIECES - 1))) << 4);
                const uint4 y = *reinterpret_cast<const uint4 *>(at);
                const int64_t m = mw + 16 * j0 + row, n = nw + piece * (16 / (int)sizeof(TY));
                if (m < a.M && n < a.N)
                    *reinterpret_cast<uint4 *>(static_cast<TY *>(a.Y) + m * a.N + n) = y;
            }
            asm volatile("" ::: "memory");
        }
    }
    if (pieces && !a.acc)
        return;
#pragma unroll
    for (int i = 0; i < TN; ++i) {
        const int64_t n = nw + 16 * i + 4 * g;
        if (n >= a.N)
            continue;
        float ws[4], bias[4];
        load_scales(a, n, ws, bias);
#pragma unroll
        for (int j = 0; j < TM; ++j) {
            const int64_t m = mw + 16 * j + r;
            if (m < a.M)
                store_outputs<TY>(a, m, n, acc[i][j], a.x_scale[m], ws, bias, !pieces);
        }
    }
}

// K == 0: acc is 0.
template <typename TY>
__global__ __launch_bounds__(256) void k_int8_zero(Int8Args a)
{
    for (int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x; id < a.M * a.N; id += (int64_t)gridDim.x * 256) {
        const float y = a.bias ? a.bias[id % a.N] : 0.f;
        if (a.acc)
            a.acc[id] = 0;
        if (a.Y)
            static_cast<TY *>(a.Y)[id] = (TY)y;
    }
}

template <typename TY, int RT, int MT, int RING, int W, bool DIRECT>
hipError_t run_few(const Int8Args &a, hipStream_t s)
{
    const dim3 grid((unsigned)((a.NB + RT - 1) / RT), (unsigned)((a.M + 16 * MT - 1) / (16 * MT)));
    k_int8_few<TY, RT, MT, RING, W, DIRECT><<<grid, 64 * W, 0, s>>>(a);
    return hipGetLastError();
}

template <typename TY, int BM, int BN, int WM, int WN>
hipError_t run_tile(Int8Args a, hipStream_t s)
{
    a.tiles_m = (int)((a.M + BM - 1) / BM);
    a.tiles_n = (int)((a.N + BN - 1) / BN);
    const int64_t run = ((int64_t)a.tiles_m * a.tiles_n + 7) / 8;
    k_int8_tile<TY, BM, BN, WM, WN><<<(unsigned)(8 * run), 64 * WM * WN, 0, s>>>(a);
    return hipGetLastError();
}

// Few workgroups, tokens through LDS: the smallest tile of which no more than one a CU is needed. In us by RT x MT: 128 x
// 2560 x 2560 in 2 x 3 7.4, 4 x 2 8.8, 2 x 2 10.6, 1 x 4 11.4, in k_int8_tile 14.5; 256 x 4096 x 11008 in 4 x 4 35, 4 x 2
// 50, k_int8_tile 59; 300 x 4096 x 11008, for which each would be more than one a CU, 61, 73 and 46. 0: there is none.
int few_tile(int64_t M, int64_t NB)
{
    constexpr int order[] = {12, 13, 14, 22, 23, 24, 42, 43, 44};  // 10 RT + MT
    int best = 0;
    for (int c : order) {
        const int rt = c / 10, mt = c % 10, area = best / 10 * (best % 10);
        const int64_t groups = (NB + rt - 1) / rt * ((M + 16 * mt - 1) / (16 * mt));
        if (groups <= 256 && (best == 0 || rt * mt < area))
            best = c;
    }
    return best;
}

template <typename TY>
hipError_t run_int8(const Int8Args &a, hipStream_t s)
{
    if (a.KC == 0) {
        const int64_t blocks = (a.M * a.N + 255) / 256;
        k_int8_zero<TY><<<(unsigned)(blocks < 4096 ? blocks : 4096), 256, 0, s>>>(a);
        return hipGetLastError();
    }
    // Up to 16 tokens: 16 weight rows a workgroup and loads four blocks ahead where that is no more than one a CU (1 x
    // 4096 x 4096: 5.5 us, two ahead 6.1), else 32 rows, two ahead (in us for 1 and 16 tokens, x 6912 x 2560: 5.6 and 6.3,
    // 16 rows and four ahead 6.4 and 8.0; x 32000 x 2560: 14.7 and 17.4, 16 rows and two ahead 14.9 and 21.9, since
    // the tokens are read twice as often).
    if (a.M <= 16)
        return a.NB <= 256 ? run_few<TY, 1, 1, 4, 8, true>(a, s) : run_few<TY, 2, 1, 2, 8, true>(a, s);
    // Up to 64, where 32 weight rows would be more than one workgroup a CU: 64 rows and tokens straight into registers
    // (40 x 13824 x 2560: 11.6 us, through LDS 12.8; 40 x 8192 x 4096: 14.4, 32 rows through LDS 11.6), by four waves where
    // even those are more than one a CU, so that more fit (40 x 18000 x 4096: 23.9 us, by eight 27.4; 16384 rows: 20.1
    // and 17.6).
    if (a.M <= 64 && a.NB > 512) {
        if (a.NB <= 1024)
            return a.M <= 32   ? run_few<TY, 4, 2, 2, 8, true>(a, s)
                   : a.M <= 48 ? run_few<TY, 4, 3, 2, 8, true>(a, s)
                               : run_few<TY, 4, 4, 2, 8, true>(a, s);
        return a.M <= 32   ? run_few<TY, 4, 2, 2, 4, true>(a, s)
               : a.M <= 48 ? run_few<TY, 4, 3, 2, 4, true>(a, s)
                           : run_few<TY, 4, 4, 2, 4, true>(a, s);
    }
    switch (few_tile(a.M, a.NB)) {
    case 12: return run_few<TY, 1, 2, 4, 8, false>(a, s);
    case 13: return run_few<TY, 1, 3, 4, 8, false>(a, s);
    case 14: return run_few<TY, 1, 4, 4, 8, false>(a, s);
    case 22: return run_few<TY, 2, 2, 4, 8, false>(a, s);
    case 23: return run_few<TY, 2, 3, 4, 8, false>(a, s);
    case 24: return run_few<TY, 2, 4, 4, 8, false>(a, s);
    case 42: return run_few<TY, 4, 2, 4, 8, false>(a, s);
    case 43: return run_few<TY, 4, 3, 4, 8, false>(a, s);
    case 44: return run_few<TY, 4, 4, 4, 8, false>(a, s);
    default: break;
    }
    // one workgroup of large tiles fills a CU, two of small ones do: from 160 large ones on they win (2048 x 5120 x 4096,
    // 160: 46.6 us, small ones 51.2; 1024 x 8192 x 4096, 128: 46.6 and 42.0; 512 x 22016 x 4096, 172: 53.8 and 67.5)
    if (((a.M + 255) / 256) * ((a.N + 255) / 256) >= 160)
        return run_tile<TY, 256, 256, 2, 4>(a, s);
    return run_tile<TY, 128, 128, 2, 2>(a, s);
}

}  // namespace

size_t int8_weight_bytes(int64_t N, int64_t K) { return (size_t)(round_up(N, 16) * round_up(K, 64)); }

hipError_t launch_int8_pack(const int8_t *W, int64_t ld, int64_t N, int64_t K, void *Wp, hipStream_t s)
{
    const int64_t pieces = (int64_t)int8_weight_bytes(N, K) / 16;
    // a launch holds less than 2^32 work-items, and the largest weights have that many pieces: 2^28 at a time
    const int64_t blocks = (pieces + 255) / 256, most = 1 << 20;
    k_int8_pack<<<(unsigned)(blocks < most ? blocks : most), 256, 0, s>>>(W, ld, N, K, pieces, (K + 63) / 64,
                                                                         static_cast<char *>(Wp));
    return hipGetLastError();
}

size_t int8_workspace_bytes(int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_int8(const void *Wp, const float *w_scale, const int8_t *X, const float *x_scale, int64_t M,
                       int64_t N, int64_t K, const float *bias, void *Y, int y_type, int32_t *acc, void *, hipStream_t s)
{
    Int8Args a{};
    a.Wp = static_cast<const char *>(Wp);
    a.w_scale = w_scale;
    a.x_scale = x_scale;
    a.bias = bias;
    a.X = X;
    a.Y = Y;
    a.acc = acc;
    a.M = M;
    a.N = N;
    a.ldx = round_up(K, 256);
    a.KC = (int)((K + 63) / 64);
    a.NB = (int)((N + 15) / 16);
    const uintptr_t four = y_type == kF32 ? 15 : 7;
    a.wide = N % 4 == 0 && !(reinterpret_cast<uintptr_t>(Y) & four) && !(reinterpret_cast<uintptr_t>(acc) & 15);
    a.pieces = N * (y_type == kF32 ? 4 : 2) % 16 == 0 && !(reinterpret_cast<uintptr_t>(Y) & 15);
    return y_type == kF32 ? run_int8<float>(a, s) : y_type == kBF16 ? run_int8<bf16_t>(a, s) : run_int8<f16_t>(a, s);
}

}  // namespace bt
