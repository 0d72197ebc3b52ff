// Attention over packed sequences with grouped heads (bt_attention): whole causal prompts, prompts
// continued behind cached keys, single tokens over a cache, and batches that share a prefix.
//
//   s[r, j] = scale * q_r . k_j over the keys j that row r sees;  out_r = sum_j softmax(s)_j v_j;
//   lse_r = ln sum_j exp(s[r, j])      (no key seen: out 0, lse -inf)
//
// One pass over the keys with a running maximum m and sum l per row (both fp32; scores are kept in
// powers of two, so exp is one v_exp_f32 of an FMA). A row's accumulator is rescaled only when its
// maximum rose by more than a factor 2^kRise: probabilities are relative to the reference m, whatever it
// is. The sum l takes a block's probabilities as one term, so that many small ones behind a large one are
// not lost to it one by one (the matrix cores add eight products at a time to an accumulator).
//
// Rows. The G = heads / kv_heads query heads of a key head read the same keys, so a tile's rows are
// (token, head of the group) pairs: row r of a sequence is token r / G, head r % G of the group. A
// decode step of one token thus already fills G rows of an MFMA with one read of the keys.
//
// Layout. Both products are computed transposed, S^T = K Q^T and O^T = V^T P^T, so that a query row
// is a column of the MFMA result: its running maximum and sum live in the lanes of that column
// (one exchange between lane halves or quarters per step), and the probabilities come out in the
// registers in which the second product takes them, with no exchange at all, as long as both of its
// operands number the keys alike. V^T operands come from row-major V in LDS through the transposing
// LDS read (ds_read_b64_tr_b16: lane i of 16 receives column i of a 4 x 16 block).
//
// Rounding: scores, statistics and accumulators are fp32. Probabilities are rounded to the type of V
// for the matrix cores, which is of the order of the output's own rounding where the output has that
// type; for fp32 outputs, and in the few-rows kernel always (the second product costs it nothing: 64 tokens
// over slabs of 8192 keys 132.4 us with and without, 8 requests behind 1000 keys 18.4 against 18.2), they
// are carried as two such values (the rounded one and the rest). For 16-bit outputs of tiles the rest would
// cost a third (7B prompt of 8192 tokens, fp16: 549 us, with the rest and fp32 outputs 744). fp16
// probabilities, and their rests, are rounded absolutely below 2^-14. All fp16 ones therefore carry a factor
// 2^9 (so does l, and it cancels), and a maximum may rise by 2^6 only: the largest lies between 2^9 and
// 2^15, and the absolute rounding is at most 2^-34 of it, a hundredth of what the fp32 accumulators round
// (2^-24 for eight keys). 2^13 and 2^2 rescale more often: 7B prompt of 8192 tokens 546 us against 541.
//
// Masked places. Scores of unseen keys are replaced, never added to, so what K holds there does not
// matter; keys past a sequence's end are not read at all. An unseen value meets a probability of
// exactly 0, and 0 * inf would still be NaN: in a block whose mask is not full, infinities and NaNs
// of V are set to 0 before the product.
//
// Infinities and NaNs of V that a row sees are its output, whatever their probability (which is positive,
// but may be 0 in fp32, or have a rest of the other sign): a row whose sum came out infinite or NaN
// although its probabilities did not, or whose masked blocks were cleaned, goes over the values once more
// (bad_values), and takes from there what it finds. The joining does the same with its slices.
//
// Work split. A work item is (row tile, slice of its keys, key head). Sequence lengths are device
// data, so every workgroup derives the items from them itself (one wave scan over the sequences).
// With `target` set, keys are cut into slices of equal length such that all items together are
// about `target`: then the slices' outputs, normalized, go to the workspace with their lse, and
// k_attn_combine joins them in slice order. No atomics, so results do not depend on timing.
#include <type_traits>

#include "attention_items.h"

namespace bt {
namespace {

__device__ inline const char *key_base(const AttnArgs &a, const Seq &s, int head, bool value)
{
    const char *p = static_cast<const char *>(value ? a.v : a.k);
    const int64_t row = value ? a.v_row : a.k_row, hd = value ? a.v_head : a.k_head;
    return p + 2 * ((int64_t)s.k0 * row + (int64_t)head * hd);
}

// A buffer over `rows` rows of D values from p, rows row_bytes apart; reads outside give 0.
__device__ inline __amdgpu_buffer_rsrc_t rows_buffer(const char *p, int rows, int row_bytes, int D)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<char *>(p), (short)0,
                                             rows > 0 ? (rows - 1) * row_bytes + 2 * D : 0, kBufferWord3);
}

// Direct load of 16 bytes per lane to LDS at dst + 16 * lane.
__device__ inline void load_lds16(__amdgpu_buffer_rsrc_t from, char *dst, uint32_t offset)
{
#if defined(__HIP_DEVICE_COMPILE__)  // the host pass does not know the 16-byte form
    __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (lds_void *)dst, 16, offset, 0, 0, 0);
#endif
}

// Adds to bad what four values at v hold of infinities and NaNs, over rows from .. to - 1.
template <typename E>
__device__ inline void bad_values(const char *v, int64_t row_bytes, int from, int to, float (&bad)[4])
{
    for (int key = from; key < to; ++key) {
        float x[4];
        load4(reinterpret_cast<const E *>(v + key * row_bytes), x);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            bad[j] += not_finite(x[j]) ? x[j] : 0.f;
    }
}

// The same, eight rows in flight (the last one again where there are no more: an infinity added twice is the
// same infinity) and no more once all four are NaN: for tiles, whose lanes have sixteen fours of a long
// prompt's values each. The few-rows kernel's short calls would pay for its size (8 requests behind 1000 keys
// 18.4 -> 19.0 us).
template <typename E>
__device__ inline void many_bad_values(const char *v, int64_t row_bytes, int from, int to, float (&bad)[4])
{
    constexpr int kFlight = 8;
    for (int key = from; key < to; key += kFlight) {
        float x[kFlight][4];
#pragma unroll
        for (int u = 0; u < kFlight; ++u)
            load4(reinterpret_cast<const E *>(v + min(key + u, to - 1) * row_bytes), x[u]);
#pragma unroll
        for (int u = 0; u < kFlight; ++u)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                bad[j] += not_finite(x[u][j]) ? x[u][j] : 0.f;
        if (bad[0] != bad[0] && bad[1] != bad[1] && bad[2] != bad[2] && bad[3] != bad[3])
            break;
    }
}

// ------------------------------------------------------------------------- prompt kernel
//
// attn_tile: 32 rows per wave (32x32x16 MFMA) against a slice of the tile's keys, 64 at a time. K and
// V blocks go to LDS by direct loads, the next block's while this one is used (two buffers each).
//
// A block is two phases: from the scores to the probabilities on the vector unit, then this block's
// product with V and the next block's scores on the matrix cores. Kept apart (the probabilities are
// pinned at the end of the first phase), the matrix phase is one unbroken run of 32 MFMAs fed from LDS,
// and the two waves of a SIMD, which belong to different workgroups, alternate: a 7B prompt of 8192
// tokens takes 542-549 us (1.0 PFLOP/s; a large bf16 matrix product of the library reaches 1.38 on the
// same card), against 592-620 us with scores, softmax and V's product in sequence. Eight waves of one
// workgroup in two groups held half a block apart by barriers: 597-620 us; a raised wave priority in
// the matrix phase: 549 us.
//
// HALVES == 2, for calls whose tiles of 128 rows would not fill the CUs: 64 rows, and the waves of a pair
// take the two halves of every block's keys and are joined at the end. Twice the workgroups, each with half
// the time per block (packed 2B prompts of 2048 tokens: 28.8 us with 128 rows, 25.0-26.2 with 64).

constexpr int kTileRows = 128, kSmallRows = 64, kTileKeys = 64;

template <typename E, int DP, bool PART, bool WIDE, int HALVES>
__device__ __forceinline__ void attn_tile(const AttnArgs &a, int block, char *kbuf0, char *kbuf1, char *vbuf0,
                                          char *vbuf1, int &poison)
{
    using V8 = typename Elem<E>::v8;
    constexpr int ROWS = kTileRows / HALVES, KB = 2 / HALVES;  // rows of the tile, 32-key parts per wave
    constexpr int CPR = DP / 8;                          // 16-byte chunks of a row
    constexpr int NS = DP / 16, ND = DP / 32;            // MFMA steps over D, 32-wide tiles of D
    constexpr int LOADS = kTileKeys * CPR / 256;         // direct loads per wave and block
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int col = lane & 31, h = lane >> 5;
    const int rg = HALVES == 2 ? wave & 1 : wave;        // the wave's 32 rows
    const int part0 = HALVES == 2 ? wave >> 1 : 0;       // its first 32-key part of a block
    const int id = block / a.Hkv, head = block % a.Hkv;
    Item it;
    if (!find_item(a, ROWS, id, false, it))
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
    const int gfull = row_limit(a, s, it.tile * ROWS / a.G);  // keys that every row of the tile sees
    const int wmost = first < rows ? row_limit(a, s, min(rows - 1, first + 31) / a.G) : 0;

    // Q^T operands: lane (col, h) holds values 16 st + 8 h .. + 7 of its row
    V8 qf[NS];
    {
        const char *p = static_cast<const char *>(a.q) + 2 * ((int64_t)(s.q0 + token) * a.q_row + (int64_t)qh * a.q_head);
#pragma unroll
        for (int st = 0; st < NS; ++st) {
            u32x4 x = {0, 0, 0, 0};
            if (live && 16 * st + 8 * h < a.D)
                x = *reinterpret_cast<const u32x4 *>(p + 2 * (16 * st + 8 * h));
            qf[st] = __builtin_bit_cast(V8, x);
        }
    }

    // direct loads: chunk L of a block (row L / CPR, place L % CPR) receives the row's chunk
    // place ^ swizzle(row)
    const int krow_bytes = (int)(2 * a.k_row), vrow_bytes = (int)(2 * a.v_row);
    uint32_t koff[LOADS], voff[LOADS];
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
        const int L = (wave * LOADS + i) * 64 + lane, r = L / CPR, c = (L % CPR) ^ swizzle<DP>(r);
        const bool in = c * 8 < a.D;
        koff[i] = in ? (uint32_t)(r * krow_bytes + c * 16) : kOutside;
        voff[i] = in ? (uint32_t)(r * vrow_bytes + c * 16) : kOutside;
    }
    const char *kp = key_base(a, s, head, false), *vp = key_base(a, s, head, true);
    auto issue = [&](const char *base, int row_bytes, const uint32_t (&off)[LOADS], int key, char *dst) __attribute__((always_inline)) {
        if (key >= hi)
            return;
        const __amdgpu_buffer_rsrc_t from =
            rows_buffer(base + (int64_t)key * row_bytes, min(kTileKeys, s.nk - key), row_bytes, a.D);
#pragma unroll
        for (int i = 0; i < LOADS; ++i)
            load_lds16(from, dst + (wave * LOADS + i) * 1024, off[i]);
    };

    f32x16 o[ND];
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i)
            o[d][i] = 0.f;
    float m = -INFINITY, l = 0.f;  // l: this lane's keys only until the end
    const float c2 = a.scale_log2;

    // S^T of a block; register i of half b: key + 32 b + 8 (i / 4) + 4 h + i % 4. Operand addresses are a
    // lane's base with bits flipped by the (constant) step.
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
                const u32x4 x = *reinterpret_cast<const u32x4 *>(kb + (kbase ^ (st << 5)) + b * 32 * DP * 2);
                sc[b] = Elem<E>::mma32(__builtin_bit_cast(V8, x), qf[st], sc[b]);
            }
        }
    };
    // The vector phase: probabilities of the block, as P^T operands (slot j of step t is register
    // 8 (t % 2) + j of half t / 2).
    u32x4 pf[2 * KB], pr[2 * KB];
    auto soften = [&](int key) __attribute__((always_inline)) {
        if (key + kTileKeys > wfull) {
#pragma unroll
            for (int b = 0; b < KB; ++b)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (key + 32 * (part0 + b) + 8 * (i / 4) + 4 * h + i % 4 >= limit)
                        sc[b][i] = -INFINITY;
        }
        float mx = sc[0][0];
#pragma unroll
        for (int b = 0; b < KB; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                mx = fmaxf(mx, sc[b][i]);
        mx = fmaxf(mx, other_half(mx));
        if (__any((mx - m) * c2 > Elem<E>::kRise || (m == -INFINITY && mx > -INFINITY))) {
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
        const float ref = m == -INFINITY ? 0.f : __builtin_fmaf(m, c2, -Elem<E>::kRaised);
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
                pf[t][j] = pack2<E>(p[0], p[1]);
                if constexpr (WIDE) {
                    const f32x2 back = unpack2<E>(pf[t][j]);
                    pr[t][j] = pack2<E>(p[0] - back[0], p[1] - back[1]);
                }
            }
        l += lb;
        // done here, not where they are used (the sum unpinned: 4% more for the 7B prompt)
        asm volatile("" : "+v"(l));
#pragma unroll
        for (int t = 0; t < 2 * KB; ++t) {
            asm volatile("" : "+v"(pf[t]));
            if constexpr (WIDE)
                asm volatile("" : "+v"(pr[t]));
        }
    };
    // The matrix phase. V^T operands: lane i of 16 reads 8 bytes of row i / 4 of its 4 x 16 block of V. Row
    // 16 t + 8 j + tr_row is swizzled by that of tr_row, with bit 1 flipped by j.
    const int tr_row = 4 * h + (lane & 15) / 4, tr_col = (lane >> 4 & 1) * 32 + (lane & 3) * 8;  // bytes
    const int vbase = tr_row * (DP * 2) + (((tr_col >> 4) ^ swizzle<DP>(tr_row)) << 4) + (tr_col & 15);
    auto weigh = [&](const char *vb) __attribute__((always_inline)) {
        vb += part0 * 32 * DP * 2;
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int t = 0; t < 2 * KB; ++t) {
                u32x4 x;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const char *p = vb + (vbase ^ (d << 6) ^ (j << 5)) + (16 * t + 8 * j) * DP * 2;
                    const u32x2 half =
                        __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)p));
                    x[2 * j] = half[0];
                    x[2 * j + 1] = half[1];
                }
                o[d] = Elem<E>::mma32(__builtin_bit_cast(V8, x), __builtin_bit_cast(V8, pf[t]), o[d]);
                if constexpr (WIDE)
                    o[d] = Elem<E>::mma32(__builtin_bit_cast(V8, x), __builtin_bit_cast(V8, pr[t]), o[d]);
            }
    };

    // End of a block: this wave's direct loads have arrived and its LDS reads are done; then all waves'.
    auto sync = [] {
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    };
    auto landed = [] { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); };
    // Masked block of V: infinities and NaNs to 0, by the whole workgroup.
    auto clean = [&](int key, char *vb) __attribute__((always_inline)) {
        if (key + kTileKeys <= gfull || key >= hi)
            return;
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            u32x4 *p = reinterpret_cast<u32x4 *>(vb + (i * 256 + threadIdx.x) * 16);
            const u32x4 x = *p;
            if (pair_not_finite<E>(x[0]) || pair_not_finite<E>(x[1]) || pair_not_finite<E>(x[2]) || pair_not_finite<E>(x[3])) {
                *p = u32x4{finite_part<E>(x[0]), finite_part<E>(x[1]), finite_part<E>(x[2]), finite_part<E>(x[3])};
                poison = 1;
            }
        }
        sync();
    };
    if (threadIdx.x == 0)
        poison = 0;
    if (lo < hi) {
        issue(kp, krow_bytes, koff, lo, kbuf0);
        landed();
        sync();
        issue(kp, krow_bytes, koff, lo + kTileKeys, kbuf1);
        issue(vp, vrow_bytes, voff, lo, vbuf0);
        scores(kbuf0);
        landed();
        sync();
        // K runs one block ahead of V; the last block's matrix phase forms scores from whatever the
        // other buffer holds, and they are not used.
        auto one = [&](int key, char *vb, char *kb, char *vnext, char *knext) __attribute__((always_inline)) {
            issue(kp, krow_bytes, koff, key + 2 * kTileKeys, knext);
            issue(vp, vrow_bytes, voff, key + kTileKeys, vnext);
            clean(key, vb);
            if (key < wmost) {
                soften(key);
                scores(kb);
                weigh(vb);
            }
            landed();
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
    bool odd = false;
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i)
            odd = odd || not_finite(o[d][i]);
    if (__builtin_expect((odd || poison) && live && l > 0.f && l < INFINITY, 0)) {
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const int e = 32 * d + 8 * b + 4 * h;
                float bad[4] = {0.f, 0.f, 0.f, 0.f};
                // finite sums lack the cleaned blocks only (four that overflow together cost a look)
                const bool all = not_finite((o[d][4 * b] + o[d][4 * b + 1]) + (o[d][4 * b + 2] + o[d][4 * b + 3]));
                const int from = all ? lo : lo + max(0, gfull - lo) / kTileKeys * kTileKeys;
                if (e < a.D && (all || poison))
                    many_bad_values<E>(vp + 2 * e, vrow_bytes, from, min(hi, limit), bad);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    o[d][4 * b + i] = bad[i] == 0.f ? o[d][4 * b + i] : bad[i];
            }
    }

    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);  // l NaN: NaN
    const float lse = l == 0.f ? -INFINITY : m * c2 * kLn2 + logf(l * Elem<E>::kLower);
    if (!live)
        return;
    const bool part = PART && (a.pieced || it.pieces > 1);
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
// attn_few: 16 rows (a decode step's heads of one group, a short draft) against a slice of their
// keys; bound by the bytes of K and V. Each of four waves takes every fourth block of 32 keys on its
// own: K goes from memory straight into the registers of the S^T operand (16x16x32 MFMA: lane (r, g)
// holds 16 bytes of key r), V through a private piece of LDS for the transposing read, and the next
// block's loads are issued before this block is used, so that no barrier and no other wave is waited
// for until the four partial results are joined at the end. 64 tokens over slabs of up to 8192 keys (2B
// heads, 678 MB): 132.5 us with the joining, 5.1 TB/s.

constexpr int kFewRows = 16, kFewKeys = 32, kFewWaves = 4;

template <typename E, int DP, bool WIDE>
__device__ __forceinline__ void attn_few(const AttnArgs &a, int block, char *buf0, char *buf1,
                                         float (&stat)[kFewWaves][4][kFewRows])
{
    using V8 = typename Elem<E>::v8;
    constexpr int CPR = DP / 8;
    constexpr int NS = DP / 32, ND = DP / 16;
    constexpr int LOADS = kFewKeys * CPR / 64;  // 16-byte V loads per lane and block
    constexpr int kVBytes = kFewKeys * DP * 2;
    static_assert(kVBytes >= kFewRows * DP * 4, "the waves' partial outputs reuse the V blocks");
    auto vlds = [&](int w) { return (w < 2 ? buf0 : buf1) + (w & 1) * kVBytes; };  // wave w's piece

    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int col = lane & 15, g = lane >> 4;
    const int id = block / a.Hkv, head = block % a.Hkv;
    Item it;
    if (!find_item(a, kFewRows, id, false, it))
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

    V8 qf[NS];
    {
        const char *p = static_cast<const char *>(a.q) + 2 * ((int64_t)(s.q0 + token) * a.q_row + (int64_t)qh * a.q_head);
#pragma unroll
        for (int st = 0; st < NS; ++st) {
            u32x4 x = {0, 0, 0, 0};
            if (live && 32 * st + 8 * g < a.D)
                x = *reinterpret_cast<const u32x4 *>(p + 2 * (32 * st + 8 * g));
            qf[st] = __builtin_bit_cast(V8, x);
        }
    }
    const int krow_bytes = (int)(2 * a.k_row), vrow_bytes = (int)(2 * a.v_row);
    const char *kp = key_base(a, s, head, false), *vp = key_base(a, s, head, true);
    uint32_t koff[NS], voff[LOADS];
#pragma unroll
    for (int st = 0; st < NS; ++st)
        koff[st] = 32 * st + 8 * g < a.D ? (uint32_t)(col * krow_bytes + 64 * st + 16 * g) : kOutside;
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
        const int L = i * 64 + lane, r = L / CPR, c = L % CPR;
        voff[i] = c * 8 < a.D ? (uint32_t)(r * vrow_bytes + c * 16) : kOutside;
    }
    struct Block {
        u32x4 k[2][NS], v[LOADS];
    };
    auto fetch = [&](int key, Block &x) {
        const int n = s.nk - key;  // <= 0: nothing is read
        const __amdgpu_buffer_rsrc_t kr = rows_buffer(kp + (int64_t)key * krow_bytes, min(kFewKeys, n), krow_bytes, a.D);
        const __amdgpu_buffer_rsrc_t vr = rows_buffer(vp + (int64_t)key * vrow_bytes, min(kFewKeys, n), vrow_bytes, a.D);
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int st = 0; st < NS; ++st)
                x.k[b][st] = __builtin_amdgcn_raw_buffer_load_b128(
                    kr, koff[st] == kOutside ? kOutside : koff[st] + b * 16 * krow_bytes, 0, 0);
#pragma unroll
        for (int i = 0; i < LOADS; ++i)
            x.v[i] = __builtin_amdgcn_raw_buffer_load_b128(vr, voff[i], 0, 0);
    };

    f32x4 o[ND];
#pragma unroll
    for (int d = 0; d < ND; ++d)
        o[d] = f32x4{0.f, 0.f, 0.f, 0.f};
    float m = -INFINITY, l = 0.f;
    const float c2 = a.scale_log2;
    char *vb = vlds(wave);
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
        return x;
    };
    bool poison = false;  // a masked block of V held an infinity or NaN
    auto step = [&](int key, Block &x) __attribute__((always_inline)) {
        f32x4 sc[2];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            sc[b] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int st = 0; st < NS; ++st)
                sc[b] = Elem<E>::mma16(__builtin_bit_cast(V8, x.k[b][st]), qf[st], sc[b]);
        }
        // register i of block b: key + 16 b + 4 g + i
        const bool masked = key + kFewKeys > wfull;
        if (masked) {
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (key + 16 * b + 4 * g + i >= limit)
                        sc[b][i] = -INFINITY;
#pragma unroll
            for (int i = 0; i < LOADS; ++i)
                if (pair_not_finite<E>(x.v[i][0]) || pair_not_finite<E>(x.v[i][1]) || pair_not_finite<E>(x.v[i][2]) ||
                    pair_not_finite<E>(x.v[i][3])) {
                    poison = true;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        x.v[i][j] = finite_part<E>(x.v[i][j]);
                }
        }
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const int L = i * 64 + lane, r = L / CPR, c = (L % CPR) ^ swizzle<DP>(r);
            *reinterpret_cast<u32x4 *>(vb + r * (DP * 2) + c * 16) = x.v[i];
        }
        float mx = fmaxf(fmaxf(fmaxf(sc[0][0], sc[0][1]), fmaxf(sc[0][2], sc[0][3])),
                         fmaxf(fmaxf(sc[1][0], sc[1][1]), fmaxf(sc[1][2], sc[1][3])));
        mx = across_quarters(mx, [](float x, float y) { return fmaxf(x, y); });
        if (__any((mx - m) * c2 > Elem<E>::kRise || (m == -INFINITY && mx > -INFINITY))) {
            const float mn = fmaxf(m, mx);
            const float f = mn == -INFINITY ? 1.f : exp2_fast((m - mn) * c2);
            l *= f;
#pragma unroll
            for (int d = 0; d < ND; ++d)
                o[d] *= f;
            m = mn;
        }
        const float ref = m == -INFINITY ? 0.f : __builtin_fmaf(m, c2, -Elem<E>::kRaised);
        u32x4 pf, pr;
        float lb = 0.f;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                sc[b][i] = exp2_fast(__builtin_fmaf(sc[b][i], c2, -ref));
                lb += sc[b][i];
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                pf[2 * b + j] = pack2<E>(sc[b][2 * j], sc[b][2 * j + 1]);
                const f32x2 back = unpack2<E>(pf[2 * b + j]);
                pr[2 * b + j] = pack2<E>(sc[b][2 * j] - back[0], sc[b][2 * j + 1] - back[1]);
            }
        }
        l += lb;
        // This wave's LDS writes before its reads: LDS operations of a wave complete in order, so
        // only the compiler has to keep them so.
        asm volatile("" ::: "memory");
#pragma unroll
        for (int d = 0; d < ND; ++d) {
            const V8 v = __builtin_bit_cast(V8, v_frag(d));
            o[d] = Elem<E>::mma16(v, __builtin_bit_cast(V8, pf), o[d]);
            o[d] = Elem<E>::mma16(v, __builtin_bit_cast(V8, pr), o[d]);
        }
        asm volatile("" ::: "memory");
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
    const bool cleaned = __any(poison);
    if (g == 0) {
        stat[wave][0][col] = m;
        stat[wave][1][col] = l;
        stat[wave][2][col] = cleaned ? 1.f : 0.f;
    }
    __syncthreads();
    float mall = stat[0][0][col];
#pragma unroll
    for (int w = 1; w < kFewWaves; ++w)
        mall = fmaxf(mall, stat[w][0][col]);
    float lall = 0.f, cleans = 0.f;  // blocks cleaned by any wave
#pragma unroll
    for (int w = 0; w < kFewWaves; ++w) {
        cleans += stat[w][2][col];
        const float mw = stat[w][0][col];
        lall += mw == -INFINITY ? stat[w][1][col] : stat[w][1][col] * exp2_fast((mw - mall) * c2);  // 0, or NaN scores
    }
    if (threadIdx.x < kFewRows)
        stat[0][3][col] = lall;
    const float inv = lall > 0.f ? 1.f / lall : (lall == 0.f ? 0.f : lall);
    const float f = m == -INFINITY ? inv : exp2_fast((m - mall) * c2) * inv;
    const float lse = lall == 0.f ? -INFINITY : mall * c2 * kLn2 + logf(lall * Elem<E>::kLower);
    // wave's O^T to LDS as [row][D]: 4 values of row col per register group
    float *mine = reinterpret_cast<float *>(vlds(wave));
#pragma unroll
    for (int d = 0; d < ND; ++d) {
        const f32x4 x = l == 0.f ? f32x4{0.f, 0.f, 0.f, 0.f} : o[d] * f;
        *reinterpret_cast<f32x4 *>(mine + col * DP + ((4 * d + g) ^ (col & 7)) * 4) = x;
    }
    __syncthreads();
    const bool part = a.pieced || it.pieces > 1;
    for (int e = threadIdx.x; e < kFewRows * (DP / 4); e += 256) {
        const int r = e / (DP / 4), c = e % (DP / 4);
        const int rr = it.tile * kFewRows + r;
        if (rr >= rows || c * 4 >= a.D)
            continue;
        f32x4 sum = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < kFewWaves; ++w)
            sum += *reinterpret_cast<const f32x4 *>(reinterpret_cast<const float *>(vlds(w)) + r * DP + (c ^ (r & 7)) * 4);
        // (a sum of four that overflows costs a look that finds nothing)
        const bool odd = not_finite((sum[0] + sum[1]) + (sum[2] + sum[3]));
        if (__builtin_expect((odd || cleans > 0.f) && stat[0][3][r] > 0.f && stat[0][3][r] < INFINITY, 0)) {
            // finite sums lack the cleaned blocks only
            const int from = odd ? lo : lo + max(0, wfull - lo) / kFewKeys * kFewKeys;
            float bad[4] = {0.f, 0.f, 0.f, 0.f};
            bad_values<E>(vp + 8 * c, vrow_bytes, from, min(hi, row_limit(a, s, rr / a.G)), bad);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                sum[j] = bad[j] == 0.f ? sum[j] : bad[j];
        }
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

// ------------------------------------------------------------------------------- kernels
//
// One launch per call, and k_attn_combine behind it where keys are cut. With a shared prefix the
// prefix's items are the first workgroups of the same launch (PRE), so that neither part waits for the
// other.

enum Kind { kNone, kFew, kTile, kSmall };

template <typename E, int DP, bool WIDE, Kind MAIN, Kind PRE, bool PART>
__global__ __launch_bounds__(256, DP > 128 ? 1 : 2) void k_attn(AttnArgs a, AttnArgs pre, int pre_blocks)
{
    constexpr bool tiles = MAIN >= kTile || PRE >= kTile;
    constexpr int bytes = kTileKeys * DP * 2;
    static_assert(bytes == 2 * kFewKeys * DP * 2, "two waves' pieces of the few-rows kernel");
    __shared__ __attribute__((aligned(1024))) char buf0[bytes], buf1[bytes];
    __shared__ __attribute__((aligned(1024))) char buf2[tiles ? bytes : 16], buf3[tiles ? bytes : 16];
    __shared__ float stat[kFewWaves][4][kFewRows];
    __shared__ int poison;  // attn_tile: a masked block of V held an infinity or NaN
    const int block = blockIdx.x;
    if constexpr (PRE == MAIN) {
        const bool p = block < pre_blocks;
        const AttnArgs &x = p ? pre : a;
        if constexpr (MAIN == kFew)
            attn_few<E, DP, WIDE>(x, p ? block : block - pre_blocks, buf0, buf1, stat);
        else
            attn_tile<E, DP, true, WIDE, 1>(x, p ? block : block - pre_blocks, buf0, buf1, buf2, buf3, poison);
    } else {
        if constexpr (PRE == kTile)
            if (block < pre_blocks) {
                attn_tile<E, DP, true, WIDE, 1>(pre, block, buf0, buf1, buf2, buf3, poison);
                return;
            }
        if constexpr (MAIN == kFew)
            attn_few<E, DP, WIDE>(a, block - pre_blocks, buf0, buf1, stat);
        else
            attn_tile<E, DP, PART, WIDE, (MAIN == kSmall ? 2 : 1)>(a, block, buf0, buf1, buf2, buf3, poison);
    }
}

// ------------------------------------------------------------------------------- joining
//
// k_attn_combine: a row's slices, and with a shared prefix the prefix's slices of the same row,
// joined by their lse: out = sum_i w_i out_i / sum_i w_i with w_i = exp(lse_i - max). 32 lanes read a
// row; the groups of a workgroup are spread over its rows, so that the slices of few rows are read
// side by side (four in flight in each group) and joined through LDS. Latency is all there is to it:
// 16 groups cost 0.6-0.9 us more in small calls, 32 groups 1-3 us, fewer workgroups fitting a CU.

constexpr int kJoinGroups = 8;  // and the largest number of rows of a workgroup

template <typename TO>
__global__ __launch_bounds__(32 * kJoinGroups) void k_attn_combine(AttnArgs a, AttnArgs pre, int bm, int pre_bm)
{
    __shared__ f32x4 sums[kJoinGroups][2][32];
    __shared__ float stat[kJoinGroups][2];
    const int l32 = threadIdx.x & 31, group = threadIdx.x >> 5;
    const int id = blockIdx.x / a.Hkv, head = blockIdx.x % a.Hkv;
    Item it;
    if (!find_item(a, bm, id, true, it))
        return;
    const bool shared = pre.shared;
    if (!shared && it.pieces == 1)
        return;  // written by its one item
    const int rows = it.s.nq * a.G;
    const int slot = first_item(a, it, bm);
    if (slot + it.pieces > a.items)
        return;  // more tiles than sequences that do not overlap can have: not computed
    const int r0 = blockIdx.y * kJoinGroups;
    const int here = min(min(bm - r0, kJoinGroups), rows - it.tile * bm - r0);  // rows of this workgroup
    if (here <= 0)
        return;
    const int ways = 32 - __builtin_clz(2 * here - 1) - 1;  // log2 of here rounded up to a power of two
    const int gp = kJoinGroups >> ways;                              // groups of a row
    const int r = r0 + (group & ((1 << ways) - 1)), part = group >> ways;
    const int row = it.tile * bm + r;
    const bool live = r < r0 + here;
    // the prefix's items of this row
    int pslot = 0, pn = 0, prow = 0;
    if (shared) {
        Item p;
        find_item(pre, pre_bm, 0, true, p);
        const int all = min(it.s.q0 * pre.G + row, pre.T * pre.G - 1);  // T * heads <= 2^30
        p.tile = all / pre_bm;
        prow = all % pre_bm;
        pslot = first_item(pre, p, pre_bm);
        pn = p.pieces;
    }
    const int n = it.pieces + pn;
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
                const bool own = j < it.pieces;
                const int64_t at = own ? ((int64_t)(slot + j) * a.Hkv + head) * bm + r
                                       : ((int64_t)(pslot + j - it.pieces) * a.Hkv + head) * pre_bm + prow;
                const float *o = (own ? a.ws_o : pre.ws_o) + at * a.D;
                v[u] = (own ? a.ws_l : pre.ws_l)[at];
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
    const f32x4 both = s0 + s1;
    const bool odd = not_finite((both[0] + both[1]) + (both[2] + both[3]));
    if (__builtin_expect(odd && total > 0.f && total < INFINITY, 0)) {
        // a weight of 0 is too small for fp32, not none: what is infinite or NaN in a slice stays
        f32x4 b0 = {0.f, 0.f, 0.f, 0.f}, b1 = b0;
        for (int j = 0; j < n; ++j) {
            const bool own = j < it.pieces;
            const int64_t at = own ? ((int64_t)(slot + j) * a.Hkv + head) * bm + r
                                   : ((int64_t)(pslot + j - it.pieces) * a.Hkv + head) * pre_bm + prow;
            const float *o = (own ? a.ws_o : pre.ws_o) + at * a.D;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                b0[i] += not_finite(o[c0 + i]) ? o[c0 + i] : 0.f;
                b1[i] += a.D > 128 && not_finite(o[c1 + i]) ? o[c1 + i] : 0.f;
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            s0[i] = b0[i] == 0.f ? s0[i] : b0[i];
            s1[i] = b1[i] == 0.f ? s1[i] : b1[i];
        }
    }
    const int token = row / a.G, qh = head * a.G + row % a.G;
    const int64_t at = (int64_t)(it.s.q0 + token) * a.o_row + (int64_t)qh * a.o_head;
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
        a.lse[(int64_t)(it.s.q0 + token) * a.Hq + qh] = total == 0.f ? -INFINITY : m + logf(total);
}

// --------------------------------------------------------------------------------- plans

template <typename E, int DP, bool WIDE>
hipError_t run_kind(const AttnArgs &a, const AttnArgs &pre, const AttnPlan &p, hipStream_t s)
{
    const int pb = (int)(p.pre.items * a.Hkv);
    const unsigned grid = (unsigned)(p.main.items * a.Hkv + pb);
    const bool few = p.main.bm == kFewRows, pre_few = p.pre.bm == kFewRows;
    if (!pb) {
        if (few)
            k_attn<E, DP, WIDE, kFew, kNone, true><<<grid, 256, 0, s>>>(a, pre, 0);
        else if (p.main.bm == kSmallRows && p.main.target)
            k_attn<E, DP, WIDE, kSmall, kNone, true><<<grid, 256, 0, s>>>(a, pre, 0);
        else if (p.main.bm == kSmallRows)
            k_attn<E, DP, WIDE, kSmall, kNone, false><<<grid, 256, 0, s>>>(a, pre, 0);
        else  // tiles enough to go uncut
            k_attn<E, DP, WIDE, kTile, kNone, false><<<grid, 256, 0, s>>>(a, pre, 0);
    } else if (few && pre_few) {
        k_attn<E, DP, WIDE, kFew, kFew, true><<<grid, 256, 0, s>>>(a, pre, pb);
    } else if (few) {
        k_attn<E, DP, WIDE, kFew, kTile, true><<<grid, 256, 0, s>>>(a, pre, pb);
    } else {  // the prefix has all sequences' rows: no fewer than one of them
        k_attn<E, DP, WIDE, kTile, kTile, true><<<grid, 256, 0, s>>>(a, pre, pb);
    }
    return hipGetLastError();
}

template <typename E, bool WIDE>
hipError_t run_dim(const AttnArgs &a, const AttnArgs &pre, const AttnPlan &p, hipStream_t s)
{
    if (a.D <= 64)
        return run_kind<E, 64, WIDE>(a, pre, p, s);
    if (a.D <= 128)
        return run_kind<E, 128, WIDE>(a, pre, p, s);
    return run_kind<E, 256, WIDE>(a, pre, p, s);
}

hipError_t run_type(const AttnArgs &a, const AttnArgs &pre, const AttnPlan &p, int type, int out_type, hipStream_t s)
{
    const bool wide = out_type == kF32;
    if (type == kBF16)
        return wide ? run_dim<bf16_t, true>(a, pre, p, s) : run_dim<bf16_t, false>(a, pre, p, s);
    return wide ? run_dim<f16_t, true>(a, pre, p, s) : run_dim<f16_t, false>(a, pre, p, s);
}

template <typename TO>
hipError_t run_combine(const AttnArgs &a, const AttnArgs &pre, const AttnPlan &p, hipStream_t s)
{
    const dim3 grid((unsigned)(p.main.tiles * a.Hkv), (unsigned)((p.main.bm + kJoinGroups - 1) / kJoinGroups));
    k_attn_combine<TO><<<grid, 32 * kJoinGroups, 0, s>>>(a, pre, p.main.bm, p.pre.bm);
    return hipGetLastError();
}

// `rows` rows of `seqs` sequences (those that have rows) over at most `keys` keys each.
AttnPart plan_part(int64_t rows, int64_t seqs, int64_t keys, int64_t Hkv, bool always)
{
    AttnPart p;
    // mean rows of a sequence: up to 16, one small tile each
    p.bm = rows <= kFewRows * seqs ? kFewRows : kTileRows;
    if (p.bm == kTileRows && !always && (rows / kTileRows + seqs) * Hkv < 512)
        p.bm = kSmallRows;
    p.tiles = seqs == 1 ? (rows + p.bm - 1) / p.bm : rows / p.bm + seqs;  // at least sum of ceil(rows_b / bm)
    // Keys are cut so that about `want` workgroups share the work: eight per CU where the bytes of the
    // keys are all that counts, and fewer for large tiles, whose outputs cost more to join. 256 / 384 / 512 of
    // those: 64 requests behind 16384 keys 71 / 67 / 74 us, 256 tokens over 8192 keys (2B) 52 / 46 / 55,
    // eight drafts of 8 tokens over 4000 keys 25.6 / 25.2 / 31.8.
    const bool few = p.bm == kFewRows;
    const int64_t want = few ? 2048 : 384;
    const int64_t target = (want + Hkv - 1) / Hkv;
    p.target = few || always || 3 * p.tiles < target ? target : 0;
    p.min_units = 4;
    // Items are sum of tiles * ceil(units / slice) <= work / slice + tiles, work / slice <= target up to
    // the rounding of the fp32 sum; and no tile has more slices than keys allow.
    const int64_t most = ((keys + kUnit - 1) / kUnit + p.min_units - 1) / p.min_units;
    // Few keys in all go uncut, in one launch. One token, 2B heads, cut / uncut: 400 keys of 512 10.7 / 9.0
    // us, 777 of 1024 10.6 / 12.2; four drafts of four tokens over up to 256 keys each 9.9 / 7.9.
    if (!always && keys <= (seqs > 1 ? 1024 : 512))
        p.target = 0;
    p.items = p.tiles + (p.target ? p.target + 8 : 0);
    if (p.target && p.tiles * (most > 1 ? most : 1) < p.items)
        p.items = p.tiles * (most > 1 ? most : 1);
    return p;
}

}  // namespace

AttnPlan attn_plan(int64_t T, int64_t S, int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t P)
{
    AttnPlan p{};
    const int64_t rows = T * (Hq / Hkv);
    p.main = plan_part(rows, B < T ? B : T, S, Hkv, P > 0);
    p.main.o_off = 0;
    auto slots = [&](const AttnPart &x) { return x.target ? x.items * Hkv * x.bm : (int64_t)0; };
    int64_t at = round_up(slots(p.main) * D * 4, 256);
    p.main.l_off = at;
    at += round_up(slots(p.main) * 4, 256);
    if (P > 0) {
        p.pre = plan_part(rows, 1, P, Hkv, true);
        p.pre.o_off = at;
        at += round_up(slots(p.pre) * D * 4, 256);
        p.pre.l_off = at;
        at += round_up(slots(p.pre) * 4, 256);
    }
    p.bytes = (size_t)at;
    return p;
}

hipError_t launch_attention(const AttnArgs &args, const AttnArgs &prefix, const AttnPlan &p, int type, int out_type,
                            hipStream_t s)
{
    AttnArgs a = args, pre = prefix;
    char *ws = reinterpret_cast<char *>(args.ws_o);
    a.target = (int)p.main.target;
    a.items = (int)p.main.items;
    a.min_units = p.main.min_units;
    a.ws_o = reinterpret_cast<float *>(ws + p.main.o_off);
    a.ws_l = reinterpret_cast<float *>(ws + p.main.l_off);
    a.pieced = prefix.shared;
    if (prefix.shared) {
        pre.target = (int)p.pre.target;
        pre.items = (int)p.pre.items;
        pre.min_units = p.pre.min_units;
        pre.ws_o = reinterpret_cast<float *>(ws + p.pre.o_off);
        pre.ws_l = reinterpret_cast<float *>(ws + p.pre.l_off);
        pre.pieced = 1;
    }
    if (hipError_t e = run_type(a, pre, p, type, out_type, s))
        return e;
    if (!p.main.target)
        return hipSuccess;
    return out_type == kF32 ? run_combine<float>(a, pre, p, s)
           : type == kBF16  ? run_combine<bf16_t>(a, pre, p, s)
                            : run_combine<f16_t>(a, pre, p, s);
}

}  // namespace bt
