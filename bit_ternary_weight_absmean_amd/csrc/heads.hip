// Per-head norms of Q and K with the position rotation, in one pass over the fused QKV rows
// that the QKV projection writes (bt_qk_norm_rope).
//
//   head x [D]:  x^ = x * w / sqrt(mean(x^2) + eps)            (w given; else x^ = x)
//   pair (a, b) of angle t = position * inv_freq[p]:  a' = a cos t - b sin t,
//                                                     b' = b cos t + a sin t
//   pairs are (p, p + rot/2), or (2p, 2p + 1) when interleaved, p < rot/2; the elements from
//   rot on stay as normalized. V heads are only converted.
//
// Bound: bytes. Every QKV value is read once and written once; the rest is kept below that (16384 tokens
// of 64 + 2 * 8 heads of 128, fp32 to bf16: 195-208 us, 4.8-5.2 TB/s; a large copy moves 4.9).
//  * Eight values per lane as two 4-value pieces chosen so that both halves of a lane's four
//    pairs are its own (pieces at 4i and rot/2 + 4i, or 8i and 8i + 4): the rotation needs no
//    exchange between lanes, and the sum of squares one reduction over the head's lanes
//    (16 lanes for D = 128, DPP only).
//  * Angles are formed in fp64 and reduced to a fraction of a turn there, so that positions
//    beyond 10^6 keep fp32 accuracy (an fp32 product pos * inv_freq is off by up to
//    pos * 2^-24 radians); sine and cosine of the fraction are fp32. A wave keeps to one token,
//    and its lanes' four angles serve every head that the wave walks.
//  * Few tokens: a token's heads are spread over several waves (`parts`), at most one pass each.
#include "bt_internal.h"
#include "convert.h"
#include "wave.h"

namespace bt {
namespace {

struct HeadsArgs {
    const void *qkv;
    int64_t ld, M;
    int heads, kv_heads, D, rot, interleaved, parts;
    const float *qw, *kw;
    float eps;
    const int *pos;
    const double *inv_freq;
    const int *rows;
    int64_t kv_rows;
    void *q, *k, *v;
    int64_t q_row, q_head, k_row, k_head, v_row, v_head;
};

// Sum over the LG lanes of a head (LG a power of two: 8 .. 64, aligned groups).
template <int LG>
__device__ inline float group_sum(float v)
{
    v += __int_as_float(dpp_i<kDppQuadXor1>(__float_as_int(v)));
    v += __int_as_float(dpp_i<kDppQuadXor2>(__float_as_int(v)));
    v += __int_as_float(dpp_i<kDppRowHalfMirror>(__float_as_int(v)));
    if constexpr (LG > 8)
        v += __int_as_float(dpp_i<kDppRowMirror>(__float_as_int(v)));
    if constexpr (LG > 16) {
        const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(p[0]) + __uint_as_float(p[1]);
    }
    if constexpr (LG > 32) {
        const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(p[0]) + __uint_as_float(p[1]);
    }
    return v;
}

template <typename TI, typename TO, int LG>
__global__ __launch_bounds__(256) void k_qk_norm_rope(HeadsArgs a)
{
    constexpr int GPW = 64 / LG;  // heads a wave holds at a time
    const int lane = threadIdx.x & 63;
    const int64_t unit = (int64_t)blockIdx.x * 4 + uniform(threadIdx.x >> 6);
    const int64_t m = unit / a.parts;
    const int part = (int)(unit % a.parts);
    if (m >= a.M)
        return;
    const int slot = lane % LG, sub = lane / LG;
    const bool live = slot * 8 < a.D;
    const bool turns = slot * 8 < a.rot;
    // first and second 4-value piece of this lane
    int e0 = slot * 8, e1 = slot * 8 + 4;
    if (turns && !a.interleaved) {
        e0 = slot * 4;
        e1 = a.rot / 2 + slot * 4;
    }
    float cs[4] = {1.f, 1.f, 1.f, 1.f}, sn[4] = {0.f, 0.f, 0.f, 0.f};
    if (turns) {
        const double p = (double)a.pos[m];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            double t = p * a.inv_freq[slot * 4 + j] * 0.15915494309189533576888;  // turns
            t -= rint(t);
            sincospif(2.0f * (float)t, &sn[j], &cs[j]);
        }
    }
    const int total = a.heads + 2 * a.kv_heads;
    int64_t row = m;
    bool kept = true;
    if (a.rows) {
        row = a.rows[m];
        kept = row >= 0 && row < a.kv_rows;
    }
    const TI *src = static_cast<const TI *>(a.qkv) + m * a.ld;
    for (int h = part * GPW + sub; h < total; h += a.parts * GPW) {
        const TI *x = src + (int64_t)h * a.D;
        float v0[4] = {}, v1[4] = {};
        if (live) {  // lanes past D stay, with zeros, for the sum below
            load4(x + e0, v0);
            load4(x + e1, v1);
        }
        const bool is_q = h < a.heads, is_v = h >= a.heads + a.kv_heads;
        if (!is_v) {
            const float *w = is_q ? a.qw : a.kw;
            if (w) {
                float ss = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    ss = __builtin_fmaf(v0[j], v0[j], __builtin_fmaf(v1[j], v1[j], ss));
                ss = group_sum<LG>(ss);
                const float rs = 1.0f / sqrtf(ss / (float)a.D + a.eps);
                float w0[4] = {}, w1[4] = {};
                if (live) {
                    load4(w + e0, w0);
                    load4(w + e1, w1);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    v0[j] = v0[j] * rs * w0[j];
                    v1[j] = v1[j] * rs * w1[j];
                }
            }
            if (turns) {
                float r0[4], r1[4];
                if (a.interleaved) {
                    r0[0] = v0[0] * cs[0] - v0[1] * sn[0];
                    r0[1] = v0[1] * cs[0] + v0[0] * sn[0];
                    r0[2] = v0[2] * cs[1] - v0[3] * sn[1];
                    r0[3] = v0[3] * cs[1] + v0[2] * sn[1];
                    r1[0] = v1[0] * cs[2] - v1[1] * sn[2];
                    r1[1] = v1[1] * cs[2] + v1[0] * sn[2];
                    r1[2] = v1[2] * cs[3] - v1[3] * sn[3];
                    r1[3] = v1[3] * cs[3] + v1[2] * sn[3];
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        r0[j] = v0[j] * cs[j] - v1[j] * sn[j];
                        r1[j] = v1[j] * cs[j] + v0[j] * sn[j];
                    }
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    v0[j] = r0[j];
                    v1[j] = r1[j];
                }
            }
        }
        TO *dst;
        if (is_q)
            dst = static_cast<TO *>(a.q) + m * a.q_row + h * a.q_head;
        else if (!kept)
            continue;  // a whole head's lanes at once
        else if (!is_v)
            dst = static_cast<TO *>(a.k) + row * a.k_row + (h - a.heads) * a.k_head;
        else
            dst = static_cast<TO *>(a.v) + row * a.v_row + (h - a.heads - a.kv_heads) * a.v_head;
        if (live) {
            store4(dst + e0, v0);
            store4(dst + e1, v1);
        }
    }
}

template <typename TI, typename TO>
hipError_t launch_types(const HeadsArgs &a, int lg, unsigned grid, hipStream_t s)
{
    switch (lg) {
    case 8: k_qk_norm_rope<TI, TO, 8><<<grid, 256, 0, s>>>(a); break;
    case 16: k_qk_norm_rope<TI, TO, 16><<<grid, 256, 0, s>>>(a); break;
    case 32: k_qk_norm_rope<TI, TO, 32><<<grid, 256, 0, s>>>(a); break;
    default: k_qk_norm_rope<TI, TO, 64><<<grid, 256, 0, s>>>(a); break;
    }
    return hipGetLastError();
}

template <typename TI>
hipError_t launch_out(const HeadsArgs &a, int out_type, int lg, unsigned grid, hipStream_t s)
{
    switch (out_type) {
    case kF32: return launch_types<TI, float>(a, lg, grid, s);
    case kBF16: return launch_types<TI, bf16_t>(a, lg, grid, s);
    default: return launch_types<TI, f16_t>(a, lg, grid, s);
    }
}

}  // namespace

hipError_t launch_qk_norm_rope(const void *qkv, int in_type, int64_t ld, int64_t M, int64_t heads, int64_t kv_heads,
                               int64_t D, const float *qw, const float *kw, float eps, const int32_t *pos,
                               const double *inv_freq, int64_t rot, int interleaved, const int32_t *rows,
                               int64_t kv_rows, void *q, void *k, void *v, int out_type, const int64_t *strides,
                               hipStream_t s)
{
    const int lg = D <= 64 ? 8 : D <= 128 ? 16 : D <= 256 ? 32 : 64;
    HeadsArgs a;
    a.qkv = qkv;
    a.ld = ld;
    a.M = M;
    a.heads = (int)heads;
    a.kv_heads = (int)kv_heads;
    a.D = (int)D;
    a.rot = (int)rot;
    a.interleaved = interleaved;
    a.qw = qw;
    a.kw = kw;
    a.eps = eps;
    a.pos = pos;
    a.inv_freq = inv_freq;
    a.rows = rows;
    a.kv_rows = kv_rows;
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_row = strides[0];
    a.q_head = strides[1];
    a.k_row = strides[2];
    a.k_head = strides[3];
    a.v_row = strides[4];
    a.v_head = strides[5];
    // Waves: one per token once tokens alone fill the CUs, else a token's head passes spread
    // over up to that many waves.
    const int64_t passes = ((heads + 2 * kv_heads) * lg + 63) / 64;
    const int64_t want = (2048 + M - 1) / M;
    a.parts = (int)(passes < want ? passes : want);
    const unsigned grid = (unsigned)((M * a.parts + 3) / 4);
    switch (in_type) {
    case kF32: return launch_out<float>(a, out_type, lg, grid, s);
    case kBF16: return launch_out<bf16_t>(a, out_type, lg, grid, s);
    default: return launch_out<f16_t>(a, out_type, lg, grid, s);
    }
}

}  // namespace bt
