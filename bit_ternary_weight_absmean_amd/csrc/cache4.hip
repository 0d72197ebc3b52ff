// Writing tokens' keys and values to the 4-bit cache and reading them back (bt_cache4_write, bt_cache4_read).
//
// A group of 32 values is quantized with the power of two 2^e for which no value lies above 7 * 2^e (e as small as
// possible): the code nearest to x / 2^e is then off by at most 2^e, which is also the widest half step of the
// codes (between 4 and 6), and values up to 7 * 2^e cost no more as a 6. Both the division and the comparison
// with the codes' middles are exact, so the result is defined bit for bit.
//
// A lane has a whole group; a wave 16 tokens (lane % 16) by four groups. What tokens that lie side by side in a page
// write and read of the cache is then contiguous, 1 KB of codes and 64 bytes of scales, and so are the 256 bytes of
// each token's row. 16384 tokens of eight key heads of 128, bf16 (85 MB): 19.2 us written, 24.3 read (4.4 and 3.5 TB/s; a
// large copy on this card: 5.2); in random places, where each group's 16 bytes and one are lines of their own, 30.8 and
// 31.4. With four lanes to a group and 64-bit index arithmetic 28.6 and 35.7 in random places. Below a few thousand tokens
// the launch is what counts (37 tokens: 3.5 us under the tracer).
#include "bt_internal.h"
#include "cache4.h"
#include "wave.h"

namespace bt {
namespace {

// Eight values from or to arrays that are aligned to four.
template <typename T>
struct Eight {
    typedef T type __attribute__((ext_vector_type(8), aligned(4 * sizeof(T))));
};

// Where a group lies: its 16 bytes of codes, and its scale.
struct Place {
    char *codes, *scale;
};
__device__ inline Place cache_place(const CacheRows &a, int row, int head, int group, bool value)
{
    const int tokens = 1 << a.page_shift, in = row & (tokens - 1);
    const int chunk = (in / kCacheTile * a.groups + group) * kCacheTile + in % kCacheTile;
    const int plane = tokens * a.groups;  // scales of K in one head
    char *base = a.cache + (int64_t)(row >> a.page_shift) * a.page_bytes + (int64_t)head * plane * 34;
    return {base + (value ? 16 * (int64_t)plane : 0) + 16 * (int64_t)chunk,
            base + 32 * (int64_t)plane + (value ? plane : 0) + chunk};
}

// This lane's group of K or V of a token's head.
struct Group {
    int token, head, group;
    bool value, live;
};
__device__ inline Group group_of(const CacheRows &a)
{
    const uint32_t half = (uint32_t)(a.Hkv * a.groups), fours = (2 * half + 3) / 4;
    const uint32_t wave = blockIdx.x * 4u + (threadIdx.x >> 6), block = wave / fours;
    uint32_t u = 4 * (wave - block * fours) + (threadIdx.x >> 4 & 3);
    Group g;
    g.token = (int)(16 * block + (threadIdx.x & 15));
    g.live = g.token < a.M && u < 2 * half;
    g.value = u >= half;
    u -= g.value ? half : 0;
    g.head = (int)(u / (uint32_t)a.groups);
    g.group = (int)(u - (uint32_t)g.head * (uint32_t)a.groups);
    return g;
}

template <typename T>
__global__ __launch_bounds__(256) void k_cache_write(CacheRows a, const T *k, const T *v)
{
    const Group g = group_of(a);
    if (!g.live)
        return;
    const int row = a.rows[g.token], d = g.group * kCacheGroup;
    if (row < 0 || row >= a.places)
        return;
    const T *src = (g.value ? v + g.token * a.v_row + g.head * a.v_head : k + g.token * a.k_row + g.head * a.k_head) + d;
    float x[4][8];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        if (d + 8 * c < a.D) {  // D is a multiple of 8
            const auto y = *reinterpret_cast<const typename Eight<T>::type *>(src + 8 * c);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                x[c][j] = (float)y[j];
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                x[c][j] = 0.f;
        }
    }
    // the group's largest magnitude, as bits: infinities and NaNs lie above every finite value
    uint32_t most = 0;
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j)
            most = max(most, __float_as_uint(x[c][j]) & 0x7FFFFFFFu);
    // e + 127: exponent - 2, one more above 1.75 * 2^exponent (subnormals: exponent field 0 gives the lowest scale)
    int byte = (int)(most >> 23) - 2 + ((most & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    byte = min(max(byte, 0), kCacheNaN);
    uint4 codes = {0, 0, 0, 0};
    if (most < 0x7F800000u) {
        const float scale = __uint_as_float((uint32_t)byte << 23);
        uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            w[c] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w[c], x[c][0], x[c][1], scale, 0);
            w[c] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w[c], x[c][2], x[c][3], scale, 1);
            w[c] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w[c], x[c][4], x[c][5], scale, 2);
            w[c] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w[c], x[c][6], x[c][7], scale, 3);
        }
        codes = uint4{w[0], w[1], w[2], w[3]};
    } else {
        byte = 255;
    }
    const Place p = cache_place(a, row, g.head, g.group, g.value);
    *reinterpret_cast<uint4 *>(p.codes) = codes;
    *p.scale = (char)byte;
}

template <typename T>
__global__ __launch_bounds__(256) void k_cache_read(CacheRows a, T *k, T *v)
{
    const Group g = group_of(a);
    if (!g.live)
        return;
    const int row = a.rows[g.token], d = g.group * kCacheGroup;
    uint4 codes = {0, 0, 0, 0};
    float scale = 0.f;
    if (row >= 0 && row < a.places) {
        const Place p = cache_place(a, row, g.head, g.group, g.value);
        codes = *reinterpret_cast<const uint4 *>(p.codes);
        scale = cache_scale((unsigned char)*p.scale);
    }
    T *dst = (g.value ? v + g.token * a.v_row + g.head * a.v_head : k + g.token * a.k_row + g.head * a.k_head) + d;
    const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        if (d + 8 * c >= a.D)
            break;
        const bf16x8 y = cache_values(w[c], scale);
        typename Eight<T>::type z;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            z[j] = (T)(float)y[j];
        *reinterpret_cast<typename Eight<T>::type *>(dst + 8 * c) = z;
    }
}

unsigned groups_grid(const CacheRows &a)
{
    const int64_t waves = ((int64_t)a.M + 15) / 16 * ((2 * (int64_t)a.Hkv * a.groups + 3) / 4);
    return (unsigned)((waves + 3) / 4);
}

template <typename T>
hipError_t run_write(const CacheRows &a, const void *k, const void *v, hipStream_t s)
{
    k_cache_write<T><<<groups_grid(a), 256, 0, s>>>(a, static_cast<const T *>(k), static_cast<const T *>(v));
    return hipGetLastError();
}

template <typename T>
hipError_t run_read(const CacheRows &a, void *k, void *v, hipStream_t s)
{
    k_cache_read<T><<<groups_grid(a), 256, 0, s>>>(a, static_cast<T *>(k), static_cast<T *>(v));
    return hipGetLastError();
}

}  // namespace

hipError_t launch_cache_write(const CacheRows &a, const void *k, const void *v, int type, hipStream_t s)
{
    return type == kF32    ? run_write<float>(a, k, v, s)
           : type == kBF16 ? run_write<bf16_t>(a, k, v, s)
                           : run_write<f16_t>(a, k, v, s);
}

hipError_t launch_cache_read(const CacheRows &a, void *k, void *v, int type, hipStream_t s)
{
    return type == kF32    ? run_read<float>(a, k, v, s)
           : type == kBF16 ? run_read<bf16_t>(a, k, v, s)
                           : run_read<f16_t>(a, k, v, s);
}

}  // namespace bt
