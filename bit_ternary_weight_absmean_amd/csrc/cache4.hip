// Writing tokens' keys and values to the 4-bit cache and reading them back (bt_cache4_write, bt_cache4_read).
//
// A group of 32 values is quantized with the power of two 2^e for which no value lies above 7 * 2^e (e as small as
// possible): the code nearest to x / 2^e is then off by at most 2^e, which is also the widest half step of the
// codes (between 4 and 6), and values up to 7 * 2^e cost no more as a 6. Both the division and the comparison
// with the codes' middles are exact, so the result is defined bit for bit.
//
// Four lanes hold a group, eight values each. Bound by memory and, below a few thousand tokens, by the launch.
#include "bt_internal.h"
#include "cache4.h"
#include "wave.h"

namespace bt {
namespace {

template <typename T>
__device__ inline void load8(const T *p, float (&v)[8])
{
    float a[4], b[4];
    load4(p, a);
    load4(p + 4, b);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        v[j] = a[j];
        v[4 + j] = b[j];
    }
}

// Where the four lanes of a group find it: piece p of the group's 16 bytes of codes, and its scale.
struct Place {
    char *codes, *scale;
};
__device__ inline Place cache_place(const CacheRows &a, int64_t row, int head, int group, bool value)
{
    const int64_t page = row >> a.page_shift;
    const int in = (int)row & ((1 << a.page_shift) - 1), tokens = 1 << a.page_shift;
    const int chunk = (in / kCacheTile * a.groups + group) * kCacheTile + in % kCacheTile;
    const int plane = tokens * a.groups;  // scales of K in one head
    char *base = a.cache + page * a.page_bytes + (int64_t)head * plane * 34;
    return {base + (value ? 16 * (int64_t)plane : 0) + 16 * (int64_t)chunk,
            base + 32 * (int64_t)plane + (value ? plane : 0) + chunk};
}

// Work item: (token, head, K or V, group, quarter of the group).
template <typename T>
__global__ __launch_bounds__(256) void k_cache_write(CacheRows a, const T *k, const T *v, int64_t items)
{
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (id >= items)  // whole groups: items is a multiple of 4
        return;
    const int part = (int)(id & 3);
    const int64_t u = id >> 2;
    const int per = 2 * a.Hkv * a.groups;
    const int token = (int)(u / per), rest = (int)(u % per);
    const int group = rest % a.groups, head = rest / a.groups % a.Hkv;
    const bool value = rest >= a.Hkv * a.groups;
    const int row = a.rows[token];
    if (row < 0 || row >= a.places)
        return;
    const int d = group * kCacheGroup + 8 * part;
    float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (d < a.D)  // D is a multiple of 8
        load8((value ? v + token * a.v_row + head * a.v_head : k + token * a.k_row + head * a.k_head) + d, x);
    // the group's largest magnitude, as bits: infinities and NaNs lie above every finite value
    uint32_t most = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        most = max(most, __float_as_uint(x[j]) & 0x7FFFFFFFu);
    most = max(most, (uint32_t)dpp_i<kDppQuadXor1>((int)most));
    most = max(most, (uint32_t)dpp_i<kDppQuadXor2>((int)most));
    // e + 127: exponent - 2, one more above 1.75 * 2^exponent (subnormals: exponent field 0 gives the lowest scale)
    int byte = (int)(most >> 23) - 2 + ((most & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    byte = min(max(byte, 0), kCacheNaN);
    uint32_t codes = 0;
    if (most < 0x7F800000u) {
        const float scale = __uint_as_float((uint32_t)byte << 23);
        codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, x[0], x[1], scale, 0);
        codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, x[2], x[3], scale, 1);
        codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, x[4], x[5], scale, 2);
        codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, x[6], x[7], scale, 3);
    } else {
        byte = 255;
    }
    const Place p = cache_place(a, row, head, group, value);
    *reinterpret_cast<uint32_t *>(p.codes + 4 * part) = codes;
    if (part == 0)
        *p.scale = (char)byte;
}

template <typename T>
__global__ __launch_bounds__(256) void k_cache_read(CacheRows a, T *k, T *v, int64_t items)
{
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (id >= items)
        return;
    const int part = (int)(id & 3);
    const int64_t u = id >> 2;
    const int per = 2 * a.Hkv * a.groups;
    const int token = (int)(u / per), rest = (int)(u % per);
    const int group = rest % a.groups, head = rest / a.groups % a.Hkv;
    const bool value = rest >= a.Hkv * a.groups;
    const int d = group * kCacheGroup + 8 * part;
    if (d >= a.D)
        return;
    const int row = a.rows[token];
    float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (row >= 0 && row < a.places) {
        const Place p = cache_place(a, row, head, group, value);
        const bf16x8 y = cache_values(*reinterpret_cast<const uint32_t *>(p.codes + 4 * part),
                                      cache_scale((unsigned char)*p.scale));
#pragma unroll
        for (int j = 0; j < 8; ++j)
            x[j] = (float)y[j];
    }
    T *dst = (value ? v + token * a.v_row + head * a.v_head : k + token * a.k_row + head * a.k_head) + d;
    const float lo[4] = {x[0], x[1], x[2], x[3]}, hi[4] = {x[4], x[5], x[6], x[7]};
    store4(dst, lo);
    store4(dst + 4, hi);
}

template <typename T>
hipError_t run_write(const CacheRows &a, const void *k, const void *v, hipStream_t s)
{
    const int64_t items = (int64_t)a.M * 2 * a.Hkv * a.groups * 4;
    k_cache_write<T><<<(unsigned)((items + 255) / 256), 256, 0, s>>>(a, static_cast<const T *>(k),
                                                                     static_cast<const T *>(v), items);
    return hipGetLastError();
}

template <typename T>
hipError_t run_read(const CacheRows &a, void *k, void *v, hipStream_t s)
{
    const int64_t items = (int64_t)a.M * 2 * a.Hkv * a.groups * 4;
    k_cache_read<T><<<(unsigned)((items + 255) / 256), 256, 0, s>>>(a, static_cast<T *>(k), static_cast<T *>(v), items);
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
