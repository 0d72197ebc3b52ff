// The 4-bit cache: places of a page and the conversion of codes, shared by the kernels that write, read back
// and attend to it.
//
// 32 values of one token and key head (a group) share a power of two as scale: values are E2M1 codes (0, 0.5, 1,
// 1.5, 2, 3, 4, 6 and their negatives) times 2^(byte - 127). gfx950 converts two codes with such a scale to
// bf16 in one instruction, exactly: a bf16 has room for the code's two significant bits and the scale's exponent.
// A key head's part of a page is K codes, V codes, K scales, V scales; within each, 16 tokens lie together as
// [group][token]: the 64 lanes of a 16x16x32 matrix operand (16 keys, four groups) then read one contiguous KB.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "convert.h"

namespace bt {

constexpr int kCacheGroup = 32;   // values that share a scale
constexpr int kCacheTile = 16;    // tokens whose codes lie together
constexpr int kCacheNaN = 252;    // scale bytes above read as NaN (the largest scale: 6 * 2^125 is finite)

__host__ __device__ inline int cache_groups(int64_t D) { return (int)((D + kCacheGroup - 1) / kCacheGroup); }
// bytes of one key head in a page: 16 + 1 for each group, of K and of V
__host__ __device__ inline int64_t cache_head_bytes(int64_t page_tokens, int64_t D)
{
    return page_tokens * cache_groups(D) * 34;
}

typedef bf16_t bf16x2 __attribute__((ext_vector_type(2)));
typedef bf16_t bf16x8 __attribute__((ext_vector_type(8)));

// The scale operand for a scale byte (only its exponent counts; all ones give NaN).
__device__ inline float cache_scale(uint32_t byte)
{
    return __uint_as_float((byte > kCacheNaN ? 255u : byte) << 23);
}

// Eight codes (lowest four bits first) times scale.
__device__ inline bf16x8 cache_values(uint32_t codes, float scale)
{
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3);
    return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

struct CacheRows {
    char *cache;
    const int *rows;
    int64_t page_bytes;
    int64_t k_row, k_head, v_row, v_head;  // strides in elements
    int64_t places;                        // pages * page_tokens
    int M, Hkv, D, groups, page_shift;
};
hipError_t launch_cache_write(const CacheRows &a, const void *k, const void *v, int type, hipStream_t s);
hipError_t launch_cache_read(const CacheRows &a, void *k, void *v, int type, hipStream_t s);

}  // namespace bt
