// Element types of the attention-block operators (fp32, bf16, fp16): four-value loads and
// stores, conversions rounding to nearest even.
#pragma once

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

namespace bt {

constexpr int kF32 = 0, kBF16 = 1, kF16 = 2;  // BT_F32, BT_BF16, BT_F16

typedef __bf16 bf16_t;
typedef _Float16 f16_t;
typedef float f32x4 __attribute__((ext_vector_type(4)));

template <typename T>
struct vec4_of;
template <>
struct vec4_of<float> {
    typedef float type __attribute__((ext_vector_type(4)));
};
template <>
struct vec4_of<bf16_t> {
    typedef bf16_t type __attribute__((ext_vector_type(4)));
};
template <>
struct vec4_of<f16_t> {
    typedef f16_t type __attribute__((ext_vector_type(4)));
};

template <typename T>
__device__ inline void load4(const T *p, float (&v)[4])
{
    const auto x = *reinterpret_cast<const typename vec4_of<T>::type *>(p);
    const f32x4 f = __builtin_convertvector(x, f32x4);
#pragma unroll
    for (int j = 0; j < 4; ++j)
        v[j] = f[j];
}

template <typename T>
__device__ inline void store4(T *p, const float (&v)[4])
{
    const f32x4 f = {v[0], v[1], v[2], v[3]};
    *reinterpret_cast<typename vec4_of<T>::type *>(p) = __builtin_convertvector(f, typename vec4_of<T>::type);
}

__device__ inline bool not_finite(float x) { return !(fabsf(x) < INFINITY); }

inline int type_bytes(int type) { return type == kF32 ? 4 : 2; }

}  // namespace bt
