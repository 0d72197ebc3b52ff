// Products of int8 tokens and int8 weights (bt_int8_gemm): acc[m,n] = sum_k W[n,k] X[m,k] in int32, exact, and
// Y[m,n] = fp32(acc) * (x_scale[m] * w_scale[n]) + bias[n].
//
// Weights are packed once (bt_int8_pack) into blocks of 16 rows x 64 k, 1 KB each, byte 16 * (r + 16 g) + e of a
// block holding row r, k = 16 g + e: the operand of v_mfma_i32_16x16x64_i8 as its 64 lanes take it, so that a wave
// reads a block as one contiguous KB.
#include "bt_internal.h"
#include "convert.h"

namespace bt {
namespace {

__global__ __launch_bounds__(256) void k_int8_pack(const int8_t *W, int64_t ld, int64_t N, int64_t K, int64_t pieces,
                                                   int64_t KC, char *Wp)
{
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;  // 16 bytes of Wp
    if (id >= pieces)
        return;
    const int64_t block = id >> 6;
    const int lane = (int)(id & 63);
    const int64_t n = block / KC * 16 + (lane & 15), k = block % KC * 64 + 16 * (lane >> 4);
    __attribute__((aligned(16))) int8_t x[16];
#pragma unroll
    for (int e = 0; e < 16; ++e)
        x[e] = n < N && k + e < K ? W[n * ld + k + e] : (int8_t)0;
    *reinterpret_cast<uint4 *>(Wp + id * 16) = *reinterpret_cast<const uint4 *>(x);
}

template <typename T>
__device__ inline void store1(T *p, float v)
{
    *p = (T)v;
}

struct Int8Args {
    const char *Wp;
    const float *w_scale, *x_scale, *bias;
    const int8_t *X;
    void *Y;
    int *acc;
    int64_t M, N, ldx;
    int KC;
};

template <typename TY>
__global__ __launch_bounds__(64) void k_int8_simple(Int8Args a)
{
    const int lane = threadIdx.x, r = lane & 15, g = lane >> 4;
    const int64_t nb = blockIdx.x, mb = blockIdx.y;
    const char *w = a.Wp + nb * a.KC * 1024 + lane * 16;
    const int64_t m = mb * 16 + r;
    const int8_t *x = a.X + (m < a.M ? m : 0) * a.ldx + 16 * g;
    v4i c = {0, 0, 0, 0};
    for (int k = 0; k < a.KC; ++k) {
        const v4i wa = *reinterpret_cast<const v4i *>(w + (int64_t)k * 1024);
        const v4i xb = *reinterpret_cast<const v4i *>(x + (int64_t)k * 64);
        c = __builtin_amdgcn_mfma_i32_16x16x64_i8(wa, xb, c, 0, 0, 0);
    }
    if (m >= a.M)
        return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t n = nb * 16 + 4 * g + i;
        if (n >= a.N)
            break;
        if (a.acc)
            a.acc[m * a.N + n] = c[i];
        if (a.Y) {
            float y = (float)c[i] * (a.x_scale[m] * a.w_scale[n]);
            if (a.bias)
                y = y + a.bias[n];
            store1(static_cast<TY *>(a.Y) + m * a.N + n, y);
        }
    }
}

}  // namespace

size_t int8_weight_bytes(int64_t N, int64_t K) { return (size_t)(round_up(N, 16) * round_up(K, 64)); }

hipError_t launch_int8_pack(const int8_t *W, int64_t ld, int64_t N, int64_t K, void *Wp, hipStream_t s)
{
    const int64_t pieces = (int64_t)int8_weight_bytes(N, K) / 16;
    k_int8_pack<<<(unsigned)((pieces + 255) / 256), 256, 0, s>>>(W, ld, N, K, pieces, (K + 63) / 64,
                                                                 static_cast<char *>(Wp));
    return hipGetLastError();
}

size_t int8_workspace_bytes(int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_int8(const void *Wp, const float *w_scale, const int8_t *X, const float *x_scale, int64_t M,
                       int64_t N, int64_t K, const float *bias, void *Y, int y_type, int32_t *acc, void *, hipStream_t s)
{
    const Int8Args a = {static_cast<const char *>(Wp), w_scale, x_scale, bias, X, Y, acc, M, N, round_up(K, 256),
                        (int)((K + 63) / 64)};
    const dim3 grid((unsigned)((N + 15) / 16), (unsigned)((M + 15) / 16));
    if (y_type == kF32)
        k_int8_simple<float><<<grid, 64, 0, s>>>(a);
    else if (y_type == kBF16)
        k_int8_simple<bf16_t><<<grid, 64, 0, s>>>(a);
    else
        k_int8_simple<f16_t><<<grid, 64, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace bt
