// 4-bit weights with group scales: quantise, read back, and the product with a
// few rows of x.
//
//   w[n,k] = (q[n,k] - zero[n,g]) * scale[n,g],  g = k / group
#include <algorithm>

#include "ep_device.cuh"
#include "ep_internal.h"

namespace ep {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float bf16_f(const __nv_bfloat16 *p, int64_t i) { return __bfloat162float(p[i]); }

__global__ void __launch_bounds__(kThreads)
w4_quantize_kernel(const __nv_bfloat16 *__restrict__ w, int64_t groups, int G, uint8_t *__restrict__ q,
                   __nv_bfloat16 *__restrict__ scale, uint8_t *__restrict__ zero)
{
    const int64_t g = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (g >= groups)
        return;
    const __nv_bfloat16 *src = w + g * G;
    float lo = 0.0f, hi = 0.0f;
    bool finite = true;
    for (int i = 0; i < G; ++i) {
        const float v = bf16_f(src, i);
        finite = finite && isfinite(v);
        lo = fminf(lo, v);
        hi = fmaxf(hi, v);
    }
    const bool asym = zero != nullptr;
    const float wide = asym ? __fsub_rn(__fdiv_rn(hi, 15.0f), __fdiv_rn(lo, 15.0f)) : __fdiv_rn(fmaxf(hi, -lo), 7.0f);
    const __nv_bfloat16 sb = finite ? __float2bfloat16_rn(wide) : __float2bfloat16_rn(__int_as_float(0x7f800000));
    const float s = __bfloat162float(sb);
    const bool plain = finite && s > 0.0f;
    const float z = asym ? (plain ? fminf(fmaxf(rintf(__fdiv_rn(-lo, s)), 0.0f), 15.0f) : 0.0f) : 8.0f;
    scale[g] = sb;
    if (asym)
        zero[g] = (uint8_t)z;
    for (int i = 0; i < G; i += 2) {
        unsigned b = 0;
        for (int j = 0; j < 2; ++j) {
            const float r = plain ? rintf(__fdiv_rn(bf16_f(src, i + j), s)) : 0.0f;
            b |= (unsigned)fminf(fmaxf(__fadd_rn(r, z), 0.0f), 15.0f) << (4 * j);
        }
        q[(g * G + i) >> 1] = (uint8_t)b;
    }
}

template <bool F32>
__global__ void __launch_bounds__(kThreads)
w4_dequantize_kernel(const uint8_t *__restrict__ q, const __nv_bfloat16 *__restrict__ scale,
                     const uint8_t *__restrict__ zero, int64_t pairs, int G, void *__restrict__ out)
{
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (i >= pairs)
        return;
    const int64_t g = 2 * i / G;
    const float s = __bfloat162float(scale[g]), z = zero != nullptr ? (float)zero[g] : 8.0f;
    const unsigned b = q[i];
    const float v0 = __fmul_rn((float)(b & 15) - z, s), v1 = __fmul_rn((float)(b >> 4) - z, s);
    if (F32)
        reinterpret_cast<float2 *>(out)[i] = make_float2(v0, v1);
    else
        reinterpret_cast<uint32_t *>(out)[i] = pack_bf16x2(v0, v1);
}

// one warp for each (row of w, row of x)
template <bool F32>
__global__ void __launch_bounds__(kThreads)
w4_matvec_kernel(const __nv_bfloat16 *__restrict__ x, const uint8_t *__restrict__ q,
                 const __nv_bfloat16 *__restrict__ scale, const uint8_t *__restrict__ zero, int64_t M, int64_t N,
                 int64_t K, int G, void *__restrict__ y)
{
    const int64_t u = (int64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
    const int lane = threadIdx.x & 31;
    if (u >= M * N)
        return;
    const int64_t n = u % N, m = u / N;
    const int64_t ng = K / G;
    float acc = 0.0f;
    for (int64_t g = 0; g < ng; ++g) {
        const float z = zero != nullptr ? (float)zero[n * ng + g] : 8.0f;
        float part = 0.0f;
        for (int64_t k = g * G + lane; k < (g + 1) * G; k += 32) {
            const unsigned b = q[(n * K + k) >> 1];
            part = __fmaf_rn(bf16_f(x, m * K + k), (float)((b >> (4 * (k & 1))) & 15) - z, part);
        }
        acc = __fmaf_rn(part, bf16_f(scale, n * ng + g), acc);
    }
    for (int o = 16; o > 0; o >>= 1)
        acc = __fadd_rn(acc, __shfl_xor_sync(kFull, acc, o));
    if (lane == 0) {
        if (F32)
            static_cast<float *>(y)[m * N + n] = acc;
        else
            static_cast<__nv_bfloat16 *>(y)[m * N + n] = __float2bfloat16_rn(acc);
    }
}

bool w4_shape_ok(int64_t N, int64_t K, int group)
{
    return N >= 0 && K >= 1 && N < ((int64_t)1 << 40) && K < ((int64_t)1 << 31) &&
           (group == 32 || group == 64 || group == 128) && K % group == 0;
}

}  // namespace
}  // namespace ep

using namespace ep;

extern "C" int ep_w4_quantize(const void *w, int64_t N, int64_t K, int group, uint8_t *q, void *scale, uint8_t *zero,
                              ep_stream_t stream_)
{
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    if (!w4_shape_ok(N, K, group))
        return EP_ERR_INVALID_ARG;
    if (N == 0)
        return EP_OK;
    if (w == nullptr || q == nullptr || scale == nullptr || !aligned(w, 16) || !aligned(q, 16) || !aligned(scale, 2))
        return EP_ERR_INVALID_ARG;
    const int64_t groups = N * (K / group), blocks = ceil_div(groups, kThreads);
    if (blocks >= ((int64_t)1 << 31))
        return EP_ERR_UNSUPPORTED;
    w4_quantize_kernel<<<(unsigned)blocks, kThreads, 0, stream>>>(static_cast<const __nv_bfloat16 *>(w), groups, group,
                                                                 q, static_cast<__nv_bfloat16 *>(scale), zero);
    return launch_status();
}

extern "C" int ep_w4_dequantize(const uint8_t *q, const void *scale, const uint8_t *zero, int64_t N, int64_t K,
                                int group, void *w, int out_dtype, ep_stream_t stream_)
{
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    if (!w4_shape_ok(N, K, group))
        return EP_ERR_INVALID_ARG;
    if (out_dtype != 0 && out_dtype != 1)
        return EP_ERR_UNSUPPORTED;
    if (N == 0)
        return EP_OK;
    if (w == nullptr || q == nullptr || scale == nullptr || !aligned(w, 16) || !aligned(q, 16) || !aligned(scale, 2))
        return EP_ERR_INVALID_ARG;
    const int64_t pairs = N * K / 2, blocks = ceil_div(pairs, kThreads);
    if (blocks >= ((int64_t)1 << 31))
        return EP_ERR_UNSUPPORTED;
    const auto *s = static_cast<const __nv_bfloat16 *>(scale);
    if (out_dtype == 1)
        w4_dequantize_kernel<true><<<(unsigned)blocks, kThreads, 0, stream>>>(q, s, zero, pairs, group, w);
    else
        w4_dequantize_kernel<false><<<(unsigned)blocks, kThreads, 0, stream>>>(q, s, zero, pairs, group, w);
    return launch_status();
}

extern "C" int ep_w4_matvec(const void *x, int64_t M, const uint8_t *q, const void *scale, const uint8_t *zero,
                            int64_t N, int64_t K, int group, void *y, int out_dtype, ep_stream_t stream_)
{
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    if (!w4_shape_ok(N, K, group) || M < 0)
        return EP_ERR_INVALID_ARG;
    if (out_dtype != 0 && out_dtype != 1)
        return EP_ERR_UNSUPPORTED;
    if (M == 0 || N == 0)
        return EP_OK;
    if (x == nullptr || q == nullptr || scale == nullptr || y == nullptr || !aligned(x, 16) || !aligned(q, 16) ||
        !aligned(scale, 2) || !aligned(y, 16))
        return EP_ERR_INVALID_ARG;
    const int64_t blocks = ceil_div(M * N, kThreads / 32);
    if (M >= ((int64_t)1 << 20) || N >= ((int64_t)1 << 31) || blocks >= ((int64_t)1 << 31))
        return EP_ERR_UNSUPPORTED;
    const auto *xb = static_cast<const __nv_bfloat16 *>(x);
    const auto *s = static_cast<const __nv_bfloat16 *>(scale);
    if (out_dtype == 1)
        w4_matvec_kernel<true><<<(unsigned)blocks, kThreads, 0, stream>>>(xb, q, s, zero, M, N, K, group, y);
    else
        w4_matvec_kernel<false><<<(unsigned)blocks, kThreads, 0, stream>>>(xb, q, s, zero, M, N, K, group, y);
    return launch_status();
}
