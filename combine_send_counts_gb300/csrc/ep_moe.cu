// The experts of a mixture-of-experts layer for a few tokens.
//
//   h[s] = silu(Wg x) * (Wu x) for every slot s = (t, k) that names a local
//   expert;  out[t] = sum over k of w[t,k] * (W2 h[t,k]).
#include <algorithm>

#include "ep_device.cuh"
#include "ep_internal.h"

namespace ep {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

struct Weights {
    const void *data;
    const __nv_bfloat16 *scale;
    const uint8_t *zero;
    int G;
};

struct Routing {
    const int64_t *idx;
    int K, E, E_local;
    int64_t first;   // first local expert

    // local expert of slot s, or -1
    __device__ __forceinline__ int local(int s, int32_t *err) const
    {
        const int64_t v = idx[s];
        if (v < -1 || v >= E) {
            raise(err, EP_ERR_INVALID_EXPERT);
            return -1;
        }
        const int64_t l = v - first;
        return v >= 0 && l >= 0 && l < E_local ? (int)l : -1;
    }
};

// one warp's dot product of row `row` ([rows, K] matrix) with v(k)
template <bool W4, class V>
__device__ __forceinline__ float dot(const Weights &w, int64_t row, int K, int lane, V v)
{
    float acc = 0.0f;
    if (W4) {
        const int ng = K / w.G;
        for (int g = 0; g < ng; ++g) {
            const float z = w.zero != nullptr ? (float)w.zero[row * ng + g] : 8.0f;
            float part = 0.0f;
            for (int k = g * w.G + lane; k < (g + 1) * w.G; k += 32) {
                const unsigned b = static_cast<const uint8_t *>(w.data)[(row * K + k) >> 1];
                part = __fmaf_rn(v(k), (float)((b >> (4 * (k & 1))) & 15) - z, part);
            }
            acc = __fmaf_rn(part, __bfloat162float(w.scale[row * ng + g]), acc);
        }
    } else {
        for (int k = lane; k < K; k += 32)
            acc = __fmaf_rn(v(k), __bfloat162float(static_cast<const __nv_bfloat16 *>(w.data)[row * K + k]), acc);
    }
    for (int o = 16; o > 0; o >>= 1)
        acc = __fadd_rn(acc, __shfl_xor_sync(kFull, acc, o));
    return acc;
}

// one warp for each (slot, row of h)
template <bool W4>
__global__ void __launch_bounds__(kThreads)
moe_up_kernel(const __nv_bfloat16 *__restrict__ x, Routing r, int n, int H, int I, Weights w13, float *__restrict__ h,
              int32_t *err)
{
    const int u = blockIdx.x * kWarps + threadIdx.x / 32, lane = threadIdx.x & 31;
    if (u >= n * I)
        return;
    const int s = u / I, i = u % I;
    const int e = r.local(s, err);
    if (e < 0)
        return;
    const __nv_bfloat16 *row = x + (int64_t)(s / r.K) * H;
    auto v = [&](int k) { return __bfloat162float(row[k]); };
    const float g = dot<W4>(w13, (int64_t)e * 2 * I + i, H, lane, v);
    const float up = dot<W4>(w13, (int64_t)e * 2 * I + I + i, H, lane, v);
    if (lane == 0)
        h[u] = __fmul_rn(__fdiv_rn(g, __fadd_rn(1.0f, expf(-g))), up);
}

// one warp for each (token, element of its row)
template <bool W4, bool F32>
__global__ void __launch_bounds__(kThreads)
moe_down_kernel(Routing r, const float *__restrict__ weights, int64_t T, int H, int I, Weights w2,
                const float *__restrict__ h, void *__restrict__ out)
{
    const int64_t u = (int64_t)blockIdx.x * kWarps + threadIdx.x / 32;
    const int lane = threadIdx.x & 31;
    if (u >= T * H)
        return;
    const int64_t t = u / H, n = u % H;
    float acc = 0.0f;
    for (int k = 0; k < r.K; ++k) {
        const int s = (int)t * r.K + k;
        const int e = r.local(s, nullptr);
        if (e < 0)
            continue;
        const float *hs = h + (int64_t)s * I;
        acc = __fmaf_rn(weights[s], dot<W4>(w2, (int64_t)e * H + n, I, lane, [&](int i) { return hs[i]; }), acc);
    }
    if (lane == 0) {
        if (F32)
            static_cast<float *>(out)[u] = acc;
        else
            static_cast<__nv_bfloat16 *>(out)[u] = __float2bfloat16_rn(acc);
    }
}

bool matrix_ok(const ep_matrix *m)
{
    return m->data != nullptr && aligned(m->data, 16) &&
           (m->format == EP_W_BF16 ? m->scale == nullptr && m->zero == nullptr && m->group == 0
                                   : m->scale != nullptr && aligned(m->scale, 2));
}

template <bool W4>
int launch(const void *x, const float *topk_weights, const Routing &r, int64_t T, int H, int I, const ep_matrix *w13,
           const ep_matrix *w2, void *out, int out_dtype, void *ws, int32_t *err, cudaStream_t stream)
{
    const int n = (int)T * r.K;
    float *h = static_cast<float *>(ws);
    const Weights a{w13->data, static_cast<const __nv_bfloat16 *>(w13->scale), w13->zero, w13->group};
    const Weights b{w2->data, static_cast<const __nv_bfloat16 *>(w2->scale), w2->zero, w2->group};
    moe_up_kernel<W4><<<(unsigned)ceil_div((int64_t)n * I, kWarps), kThreads, 0, stream>>>(
        static_cast<const __nv_bfloat16 *>(x), r, n, H, I, a, h, err);
    int rc = launch_status();
    if (rc != EP_OK)
        return rc;
    const unsigned blocks = (unsigned)ceil_div(T * H, kWarps);
    if (out_dtype == 1)
        moe_down_kernel<W4, true><<<blocks, kThreads, 0, stream>>>(r, topk_weights, T, H, I, b, h, out);
    else
        moe_down_kernel<W4, false><<<blocks, kThreads, 0, stream>>>(r, topk_weights, T, H, I, b, h, out);
    return launch_status();
}

}  // namespace
}  // namespace ep

using namespace ep;

extern "C" size_t ep_moe_workspace_size(int64_t T, int K, int I)
{
    if (T < 0 || K < 1 || I < 1)
        return 0;
    return std::max<size_t>(align_up((size_t)T * K * I * 6, kWsAlign), kWsAlign);
}

extern "C" int ep_moe_decode(const void *x, const int64_t *topk_idx, const float *topk_weights, int64_t T, int K,
                             int H, int I, int E, int E_local, int rank, const ep_matrix *w13, const ep_matrix *w2,
                             void *out, int out_dtype, void *ws, size_t ws_bytes, int32_t *err, ep_stream_t stream_)
{
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    if (T < 0 || K < 1 || K > EP_MAX_TOPK || H < 8 || H % 8 != 0 || I < 8 || I % 8 != 0 || E < 1 ||
        E > EP_MAX_EXPERTS || E_local < 1 || E % E_local != 0 || rank < 0 || rank >= E / E_local || w13 == nullptr ||
        w2 == nullptr)
        return EP_ERR_INVALID_ARG;
    if ((out_dtype != 0 && out_dtype != 1) || (w13->format != EP_W_BF16 && w13->format != EP_W_INT4) ||
        w2->format != w13->format || w2->group != w13->group)
        return EP_ERR_UNSUPPORTED;
    if (w13->format == EP_W_INT4) {
        const int g = w13->group;
        if ((g != 32 && g != 64 && g != 128) || H % g != 0 || I % g != 0)
            return EP_ERR_INVALID_ARG;
    }
    if (T * K > EP_MOE_MAX_SLOTS || H >= (1 << 20) || I >= (1 << 20))
        return EP_ERR_UNSUPPORTED;
    if (T == 0)
        return EP_OK;
    if (x == nullptr || topk_idx == nullptr || topk_weights == nullptr || out == nullptr || !aligned(x, 16) ||
        !aligned(out, 16) || !matrix_ok(w13) || !matrix_ok(w2) || ws == nullptr || !aligned(ws, kWsAlign) ||
        ws_bytes < ep_moe_workspace_size(T, K, I))
        return EP_ERR_INVALID_ARG;
    const Routing r{topk_idx, K, E, E_local, (int64_t)rank * E_local};
    if (w13->format == EP_W_INT4)
        return launch<true>(x, topk_weights, r, T, H, I, w13, w2, out, out_dtype, ws, err, stream);
    return launch<false>(x, topk_weights, r, T, H, I, w13, w2, out, out_dtype, ws, err, stream);
}
