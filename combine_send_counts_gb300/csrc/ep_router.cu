// The router: logits of a few tokens over all experts, and each token's top-k
// experts with their weights.
//
//   l[t,e] = sum over h of x[t,h] w[e,h];  score = softmax(l) or sigmoid(l);
//   key = l, or score + bias;  the K largest keys, the lower id on ties.
#include <algorithm>

#include "ep_device.cuh"
#include "ep_internal.h"

namespace ep {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

struct Select {
    const float *bias;
    int E, K, sigmoid, renormalize;
    float scale;
    int64_t *idx;
    float *weights;
};

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }

// a NaN logit counts as -inf
__device__ __forceinline__ float clean(float l) { return isnan(l) ? neg_inf() : l; }

// One warp: the top-k of one token.  l: its E logits (shared or global);
// key: E floats of the warp's own in shared memory.
__device__ __forceinline__ void select_topk(const Select &a, const float *l, float *key, int64_t t, int lane)
{
    float mx = neg_inf(), sum = 0.0f;
    if (!a.sigmoid) {
        for (int e = lane; e < a.E; e += 32)
            mx = fmaxf(mx, clean(l[e]));
        for (int o = 16; o > 0; o >>= 1)
            mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o));
        for (int e = lane; e < a.E; e += 32) {
            const float v = clean(l[e]);
            sum = __fadd_rn(sum, v == mx ? 1.0f : expf(__fsub_rn(v, mx)));
        }
        for (int o = 16; o > 0; o >>= 1)
            sum = __fadd_rn(sum, __shfl_xor_sync(kFull, sum, o));
    }
    // v == mx also where both are infinite, whose difference would be NaN
    auto score = [&](float v) {
        return a.sigmoid ? __fdiv_rn(1.0f, __fadd_rn(1.0f, expf(-v)))
                         : __fdiv_rn(v == mx ? 1.0f : expf(__fsub_rn(v, mx)), sum);
    };
    for (int e = lane; e < a.E; e += 32) {
        const float v = l[e];
        // a NaN logit is never chosen, whatever its score and bias
        float k = isnan(v) ? neg_inf() : a.bias != nullptr ? __fadd_rn(score(v), a.bias[e]) : v;
        key[e] = isnan(k) ? neg_inf() : k;
    }
    __syncwarp();
    float mine = 0.0f, chosen = 0.0f;   // lane k holds slot k
    int mine_e = -1;
    for (int k = 0; k < a.K; ++k) {
        float best = neg_inf();
        int at = -1;
        for (int e = lane; e < a.E; e += 32)
            if (key[e] > best) {
                best = key[e];
                at = e;
            }
        for (int o = 16; o > 0; o >>= 1) {
            const float b = __shfl_xor_sync(kFull, best, o);
            const int p = __shfl_xor_sync(kFull, at, o);
            if (b > best || (b == best && p >= 0 && (at < 0 || p < at))) {
                best = b;
                at = p;
            }
        }
        if (at >= 0) {
            const float s = score(l[at]);
            chosen = __fadd_rn(chosen, s);
            if (lane == k) {
                mine = s;
                mine_e = at;
            }
            if (lane == (at & 31))
                key[at] = neg_inf();
        }
        __syncwarp();
    }
    if (lane < a.K) {
        float w = mine;
        if (a.renormalize)
            w = chosen > 0.0f ? __fdiv_rn(w, chosen) : 0.0f;
        a.idx[t * a.K + lane] = mine_e;
        a.weights[t * a.K + lane] = mine_e >= 0 ? __fmul_rn(w, a.scale) : 0.0f;
    }
}

// one warp for each (token, expert)
template <bool WF32>
__global__ void __launch_bounds__(kThreads)
router_logits_kernel(const __nv_bfloat16 *__restrict__ x, const void *__restrict__ w, int64_t T, int H, int E,
                     float *__restrict__ logits)
{
    const int64_t u = (int64_t)blockIdx.x * kWarps + threadIdx.x / 32;
    const int lane = threadIdx.x & 31;
    if (u >= T * E)
        return;
    const int64_t e = u % E, t = u / E;
    float acc = 0.0f;
    for (int h = lane; h < H; h += 32) {
        const float b = WF32 ? static_cast<const float *>(w)[e * H + h]
                             : __bfloat162float(static_cast<const __nv_bfloat16 *>(w)[e * H + h]);
        acc = __fmaf_rn(__bfloat162float(x[t * H + h]), b, acc);
    }
    for (int o = 16; o > 0; o >>= 1)
        acc = __fadd_rn(acc, __shfl_xor_sync(kFull, acc, o));
    if (lane == 0)
        logits[u] = acc;
}

__global__ void __launch_bounds__(32)
router_select_kernel(Select a, const float *__restrict__ logits)
{
    extern __shared__ float s_key[];
    const int64_t t = blockIdx.x;
    select_topk(a, logits + t * a.E, s_key, t, threadIdx.x);
}

}  // namespace
}  // namespace ep

using namespace ep;

extern "C" size_t ep_router_workspace_size(int64_t T, int H, int E)
{
    if (T < 0 || H < 1 || E < 1)
        return 0;
    return std::max<size_t>(align_up((size_t)T * E * sizeof(float), kWsAlign), kWsAlign);
}

extern "C" int ep_router_topk(const void *x, int64_t T, int H, const void *w, int w_dtype, int E, const float *bias,
                              int K, int scoring, int renormalize, float scale, int64_t *topk_idx,
                              float *topk_weights, float *logits, void *ws, size_t ws_bytes, ep_stream_t stream_)
{
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    if (T < 0 || T >= ((int64_t)1 << 31) || H < 8 || H % 8 != 0 || E < 1 || E > EP_MAX_EXPERTS || K < 1 ||
        K > EP_MAX_TOPK || K > E || (scoring != EP_SCORE_SOFTMAX && scoring != EP_SCORE_SIGMOID))
        return EP_ERR_INVALID_ARG;
    if (w_dtype != 0 && w_dtype != 1)
        return EP_ERR_UNSUPPORTED;
    if (T == 0)
        return EP_OK;
    if (x == nullptr || w == nullptr || topk_idx == nullptr || topk_weights == nullptr || !aligned(x, 16) ||
        !aligned(w, 16) || ws == nullptr || !aligned(ws, kWsAlign) || ws_bytes < ep_router_workspace_size(T, H, E))
        return EP_ERR_INVALID_ARG;
    float *l = logits != nullptr ? logits : static_cast<float *>(ws);
    const int64_t blocks = ceil_div(T * E, kWarps);
    if (blocks >= ((int64_t)1 << 31))
        return EP_ERR_UNSUPPORTED;
    const auto *xb = static_cast<const __nv_bfloat16 *>(x);
    if (w_dtype == 1)
        router_logits_kernel<true><<<(unsigned)blocks, kThreads, 0, stream>>>(xb, w, T, H, E, l);
    else
        router_logits_kernel<false><<<(unsigned)blocks, kThreads, 0, stream>>>(xb, w, T, H, E, l);
    int rc = launch_status();
    if (rc != EP_OK)
        return rc;
    const Select a{bias, E, K, scoring == EP_SCORE_SIGMOID, renormalize, scale, topk_idx, topk_weights};
    router_select_kernel<<<(unsigned)T, 32, (size_t)E * sizeof(float), stream>>>(a, l);
    return launch_status();
}
