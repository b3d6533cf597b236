// The choice of experts from logits, with groups of experts, and its backward
// pass.
//
//   score = softmax(l) or sigmoid(l);  key = l, or score + bias;
//   a group's mark = its largest key, or the sum of its two largest (of scores
//   where there is no bias); the `kept` groups of largest mark stay;
//   the K largest keys in them, the lower id on ties;
//   w = score (/ sum of the chosen scores) * scale.
//
// Keys and marks are compared as they come out in 64 bits: with a million
// scores in a batch some two are nearer than fp32 tells apart.
#include <algorithm>

#include "ep_device.cuh"
#include "ep_internal.h"
#include "ep_launch.cuh"
#include "ep_select.cuh"

namespace ep {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ double neg_inf64() { return __longlong_as_double(0xfff0000000000000ll); }
__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }

__device__ __forceinline__ float ld_float(const float *p)
{
    return __uint_as_float(ld_global(reinterpret_cast<const uint32_t *>(p)));
}

__device__ __forceinline__ float ld_logit(const void *p, int dtype, int64_t at)
{
    if (dtype == 0)
        return ld_float(static_cast<const float *>(p) + at);
    return __uint_as_float((uint32_t)ld_global(static_cast<const uint16_t *>(p) + at) << 16);
}

// Logit e of token t; its slices are added in their order.
__device__ __forceinline__ float logit_of(const Choice &c, int64_t t, int e)
{
    float v = ld_logit(c.logits, c.dtype, t * c.E + e);
    for (int z = 1; z < c.slices; ++z)
        v = __fadd_rn(v, ld_float(static_cast<const float *>(c.logits) + ((int64_t)z * c.T + t) * c.E + e));
    return v;
}

// Scores of a token in 64 bits; v == mx also where both are infinite, whose difference is NaN.
struct Score64 {
    int sigmoid;
    double mx, sum;

    __device__ __forceinline__ double operator()(float l) const
    {
        if (isnan(l))
            return 0.0;
        if (sigmoid)
            return 1.0 / (1.0 + exp(-(double)l));
        return ((double)l == mx ? 1.0 : exp((double)l - mx)) / sum;
    }
};

__device__ __forceinline__ double shfl_xor64(double v, int o) { return __shfl_xor_sync(kFull, v, o); }

template <bool MAX>
__device__ __forceinline__ double block_reduce64(double v, double *s)
{
    for (int o = 16; o > 0; o >>= 1) {
        const double u = shfl_xor64(v, o);
        v = MAX ? fmax(v, u) : v + u;
    }
    if ((threadIdx.x & 31) == 0)
        s[threadIdx.x >> 5] = v;
    __syncthreads();
    v = s[0];
    for (int w = 1; w < kWarps; ++w)
        v = MAX ? fmax(v, s[w]) : v + s[w];
    return v;
}

// Any number of experts: a block per token, all keys in 64 bits in shared memory.
__global__ void __launch_bounds__(kThreads)
select_kernel(Choice c)
{
    extern __shared__ double dynamic[];   // [E] keys, [E] logits
    __shared__ double s_max[kWarps], s_sum[kWarps], mark[kMaxGroups];
    double *key = dynamic;
    float *l = reinterpret_cast<float *>(dynamic + c.E);
    const int64_t t = blockIdx.x;
    grid_dependency_wait();
    allow_dependents();
    double mx = neg_inf64();
    for (int e = threadIdx.x; e < c.E; e += kThreads) {
        const float v = logit_of(c, t, e);
        if (c.sums != nullptr)
            c.sums[t * c.E + e] = v;
        l[e] = v;
        mx = fmax(mx, isnan(v) ? neg_inf64() : (double)v);
    }
    Score64 score{c.sigmoid, 0.0, 1.0};
    if (!c.sigmoid) {
        score.mx = block_reduce64<true>(mx, s_max);
        double part = 0.0;
        for (int e = threadIdx.x; e < c.E; e += kThreads)
            part += score(l[e]);
        score.sum = block_reduce64<false>(part, s_sum);
    }
    for (int e = threadIdx.x; e < c.E; e += kThreads) {
        const float v = l[e];
        const double k = isnan(v) ? neg_inf64()
                         : c.bias != nullptr ? score(v) + (double)ld_float(c.bias + e) : (double)v;
        key[e] = isnan(k) ? neg_inf64() : k + 0.0;   // -0 and +0 are one key
    }
    __syncthreads();
    if (c.groups > 1) {
        const int size = c.E / c.groups;
        const bool of_scores = c.top2 && c.bias == nullptr;
        for (int g = threadIdx.x; g < c.groups; g += kThreads) {
            double a = neg_inf64(), b = neg_inf64();
            for (int e = g * size; e < (g + 1) * size; ++e) {
                if (key[e] == neg_inf64())
                    continue;
                const double k = of_scores ? score(l[e]) : key[e];
                if (k > a) {
                    b = a;
                    a = k;
                } else if (k > b) {
                    b = k;
                }
            }
            mark[g] = c.top2 && b != neg_inf64() ? a + b : a;
        }
        __syncthreads();
        for (int e = threadIdx.x; e < c.E; e += kThreads) {
            const int g = e / size;
            int ahead = 0;
            for (int o = 0; o < c.groups; ++o)
                ahead += mark[o] > mark[g] || (mark[o] == mark[g] && o < g);
            if (ahead >= c.kept)
                key[e] = neg_inf64();
        }
        __syncthreads();
    }
    if (threadIdx.x >= 32)
        return;
    const int lane = threadIdx.x;
    double best;   // this lane's best key and where it is
    int at;
    auto scan = [&]() {
        best = neg_inf64();
        at = -1;
        for (int e = lane; e < c.E; e += 32)
            if (key[e] > best) {
                best = key[e];
                at = e;
            }
    };
    scan();
    int mine_e = -1;   // lane k holds slot k
    for (int k = 0; k < c.K; ++k) {
        double top = best;
        int e = at;
        for (int o = 16; o > 0; o >>= 1) {
            const double u = shfl_xor64(top, o);
            const int f = __shfl_xor_sync(kFull, e, o);
            if (u > top || (u == top && (unsigned)f < (unsigned)e)) {
                top = u;
                e = f;
            }
        }
        if (e < 0)
            break;
        if (lane == k)
            mine_e = e;
        if (lane == (e & 31)) {
            key[e] = neg_inf64();
            scan();
        }
        __syncwarp();
    }
    const double mine = mine_e >= 0 ? score(l[mine_e]) : 0.0;
    double chosen = 0.0;   // the scores are positive or +0: those of empty slots change nothing
    for (int k = 0; k < c.K; ++k)
        chosen += __shfl_sync(kFull, mine, k);
    if (lane < c.K) {
        const double w = !c.renormalize ? mine : chosen > 0.0 ? mine / chosen : 0.0;
        c.idx[t * c.K + lane] = mine_e;
        c.weights[t * c.K + lane] = mine_e >= 0 ? (float)(w * (double)c.scale) : 0.0f;
    }
}

// ------------------------------------------------------------ backward pass --
struct Backward {
    const void *logits;
    int dtype, T, E, K, sigmoid, renormalize;
    float scale;
    const int64_t *idx;
    const float *dw;
    void *out;
    int32_t *err;
};

__device__ __forceinline__ float warp_sum(float v)
{
    for (int o = 16; o > 0; o >>= 1)
        v = __fadd_rn(v, __shfl_xor_sync(kFull, v, o));
    return v;
}

__device__ __forceinline__ float warp_max(float v)
{
    for (int o = 16; o > 0; o >>= 1)
        v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
    return v;
}

__device__ __forceinline__ void st_logit(void *p, int dtype, int64_t at, float v)
{
    if (dtype == 0)
        static_cast<float *>(p)[at] = v;
    else
        static_cast<uint16_t *>(p)[at] = (uint16_t)(pack_bf16x2(v, 0.0f) & 0xffffu);
}

// A warp per token, lane k with slot k.  First what every logit gets, then the chosen ones over it.
__global__ void __launch_bounds__(kThreads)
select_backward_kernel(Backward b)
{
    const int lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    grid_dependency_wait();
    allow_dependents();
    if (t >= b.T)
        return;
    int e = -1;
    float g = 0.0f;
    if (lane < b.K) {
        const uint2 w = ld_global(reinterpret_cast<const uint2 *>(b.idx) + t * b.K + lane);
        const int64_t id = (int64_t)((uint64_t)w.y << 32 | w.x);
        if (id < -1 || id >= b.E)
            raise(b.err, EP_ERR_INVALID_EXPERT);
        else
            e = (int)id;
        if (e >= 0)
            g = __fmul_rn(ld_float(b.dw + t * b.K + lane), b.scale);
    }
    const float l = e >= 0 ? ld_logit(b.logits, b.dtype, t * b.E + e) : neg_inf();
    const bool there = l > neg_inf();   // a logit of NaN or -inf gets nothing
    // softmax divided by the chosen ones' sum: the others cancel
    const bool whole = !b.sigmoid && !b.renormalize;
    float mx = there ? l : neg_inf();
    if (whole)
        for (int i = lane; i < b.E; i += 32)
            mx = fmaxf(mx, ld_logit(b.logits, b.dtype, t * b.E + i));
    mx = warp_max(mx);
    auto power = [&](float v) { return isnan(v) ? 0.0f : v == mx ? 1.0f : expf(__fsub_rn(v, mx)); };
    float sum = 1.0f;
    if (whole) {
        sum = 0.0f;
        for (int i = lane; i < b.E; i += 32)
            sum = __fadd_rn(sum, power(ld_logit(b.logits, b.dtype, t * b.E + i)));
        sum = warp_sum(sum);
    }
    // s: the score, or, where only its share of the chosen ones' sum counts, a multiple of it that does
    // not vanish; rest: the derivative of its logarithm by the logit, but for what `whole` takes off
    float s = 0.0f, rest = 1.0f;
    if (there && b.sigmoid) {
        const float x = expf(-fabsf(l)), d = __fdiv_rn(1.0f, __fadd_rn(1.0f, x)), m = __fmul_rn(x, d);
        rest = l >= 0.0f ? m : d;
        s = l >= 0.0f ? d : b.renormalize && mx < 0.0f ? __fmul_rn(expf(__fsub_rn(l, mx)), d) : m;
    } else if (there) {
        s = __fdiv_rn(power(l), sum);
    }
    if (b.renormalize) {
        const float chosen = warp_sum(s);
        s = chosen > 0.0f ? __fdiv_rn(s, chosen) : 0.0f;
        g = __fsub_rn(g, warp_sum(__fmul_rn(g, s)));
    }
    const float dot = whole ? warp_sum(__fmul_rn(g, s)) : 0.0f;
    for (int i = lane; i < b.E; i += 32) {
        float v = 0.0f;
        if (whole)
            v = -__fmul_rn(__fdiv_rn(power(ld_logit(b.logits, b.dtype, t * b.E + i)), sum), dot);
        st_logit(b.out, b.dtype, t * b.E + i, v);
    }
    // slots that name the same expert are added in their order, by the first
    float total = 0.0f;
    bool first = there;
    for (int k = 0; k < b.K; ++k) {
        const int o = __shfl_sync(kFull, e, k);
        const float u = __shfl_sync(kFull, g, k);
        if (o == e)
            total = __fadd_rn(total, u);
        if (o == e && k < lane)
            first = false;
    }
    __syncwarp();
    if (first)
        st_logit(b.out, b.dtype, t * b.E + e, __fmul_rn(__fmul_rn(s, rest), __fsub_rn(total, dot)));
}

}  // namespace

int choice_status(int E, int K, int scoring, int num_groups, int topk_groups, int group_score)
{
    if (E < 1 || E > EP_MAX_EXPERTS || K < 1 || K > EP_MAX_TOPK || K > E ||
        (scoring != EP_SCORE_SOFTMAX && scoring != EP_SCORE_SIGMOID) || num_groups < 1 || E % num_groups != 0 ||
        topk_groups < 1 || topk_groups > num_groups ||
        (group_score != EP_GROUP_MAX && group_score != EP_GROUP_TOP2))
        return EP_ERR_INVALID_ARG;
    return num_groups > kMaxGroups ? EP_ERR_UNSUPPORTED : EP_OK;
}

int launch_choice(const Choice &c, cudaStream_t stream)
{
    static PerDevice set;
    const int rc = raise_smem(select_kernel, EP_MAX_EXPERTS * (sizeof(double) + sizeof(float)), set);
    if (rc != EP_OK)
        return rc;
    return launch_dependent(select_kernel, dim3((unsigned)c.T), kThreads, (size_t)c.E * (sizeof(double) + sizeof(float)),
                            stream, c);
}

}  // namespace ep

using namespace ep;

extern "C" int ep_router_select(const void *logits, int dtype, int64_t T, int E, const float *bias, int K, int scoring,
                                int num_groups, int topk_groups, int group_score, int renormalize, float scale,
                                int64_t *topk_idx, float *topk_weights, ep_stream_t stream_)
{
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    const int rc = choice_status(E, K, scoring, num_groups, topk_groups, group_score);
    if (T < 0 || rc == EP_ERR_INVALID_ARG)
        return EP_ERR_INVALID_ARG;
    if (rc != EP_OK || (dtype != 0 && dtype != 1) || T > INT32_MAX)
        return EP_ERR_UNSUPPORTED;
    if (T == 0)
        return EP_OK;
    if (logits == nullptr || topk_idx == nullptr || topk_weights == nullptr || !aligned(logits, dtype == 0 ? 4 : 2) ||
        !aligned(bias, 4) || !aligned(topk_idx, 8) || !aligned(topk_weights, 4))
        return EP_ERR_INVALID_ARG;
    const Choice c{logits, dtype, 1, bias, (int)T, E, K, scoring == EP_SCORE_SIGMOID, num_groups, topk_groups,
                   group_score == EP_GROUP_TOP2, renormalize, scale, topk_idx, topk_weights, nullptr};
    return launch_choice(c, stream);
}

extern "C" int ep_router_select_backward(const void *logits, int dtype, int64_t T, int E, const int64_t *topk_idx,
                                         const float *dweights, int K, int scoring, int renormalize, float scale,
                                         void *dlogits, int32_t *err, ep_stream_t stream_)
{
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    if (T < 0 || choice_status(E, std::min(K, E), scoring, 1, 1, EP_GROUP_MAX) != EP_OK || K < 1 || K > EP_MAX_TOPK)
        return EP_ERR_INVALID_ARG;
    if ((dtype != 0 && dtype != 1) || T > INT32_MAX)
        return EP_ERR_UNSUPPORTED;
    if (T == 0)
        return EP_OK;
    if (logits == nullptr || topk_idx == nullptr || dweights == nullptr || dlogits == nullptr || logits == dlogits ||
        !aligned(logits, dtype == 0 ? 4 : 2) || !aligned(dlogits, dtype == 0 ? 4 : 2) || !aligned(topk_idx, 8) ||
        !aligned(dweights, 4) || !aligned(err, 4))
        return EP_ERR_INVALID_ARG;
    const Backward b{logits, dtype, (int)T, E, K, scoring == EP_SCORE_SIGMOID, renormalize, scale, topk_idx, dweights,
                     dlogits, err};
    return launch_dependent(select_backward_kernel, dim3((unsigned)ceil_div(T, kWarps)), kThreads, 0, stream, b);
}
