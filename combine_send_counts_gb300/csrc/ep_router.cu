// The router: logits of the tokens over all experts, and each token's top-k
// experts with their weights.
//
//   l[t,e] = sum over h of x[t,h] w[e,h];  score = softmax(l) or sigmoid(l);
//   key = l, or score + bias;  the K largest keys, the lower id on ties.
//
// Two kernels, the second launched while the first drains.  For a few tokens
// the whole is latency: 256 experts of 7168 columns are 3.7 MB, half a
// microsecond of HBM.
//
//   logits: matrix steps of 16 experts with 8 tokens as columns, weights loaded
//   straight into their registers.  A block has 16 experts, 8 or 16 tokens and
//   one of `slices` parts of the columns, its 8 warps an eighth of that each;
//   there are as many slices as fill the GPU once, so that a warp has one or
//   two rounds of loads.  The slices' sums are left in the workspace.  (Blocks
//   of 64 experts, which read x a quarter as often, took 25.9 us instead of
//   16.6 for 200 tokens, 256 experts and 7168 columns, 170 instead of 126 for
//   4096 tokens, and 611 instead of 678 only at 16384.)
//   select: a block per token adds the slices in ascending order and scores;
//   its first warp takes the K experts, each lane keeping the best of its own
//   keys so that a round is two reductions and one lane's rescan.
//
// Measured: one token, 256 experts of 7168, 6.6 us; 200 tokens, 64 experts of
// 2048, 5.8 us; 1024 tokens, 256 experts of 7168, 40 us; 16384 tokens, 672 us.
// Two launches, the first loads and K rounds of reductions are what is left of
// the small ones; the large ones read x once for each 16 experts.
#include <algorithm>

#include "ep_device.cuh"
#include "ep_internal.h"
#include "ep_launch.cuh"
#include "ep_select.cuh"
#include "ep_skinny.cuh"

namespace ep {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kUnit = 32;             // columns of a lane's 16-byte pieces: two k16 steps
constexpr int kSelectThreads = 128;
constexpr int kAtOnce = 8;            // slices whose sums select loads together

struct LogitsArgs {
    const uint8_t *x, *w;
    int T, H, E, slices;
    float *sums;        // [slices][T][E]
};

struct Select {
    const float *sums;
    const float *bias;
    int T, E, K, slices, sigmoid, renormalize;
    float scale;
    int64_t *idx;
    float *weights, *logits;
};

// A lane's 8 columns of a row as TERMS sums of bf16: bf16 weights as they are,
// fp32 ones split exactly into three (8 bits each).
template <int TERMS>
struct Piece {
    uint4 v[TERMS == 1 ? 1 : 2];

    __device__ __forceinline__ void load(const uint8_t *row, int k, bool ok)
    {
#pragma unroll
        for (int i = 0; i < (TERMS == 1 ? 1 : 2); ++i) {
            v[i] = make_uint4(0, 0, 0, 0);
            if (ok)
                v[i] = ld_global(reinterpret_cast<const uint4 *>(row + (int64_t)k * (TERMS == 1 ? 2 : 4)) + i);
        }
    }

    __device__ __forceinline__ static uint32_t term(float &a, float &b)
    {
        const uint32_t ha = __float_as_uint(a) & 0xffff0000u, hb = __float_as_uint(b) & 0xffff0000u;
        // what is left of an infinity or NaN is nothing
        a = isfinite(a) ? __fsub_rn(a, __uint_as_float(ha)) : 0.0f;
        b = isfinite(b) ? __fsub_rn(b, __uint_as_float(hb)) : 0.0f;
        return (ha >> 16) | hb;
    }

    __device__ __forceinline__ void split(uint4 (&t)[TERMS]) const
    {
        if (TERMS == 1) {
            t[0] = v[0];
            return;
        }
        const uint4 a = v[0], b = v[TERMS > 1];
        float f[8] = {__uint_as_float(a.x), __uint_as_float(a.y), __uint_as_float(a.z), __uint_as_float(a.w),
                      __uint_as_float(b.x), __uint_as_float(b.y), __uint_as_float(b.z), __uint_as_float(b.w)};
#pragma unroll
        for (int i = 0; i < 8; ++i)
            f[i] = isnan(f[i]) ? __int_as_float(0x7fffffff) : f[i];   // set where the first term looks
#pragma unroll
        for (int i = 0; i < TERMS; ++i) {
            t[i].x = term(f[0], f[1]);
            t[i].y = term(f[2], f[3]);
            t[i].z = term(f[4], f[5]);
            t[i].w = term(f[6], f[7]);
        }
    }
};

// Two bf16 with 0 in place of an infinity or NaN.
__device__ __forceinline__ uint32_t finite_bf16x2(uint32_t v)
{
    return v & ~__vcmpeq2(v & 0x7f807f80u, 0x7f807f80u);
}

template <int TERMS, int NT>
__global__ void __launch_bounds__(kThreads)
router_logits_kernel(LogitsArgs a)
{
    __shared__ __align__(16) float red[kWarps][NT * 32 * 4];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int t0 = blockIdx.x * (8 * NT), e0 = blockIdx.y * 16, z = blockIdx.z;
    const int units = (a.H + kUnit - 1) / kUnit, parts = a.slices * kWarps, part = z * kWarps + warp;
    const int u0 = (int)((int64_t)units * part / parts), u1 = (int)((int64_t)units * (part + 1) / parts);
    const int64_t row_bytes = (int64_t)a.H * (TERMS == 1 ? 2 : 4);
    constexpr int kBatch = TERMS == 1 ? 4 : 2;   // units loaded together
    grid_dependency_wait();
    allow_dependents();
    float acc[1][NT][4] = {};
    for (int u = u0; u < u1; u += kBatch) {
        Piece<TERMS> pa[kBatch], pb[kBatch];
        uint4 x[kBatch][NT];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int k = (u + i) * kUnit + 8 * t;
            const bool in = u + i < u1 && k < a.H;
            const int e = e0 + g;
            pa[i].load(a.w + e * row_bytes, k, in && e < a.E);
            pb[i].load(a.w + (e + 8) * row_bytes, k, in && e + 8 < a.E);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int tok = t0 + n * 8 + g;
                x[i][n] = make_uint4(0, 0, 0, 0);
                if (in && tok < a.T)
                    x[i][n] = ld_global(reinterpret_cast<const uint4 *>(a.x + ((int64_t)tok * a.H + k) * 2));
            }
        }
        float sum[NT][4] = {};   // of at most 128 columns, then added with IEEE operations
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            uint4 wa[TERMS], wb[TERMS];
            pa[i].split(wa);
            pb[i].split(wb);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const uint4 v = x[i][n];
                if (TERMS > 1) {
                    // an infinite or NaN x meets the first term only: the later ones may be 0 where the weight is not
                    const uint4 f = make_uint4(finite_bf16x2(v.x), finite_bf16x2(v.y), finite_bf16x2(v.z),
                                               finite_bf16x2(v.w));
#pragma unroll
                    for (int s = TERMS - 1; s >= 1; --s) {
                        mma_bf16(sum[n], wa[s].x, wb[s].x, wa[s].y, wb[s].y, f.x, f.y);
                        mma_bf16(sum[n], wa[s].z, wb[s].z, wa[s].w, wb[s].w, f.z, f.w);
                    }
                }
                mma_bf16(sum[n], wa[0].x, wb[0].x, wa[0].y, wb[0].y, v.x, v.y);
                mma_bf16(sum[n], wa[0].z, wb[0].z, wa[0].w, wb[0].w, v.z, v.w);
            }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c)
                acc[0][n][c] = __fadd_rn(acc[0][n][c], sum[n][c]);
    }
    keep<1, NT>(red[warp], acc);
    __syncthreads();
    for (int v = threadIdx.x; v < 16 * 8 * NT; v += kThreads) {
        const int r = v % 16, c = v / 16, at = side_index(0, r, NT, c);
        float s = red[0][at];
#pragma unroll
        for (int w = 1; w < kWarps; ++w)
            s = __fadd_rn(s, red[w][at]);
        if (e0 + r < a.E && t0 + c < a.T)
            a.sums[((int64_t)z * a.T + t0 + c) * a.E + e0 + r] = s;
    }
}

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }

// order-preserving map of floats to unsigned (-inf maps to 0x007fffff, +0 above -0)
__device__ __forceinline__ uint32_t ordered(float v)
{
    const uint32_t b = __float_as_uint(v);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float block_max(float v, float *s)
{
    for (int o = 16; o > 0; o >>= 1)
        v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
    if ((threadIdx.x & 31) == 0)
        s[threadIdx.x >> 5] = v;
    __syncthreads();
    v = s[0];
    for (int w = 1; w < kSelectThreads / 32; ++w)
        v = fmaxf(v, s[w]);
    return v;
}

__device__ __forceinline__ float block_sum(float v, float *s)
{
    for (int o = 16; o > 0; o >>= 1)
        v = __fadd_rn(v, __shfl_xor_sync(kFull, v, o));
    if ((threadIdx.x & 31) == 0)
        s[threadIdx.x >> 5] = v;
    __syncthreads();
    v = s[0];
    for (int w = 1; w < kSelectThreads / 32; ++w)
        v = __fadd_rn(v, s[w]);
    return v;
}

// One token.  A NaN logit counts as -inf and is never chosen, nor is a key of
// NaN or -inf; v == mx also where both are infinite, whose difference is NaN.
__global__ void __launch_bounds__(kSelectThreads)
router_select_kernel(Select a)
{
    extern __shared__ float dynamic[];   // [E] logits, [E] keys
    __shared__ float s_max[kSelectThreads / 32], s_sum[kSelectThreads / 32];
    float *l = dynamic, *key = dynamic + a.E;
    const int64_t t = blockIdx.x;
    grid_dependency_wait();
    allow_dependents();
    float mx = neg_inf();
    for (int e = threadIdx.x; e < a.E; e += kSelectThreads) {
        float v = a.sums[t * a.E + e];
        for (int z = 1; z < a.slices; z += kAtOnce) {
            float part[kAtOnce];
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i)
                part[i] = z + i < a.slices ? a.sums[((int64_t)(z + i) * a.T + t) * a.E + e] : 0.0f;
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i)
                if (z + i < a.slices)
                    v = __fadd_rn(v, part[i]);
        }
        if (a.logits != nullptr)
            a.logits[t * a.E + e] = v;
        l[e] = v;
        mx = fmaxf(mx, isnan(v) ? neg_inf() : v);
    }
    float sum = 1.0f;
    if (!a.sigmoid) {
        mx = block_max(mx, s_max);
        float part = 0.0f;
        for (int e = threadIdx.x; e < a.E; e += kSelectThreads) {
            const float v = isnan(l[e]) ? neg_inf() : l[e];
            part = __fadd_rn(part, v == mx ? 1.0f : expf(__fsub_rn(v, mx)));
        }
        sum = block_sum(part, s_sum);
    }
    auto score = [&](float v) {
        return a.sigmoid ? __fdiv_rn(1.0f, __fadd_rn(1.0f, expf(-v)))
                         : __fdiv_rn(v == mx ? 1.0f : expf(__fsub_rn(v, mx)), sum);
    };
    for (int e = threadIdx.x; e < a.E; e += kSelectThreads) {
        const float v = l[e];
        const float k = isnan(v) ? neg_inf() : a.bias != nullptr ? __fadd_rn(score(v), a.bias[e]) : v;
        key[e] = isnan(k) ? neg_inf() : __fadd_rn(k, 0.0f);   // -0 and +0 are one key
    }
    __syncthreads();
    if (threadIdx.x >= 32)
        return;
    const int lane = threadIdx.x;
    const uint32_t none = ordered(neg_inf());
    uint32_t best = none;   // this lane's best key and where it is
    int at = -1;
    auto scan = [&]() {
        best = none;
        at = -1;
        for (int e = lane; e < a.E; e += 32) {
            const uint32_t k = ordered(key[e]);
            if (k > best) {
                best = k;
                at = e;
            }
        }
    };
    scan();
    int mine_e = -1;   // lane k holds slot k
    for (int k = 0; k < a.K; ++k) {
        const uint32_t top = __reduce_max_sync(kFull, best);
        if (top == none)
            break;
        const int e = (int)__reduce_min_sync(kFull, best == top ? (uint32_t)at : 0xffffffffu);
        if (lane == k)
            mine_e = e;
        if (lane == (e & 31)) {
            key[e] = neg_inf();
            scan();
        }
        __syncwarp();
    }
    const float mine = mine_e >= 0 ? score(l[mine_e]) : 0.0f;
    float chosen = 0.0f;   // the scores are positive or +0: those of empty slots change nothing
    for (int k = 0; k < a.K; ++k)
        chosen = __fadd_rn(chosen, __shfl_sync(kFull, mine, k));
    if (lane < a.K) {
        float w = mine;
        if (a.renormalize)
            w = chosen > 0.0f ? __fdiv_rn(w, chosen) : 0.0f;
        a.idx[t * a.K + lane] = mine_e;
        a.weights[t * a.K + lane] = mine_e >= 0 ? __fmul_rn(w, a.scale) : 0.0f;
    }
}

// Blocks that fill the GPU once: a GB300's SMs.  A constant, so that the workspace has one size wherever it is asked.
constexpr int kBlocks = 152;

// As many slices of the columns as make that many blocks, at least a unit to a warp.
int slices_of(int64_t T, int H, int E)
{
    const int64_t blocks = ceil_div(E, 16) * ceil_div(T, T <= 8 ? 8 : 16);
    const int64_t most = std::max<int64_t>(1, ceil_div(H, kUnit * kWarps));
    return (int)std::max<int64_t>(1, std::min<int64_t>(most, kBlocks / std::max<int64_t>(1, blocks)));
}

template <int TERMS>
int launch_logits(const LogitsArgs &a, cudaStream_t stream)
{
    const unsigned experts = (unsigned)ceil_div(a.E, 16);
    if (a.T <= 8)
        return launch_dependent(router_logits_kernel<TERMS, 1>, dim3(1, experts, a.slices), kThreads, 0, stream, a);
    const dim3 grid((unsigned)ceil_div(a.T, 16), experts, a.slices);
    return launch_dependent(router_logits_kernel<TERMS, 2>, grid, kThreads, 0, stream, a);
}

int launch_logits(const void *x, int64_t T, int H, const void *w, int w_dtype, int E, int slices, float *sums,
                  cudaStream_t stream)
{
    const LogitsArgs a{static_cast<const uint8_t *>(x), static_cast<const uint8_t *>(w), (int)T, H, E, slices, sums};
    return w_dtype == 1 ? launch_logits<3>(a, stream) : launch_logits<1>(a, stream);
}

}  // namespace
}  // namespace ep

using namespace ep;

extern "C" size_t ep_router_workspace_size(int64_t T, int H, int E)
{
    if (T < 0 || H < 1 || E < 1)
        return 0;
    // slices_of(t) * t is at most this for every t <= T, so that a workspace serves smaller batches too
    const size_t most = (size_t)std::max<int64_t>(1, ceil_div(H, kUnit * kWarps)) * T;
    const size_t rows = std::min(most, std::max((size_t)T, (size_t)(kBlocks * 16 / ceil_div(E, 16))));
    return align_up(rows * E * sizeof(float), kWsAlign) + kWsAlign;
}

// Whether the call goes on: EP_OK with *done unset.
static int router_arguments(const void *x, int64_t T, int H, const void *w, int w_dtype, int E, int K, int scoring,
                            const int64_t *topk_idx, const float *topk_weights, const void *ws, size_t ws_bytes,
                            bool *done)
{
    if (T < 0 || H < 8 || H % 8 != 0 || E < 1 || E > EP_MAX_EXPERTS || K < 1 || K > EP_MAX_TOPK || K > E ||
        (scoring != EP_SCORE_SOFTMAX && scoring != EP_SCORE_SIGMOID))
        return EP_ERR_INVALID_ARG;
    if ((w_dtype != 0 && w_dtype != 1) || T > (1 << 20))
        return EP_ERR_UNSUPPORTED;
    if (T == 0) {
        *done = true;
        return EP_OK;
    }
    if (x == nullptr || w == nullptr || topk_idx == nullptr || topk_weights == nullptr || !aligned(x, 16) ||
        !aligned(w, 16) || ws == nullptr || !aligned(ws, kWsAlign) || ws_bytes < ep_router_workspace_size(T, H, E))
        return EP_ERR_INVALID_ARG;
    return EP_OK;
}

extern "C" int ep_router_topk(const void *x, int64_t T, int H, const void *w, int w_dtype, int E, const float *bias,
                              int K, int scoring, int renormalize, float scale, int64_t *topk_idx,
                              float *topk_weights, float *logits, void *ws, size_t ws_bytes, ep_stream_t stream_)
{
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    bool done = false;
    int rc = router_arguments(x, T, H, w, w_dtype, E, K, scoring, topk_idx, topk_weights, ws, ws_bytes, &done);
    if (rc != EP_OK || done)
        return rc;
    // for every E: the kernel's static part counts toward the 48 KB that need no raising
    static PerDevice set;
    rc = raise_smem(router_select_kernel, 2 * EP_MAX_EXPERTS * sizeof(float), set);
    if (rc != EP_OK)
        return rc;
    const int slices = slices_of(T, H, E);
    float *sums = static_cast<float *>(ws);
    rc = launch_logits(x, T, H, w, w_dtype, E, slices, sums, stream);
    if (rc != EP_OK)
        return rc;
    const Select s{sums, bias, (int)T, E, K, slices, scoring == EP_SCORE_SIGMOID, renormalize, scale, topk_idx,
                   topk_weights, logits};
    return launch_dependent(router_select_kernel, dim3((unsigned)T), kSelectThreads, 2 * (size_t)E * sizeof(float), stream,
                            s);
}

extern "C" int ep_router_topk_groups(const void *x, int64_t T, int H, const void *w, int w_dtype, int E,
                                     const float *bias, int K, int scoring, int num_groups, int topk_groups,
                                     int group_score, int renormalize, float scale, int64_t *topk_idx,
                                     float *topk_weights, float *logits, void *ws, size_t ws_bytes,
                                     ep_stream_t stream_)
{
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    int rc = choice_status(E, K, scoring, num_groups, topk_groups, group_score);
    if (rc != EP_OK)
        return rc;
    if (num_groups == 1)
        return ep_router_topk(x, T, H, w, w_dtype, E, bias, K, scoring, renormalize, scale, topk_idx, topk_weights,
                              logits, ws, ws_bytes, stream_);
    bool done = false;
    rc = router_arguments(x, T, H, w, w_dtype, E, K, scoring, topk_idx, topk_weights, ws, ws_bytes, &done);
    if (rc != EP_OK || done)
        return rc;
    const int slices = slices_of(T, H, E);
    float *sums = static_cast<float *>(ws);
    rc = launch_logits(x, T, H, w, w_dtype, E, slices, sums, stream);
    if (rc != EP_OK)
        return rc;
    const Choice c{sums, 0, slices, bias, (int)T, E, K, scoring == EP_SCORE_SIGMOID, num_groups, topk_groups,
                   group_score == EP_GROUP_TOP2, renormalize, scale, topk_idx, topk_weights, logits};
    return launch_choice(c, stream);
}
