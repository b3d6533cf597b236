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

// ------------------------------------------- up to 512 experts: a warp a token --
// Lanes share the groups out evenly: `per` lanes (a power of two) to a group, C
// neighbouring experts of it to a lane.  Keys are fp32 with a bound on what they
// are off by; the K largest are taken one at a time, the warp's best by one
// reduction.  Where two keys, or two marks, that decide something are nearer than
// their bounds allow, the few candidates are compared in 64 bits.
//
// The bounds, in units u = 2^-24 (ex2.approx 4u of its result, rcp.approx 2u):
//   sigmoid: an exponential off by 4u + 1.5 |l| u of itself moves the score by at
//     most (1 + 0.34) u, as s (1 - s) <= 1/4 and |l| s (1 - s) <= 0.23; 1 + e
//     and the reciprocal by 3u: below 8u in all.
//   softmax: exponentials of x = l - max off by (4 + 2.6 |x|) u of themselves; their sum by
//     (4 + 2.6 log E) u, as the mean of |x| is at most log E, and 21 u for its
//     additions: below 64 u of the score, and u as |x| e^-|x| <= 0.37.
//   the addition of the bias: u of the key.
constexpr float kU = 1.0f / (1 << 24);

__device__ __forceinline__ float exp2_quick(float v)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

__device__ __forceinline__ float reciprocal_quick(float v)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

constexpr float kLog2e = 1.44269504f;
constexpr float kLeastLog = -745.0f;   // logarithm of the least score that 64 bits tell from 0

// order-preserving map of floats to unsigned (-inf maps to kNone, +0 above -0)
__device__ __forceinline__ uint32_t ordered(float v)
{
    const uint32_t b = __float_as_uint(v);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float unordered(uint32_t v)
{
    return __uint_as_float(v & 0x80000000u ? v & 0x7fffffffu : ~v);
}

constexpr uint32_t kNone = 0x007fffffu;

__device__ __forceinline__ float warp_sum(float v)
{
    for (int o = 16; o > 0; o >>= 1)
        v = __fadd_rn(v, __shfl_xor_sync(kFull, v, o));
    return v;
}

__device__ __forceinline__ float warp_max(float v) { return unordered(__reduce_max_sync(kFull, ordered(v))); }

__device__ __forceinline__ float warp_min(float v) { return unordered(__reduce_min_sync(kFull, ordered(v))); }

__device__ __forceinline__ double warp_sum64(double v)
{
    for (int o = 16; o > 0; o >>= 1)
        v += shfl_xor64(v, o);
    return v;
}

// A token's 64-bit scores, for the comparisons that need them.
__device__ __noinline__ Score64 scores64(const Choice &c, int64_t t, float mx)
{
    Score64 s{c.sigmoid, (double)mx, 1.0};
    if (!c.sigmoid) {
        double part = 0.0;
        for (int e = threadIdx.x & 31; e < c.E; e += 32)
            part += s(logit_of(c, t, e));
        s.sum = warp_sum64(part);
    }
    return s;
}

__device__ __forceinline__ double key64(const Choice &c, const Score64 &score, float l, int e)
{
    const double k = isnan(l) ? neg_inf64() : c.bias != nullptr ? score(l) + (double)ld_float(c.bias + e) : (double)l;
    return isnan(k) ? neg_inf64() : k + 0.0;
}

// A lane's experts.
struct Share {
    int first, count;   // neighbours, of group `group`
    int group, per;     // lanes to a group
};

// Which groups stay, by marks in 64 bits: a bit for each group.
__device__ __noinline__ uint32_t groups64(const Choice &c, int64_t t, float mx, Share mine)
{
    const Score64 score = scores64(c, t, mx);
    const bool of_scores = c.top2 && c.bias == nullptr;
    double a = neg_inf64(), b = neg_inf64();
    for (int i = 0; i < mine.count; ++i) {
        const float l = logit_of(c, t, mine.first + i);
        double k = key64(c, score, l, mine.first + i);
        if (k != neg_inf64() && of_scores)
            k = score(l);
        b = fmax(b, fmin(a, k));
        a = fmax(a, k);
    }
    for (int o = 1; o < mine.per; o *= 2) {
        const double a2 = shfl_xor64(a, o), b2 = shfl_xor64(b, o);
        b = fmax(fmin(a, a2), fmax(b, b2));
        a = fmax(a, a2);
    }
    const double mark = c.top2 && b != neg_inf64() ? a + b : a;
    int ahead = 0;
    for (int o = 0; o < c.groups; ++o) {
        const double m = __shfl_sync(kFull, mark, o * mine.per);
        ahead += m > mark || (m == mark && o < mine.group);
    }
    const bool stays = mine.group < c.groups && ahead < c.kept;
    return __reduce_or_sync(kFull, stays ? 1u << mine.group : 0u);
}

// The K largest of the candidates (bit i of `mask`: this lane's expert first + i) by keys in 64 bits; lane k gets the
// k-th, or -1.
__device__ __noinline__ int choose64(const Choice &c, int64_t t, float mx, Share mine, uint32_t mask)
{
    const int lane = threadIdx.x & 31;
    const Score64 score = scores64(c, t, mx);
    int chosen = -1;
    int before = 0, all = 0;   // candidates in the lanes before this one, and in all
    for (int o = 0; o < 32; ++o) {
        const int n = __popc(__shfl_sync(kFull, mask, o));
        before += o < lane ? n : 0;
        all += n;
    }
    if (all <= 32) {   // one to a lane, ranked
        int e = -1;
        for (int o = 0; o < 32; ++o) {
            const uint32_t m = __shfl_sync(kFull, mask, o);
            const int b = __shfl_sync(kFull, before, o), f = __shfl_sync(kFull, mine.first, o);
            if (lane >= b && lane < b + __popc(m)) {
                uint32_t left = m;
                for (int skip = lane - b; skip > 0; --skip)
                    left &= left - 1u;
                e = f + __ffs(left) - 1;
            }
        }
        const double k = e >= 0 ? key64(c, score, logit_of(c, t, e), e) : neg_inf64();
        int ahead = 0;
        for (int o = 0; o < all; ++o) {
            const double u = __shfl_sync(kFull, k, o);
            const int f = __shfl_sync(kFull, e, o);
            ahead += u > k || (u == k && f < e);
        }
        for (int o = 0; o < all; ++o) {
            const int place = __shfl_sync(kFull, ahead, o), f = __shfl_sync(kFull, e, o);
            if (place == lane && place < c.K)
                chosen = f;
        }
        return chosen;
    }
    for (int k = 0; k < c.K; ++k) {
        double top = neg_inf64();
        int at = -1;
        for (int i = 0; i < mine.count; ++i)
            if (mask >> i & 1u) {
                const double u = key64(c, score, logit_of(c, t, mine.first + i), mine.first + i);
                if (u > top) {
                    top = u;
                    at = mine.first + i;
                }
            }
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
        if (e == at)
            mask &= ~(1u << (e - mine.first));
        if (lane == k)
            chosen = e;
    }
    return chosen;
}

template <int C>
__global__ void __launch_bounds__(kThreads)
select_warp_kernel(const __grid_constant__ Choice c, int per, int wide)
{
    const int lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    grid_dependency_wait();
    allow_dependents();
    if (t >= c.T)
        return;
    const int size = c.E / c.groups, group = lane / per, in_group = (lane % per) * C;
    const int count = group < c.groups ? max(0, min(C, size - in_group)) : 0;
    const Share mine{group * size + in_group, count, group, per};

    float l[C];
    if (C % 4 == 0 && wide) {   // fours of experts, whole
#pragma unroll
        for (int i = 0; i < C; i += 4) {
            if (C % 4 != 0)
                break;
            if (i < count) {
                const int64_t at = t * c.E + mine.first + i;
                if (c.dtype == 0) {
                    const uint4 v = ld_global(reinterpret_cast<const uint4 *>(static_cast<const float *>(c.logits) + at));
                    l[i] = __uint_as_float(v.x);
                    l[(i + 1) % C] = __uint_as_float(v.y);
                    l[(i + 2) % C] = __uint_as_float(v.z);
                    l[(i + 3) % C] = __uint_as_float(v.w);
                } else {
                    const uint2 v = ld_global(reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(c.logits) + at));
                    l[i] = bf16_lo(v.x);
                    l[(i + 1) % C] = bf16_hi(v.x);
                    l[(i + 2) % C] = bf16_lo(v.y);
                    l[(i + 3) % C] = bf16_hi(v.y);
                }
            } else {
                l[i] = l[(i + 1) % C] = l[(i + 2) % C] = l[(i + 3) % C] = neg_inf();
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < C; ++i)
            l[i] = i < count ? logit_of(c, t, mine.first + i) : neg_inf();
    }
    if (c.sums != nullptr)
#pragma unroll
        for (int i = 0; i < C; ++i)
            if (i < count)
                c.sums[t * c.E + mine.first + i] = l[i];

    const bool marks_of_scores = c.groups > 1 && c.top2 && c.bias == nullptr;
    const bool scored = c.bias != nullptr || marks_of_scores;   // something compared is made of scores
    float mx = 0.0f, sum = 1.0f, off = 8 * kU;   // off: of a score
    if (!c.sigmoid) {
        mx = neg_inf();
#pragma unroll
        for (int i = 0; i < C; ++i)
            mx = fmaxf(mx, l[i]);
        mx = warp_max(mx);
        if (scored || !c.renormalize) {
            float part = 0.0f;
#pragma unroll
            for (int i = 0; i < C; ++i) {
                const float p = l[i] == mx ? 1.0f : exp2_quick(__fmul_rn(__fsub_rn(l[i], mx), kLog2e));
                part = __fadd_rn(part, i < count && !isnan(l[i]) ? p : 0.0f);
            }
            sum = warp_sum(part);
            off = __fadd_rn(__fmul_rn(64 * kU, __fdividef(1.0f, sum)), kU);
        }
    }
    auto score = [&](float v) {
        if (c.sigmoid)
            return reciprocal_quick(__fadd_rn(1.0f, exp2_quick(__fmul_rn(v, -kLog2e))));
        return __fmul_rn(v == mx ? 1.0f : exp2_quick(__fmul_rn(__fsub_rn(v, mx), kLog2e)), reciprocal_quick(sum));
    };
    uint32_t key[C];
    float s[C];
#pragma unroll
    for (int i = 0; i < C; ++i) {
        s[i] = scored ? score(l[i]) : 0.0f;
        float k = l[i];
        if (c.bias != nullptr && i < count)
            k = isnan(k) ? k : __fadd_rn(s[i], ld_float(c.bias + mine.first + i));
        key[i] = isnan(k) || i >= count ? kNone : ordered(__fadd_rn(k, 0.0f));
    }

    if (c.groups > 1) {
        float a = neg_inf(), b = neg_inf();
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const float k = marks_of_scores && key[i] != kNone ? s[i] : unordered(key[i]);
            b = fmaxf(b, fminf(a, k));
            a = fmaxf(a, k);
        }
        for (int o = 1; o < per; o *= 2) {
            const float a2 = __shfl_xor_sync(kFull, a, o), b2 = __shfl_xor_sync(kFull, b, o);
            b = fmaxf(fminf(a, a2), fmaxf(b, b2));
            a = fmaxf(a, a2);
        }
        const bool both = c.top2 && b != neg_inf();
        const float mark = both ? __fadd_rn(a, b) : a;
        int ahead = 0;
        for (int o = 0; o < c.groups; ++o) {
            const float m = __shfl_sync(kFull, mark, o * per);
            ahead += m > mark || (m == mark && o < group);
        }
        bool stays = group < c.groups && ahead < c.kept;
        if (scored && c.kept < c.groups) {
            const float wrong = __fadd_rn(both ? 2 * off : off, __fmul_rn(2 * kU, __fadd_rn(fabsf(a), both ? fabsf(b) : 0.0f)));
            const float inf = -neg_inf();   // infinite marks are what they are
            // the least that a group which stays may have, the most of one that goes
            const float least = warp_min(stays && fabsf(mark) < inf ? __fsub_rn(mark, wrong) : inf);
            const float most = warp_max(!stays && group < c.groups && mark > neg_inf() ? __fadd_rn(mark, wrong) : neg_inf());
            if (most >= least)
                stays = groups64(c, t, mx, mine) >> group & 1u;
        }
        if (!stays)
#pragma unroll
            for (int i = 0; i < C; ++i)
                key[i] = kNone;
    }

    uint32_t best = kNone;   // this lane's best key and where it is
    int at = 0;
    auto scan = [&]() {
        best = kNone;
#pragma unroll
        for (int i = 0; i < C; ++i)
            if (key[i] > best) {
                best = key[i];
                at = i;
            }
    };
    scan();
    uint32_t taken = 0, mine_key = kNone;   // of this lane's experts; lane k holds slot k
    int mine_e = -1;
    for (int k = 0; k < c.K; ++k) {
        const uint32_t top = __reduce_max_sync(kFull, best);
        if (top == kNone)
            break;
        const int owner = __ffs(__ballot_sync(kFull, best == top)) - 1;
        const int e = __shfl_sync(kFull, mine.first + at, owner);
        if (lane == k) {
            mine_e = e;
            mine_key = top;
        }
        if (lane == owner) {
            taken |= 1u << at;
#pragma unroll
            for (int i = 0; i < C; ++i)
                if (i == at)
                    key[i] = kNone;
            scan();
        }
    }
    float mine_l = mine_e >= 0 ? logit_of(c, t, mine_e) : neg_inf();
    if (c.bias != nullptr) {
        // neighbours in the order that 32 bits give, unless they are the same score and bias
        auto wrong = [&](float k) { return __fadd_rn(off, __fmul_rn(2 * kU, fabsf(k))); };
        const float mine_b = mine_e >= 0 ? ld_float(c.bias + mine_e) : 0.0f;
        const int chosen = __popc(__ballot_sync(kFull, mine_e >= 0));
        const float k = unordered(mine_key), next = __shfl_down_sync(kFull, k, 1);
        const float next_l = __shfl_down_sync(kFull, mine_l, 1), next_b = __shfl_down_sync(kFull, mine_b, 1);
        bool near = lane + 1 < chosen && __fadd_rn(next, wrong(next)) >= __fsub_rn(k, wrong(k)) &&
                    !(mine_l == next_l && mine_b == next_b);
        // those left, against the last chosen
        const int end = max(chosen - 1, 0);
        const float last = __shfl_sync(kFull, k, end), least = __fsub_rn(last, wrong(last));
        const float last_l = __shfl_sync(kFull, mine_l, end), last_b = __shfl_sync(kFull, mine_b, end);
        const float rest = unordered(best);
        if (best != kNone && chosen > 0 && __fadd_rn(rest, wrong(rest)) >= least)
#pragma unroll
            for (int i = 0; i < C; ++i) {
                const float u = unordered(key[i]);
                if (key[i] != kNone && __fadd_rn(u, wrong(u)) >= least &&
                    !(l[i] == last_l && ld_float(c.bias + mine.first + i) == last_b))
                    near = true;
            }
        if (__any_sync(kFull, near)) {
            uint32_t mask = taken;
#pragma unroll
            for (int i = 0; i < C; ++i) {
                const float u = unordered(key[i]);
                if (key[i] != kNone && __fadd_rn(u, wrong(u)) >= least)
                    mask |= 1u << i;
            }
            mine_e = choose64(c, t, mx, mine, mask);
            mine_l = mine_e >= 0 ? logit_of(c, t, mine_e) : neg_inf();
        }
    }
    // the weights: shares of the chosen ones' sum from a multiple of the scores that does not vanish
    float w = 0.0f;
    if (c.renormalize) {
        const float top = warp_max(mine_l);
        if (c.sigmoid) {
            const float x = expf(-fabsf(mine_l));
            if (mine_l >= kLeastLog)
                w = __fdiv_rn(mine_l >= 0.0f ? 1.0f : expf(__fsub_rn(mine_l, fminf(top, 0.0f))), __fadd_rn(1.0f, x));
        } else if (mine_e >= 0) {
            w = mine_l == mx || (mine_l == top && __fsub_rn(top, mx) >= kLeastLog) ? 1.0f
                : __fsub_rn(mine_l, mx) >= kLeastLog ? expf(__fsub_rn(mine_l, top)) : 0.0f;
        }
        const float all = warp_sum(w);
        w = all > 0.0f ? __fdiv_rn(w, all) : 0.0f;
    } else if (mine_e >= 0) {
        const float x = expf(-fabsf(mine_l));
        w = c.sigmoid ? __fdiv_rn(mine_l >= 0.0f ? 1.0f : x, __fadd_rn(1.0f, x))
                      : __fdiv_rn(mine_l == mx ? 1.0f : expf(__fsub_rn(mine_l, mx)), sum);
    }
    if (lane < c.K) {
        c.idx[t * c.K + lane] = mine_e;
        c.weights[t * c.K + lane] = mine_e >= 0 ? __fmul_rn(w, c.scale) : 0.0f;
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
        s = l < kLeastLog ? 0.0f : l >= 0.0f ? d : b.renormalize && mx < 0.0f ? __fmul_rn(expf(__fsub_rn(l, mx)), d) : m;
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
    int per = 32;   // lanes to a group
    while (per > 1 && per * c.groups > 32)
        per /= 2;
    const int size = c.E / c.groups, share = (int)ceil_div(size, per);
    if (per * c.groups <= 32 && share <= 16) {
        const dim3 grid((unsigned)ceil_div(c.T, kWarps));
        const int wide = c.slices == 1 && size % 4 == 0 && aligned(c.logits, c.dtype == 0 ? 16 : 8);
        if (share <= 1)
            return launch_dependent(select_warp_kernel<1>, grid, kThreads, 0, stream, c, per, wide);
        if (share <= 2)
            return launch_dependent(select_warp_kernel<2>, grid, kThreads, 0, stream, c, per, wide);
        if (share <= 4)
            return launch_dependent(select_warp_kernel<4>, grid, kThreads, 0, stream, c, per, wide);
        if (share <= 8)
            return launch_dependent(select_warp_kernel<8>, grid, kThreads, 0, stream, c, per, wide);
        return launch_dependent(select_warp_kernel<16>, grid, kThreads, 0, stream, c, per, wide);
    }
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
