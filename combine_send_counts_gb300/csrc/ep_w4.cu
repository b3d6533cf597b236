// 4-bit weights with group scales: quantise, read back, and the product with a
// few rows of x.
//
//   w[n,k] = (q[n,k] - zero[n,g]) * scale[n,g],  g = k / group
#include <algorithm>

#include "ep_device.cuh"
#include "ep_internal.h"
#include "ep_launch.cuh"
#include "ep_skinny.cuh"

namespace ep {
namespace {

constexpr int kThreads = 256;

// ----------------------------------------------------- quantise, read back --
// Both are bound by HBM (2.5 bytes a weight and the scales); what matters is
// that the arithmetic between stays under it.  A lane holds 8 consecutive
// weights of kVectors groups; G/8 neighbouring lanes share a group and find its
// extremes with shuffles of bf16 pairs.  98304x4096 in groups of 128: 172 us to
// codes and 163 back, 5.9 and 6.2 TB/s (0.87 and 0.92 of what a copy reaches); as
// fp32 334 us, 5.4 TB/s.
constexpr int kVectors = 4;
constexpr int64_t kMostVectors = (((int64_t)1 << 31) - 1) * kThreads * kVectors;   // of a grid

__device__ __forceinline__ uint32_t min_bf16x2(uint32_t a, uint32_t b)   // NaN if either is
{
    uint32_t d;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// 1.5 * 2^23: adding it leaves the nearest integer (ties to even) of a small number in the low mantissa bits.
constexpr float kRound = 12582912.0f;
constexpr uint32_t kRoundBits = 0x4b400000u;

// rint(w / s) + kRound of two weights.  With rs the correctly rounded 1/s, q0 = w * rs and the exact remainder r =
// w - q0 * s, q0 + r * rs rounds to the correctly rounded quotient (Markstein, 1990), so that ties are exact and go
// to even.  Two per instruction.
__device__ __forceinline__ float2 round_quotients(float2 w, float s, float rs)
{
    const float2 rs2 = make_float2(rs, rs);
    const float2 q0 = mul2_rn(w, rs2);
    const float2 r = fma2_rn(q0, make_float2(-s, -s), w);
    const float2 q = fma2_rn(r, rs2, q0);
    return fma2_rn(q, make_float2(1.0f, 1.0f), make_float2(kRound, kRound));
}

// a group's scale, its reciprocal (0: the codes take the slow way) and its zero point
struct GroupScale {
    float s, rs, z;
};

template <bool ZERO>
__device__ __forceinline__ GroupScale group_scale(float least, float most)   // NaN where the group holds one
{
    const bool finite = isfinite(least) && isfinite(most);
    const float lo = fminf(least, 0.0f), hi = fmaxf(most, 0.0f);
    const float wide = ZERO ? __fsub_rn(__fdiv_rn(hi, 15.0f), __fdiv_rn(lo, 15.0f)) : __fdiv_rn(fmaxf(hi, -lo), 7.0f);
    GroupScale g;
    g.s = __bfloat162float(__float2bfloat16_rn(finite ? wide : __int_as_float(0x7f800000)));
    const bool plain = finite && g.s > 0.0f;
    g.z = ZERO ? (plain ? fminf(fmaxf(rintf(__fdiv_rn(-lo, g.s)), 0.0f), 15.0f) : 0.0f) : 8.0f;
    // where nothing above over- or underflows
    g.rs = finite && g.s >= 7.9e-31f && g.s <= 1.2e30f ? __fdiv_rn(1.0f, g.s) : 0.0f;
    return g;
}

template <int G, bool ZERO>
__global__ void __launch_bounds__(kThreads)
w4_quantize_kernel(const uint4 *w, int64_t vectors, uint32_t *q, __nv_bfloat16 *scale, uint8_t *zero)
{
    constexpr int kLanes = G / 8;
    static_assert(kVectors == 4 && kLanes % kVectors == 0, "a lane of each group for each of a lane's groups");
    const int64_t first = (int64_t)blockIdx.x * (kThreads * kVectors) + threadIdx.x;
    const int lane = threadIdx.x & 31;
    grid_dependency_wait();
    allow_dependents();
    uint4 v[kVectors];
#pragma unroll
    for (int i = 0; i < kVectors; ++i) {
        v[i] = make_uint4(0, 0, 0, 0);
        if (first + i * kThreads < vectors)   // a group's lanes are in or out together
            v[i] = ld_global_stream(w + first + i * kThreads);
    }
    uint32_t lo2[kVectors], hi2[kVectors];
#pragma unroll
    for (int i = 0; i < kVectors; ++i) {
        lo2[i] = min_bf16x2(min_bf16x2(v[i].x, v[i].y), min_bf16x2(v[i].z, v[i].w));
        hi2[i] = max_bf16x2(max_bf16x2(v[i].x, v[i].y), max_bf16x2(v[i].z, v[i].w));
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) {
            lo2[i] = min_bf16x2(lo2[i], __shfl_xor_sync(kFull, lo2[i], o));
            hi2[i] = max_bf16x2(hi2[i], __shfl_xor_sync(kFull, hi2[i], o));
        }
    }
    // the divisions: lane i of each four for the lane's i-th group
    const int mine = lane & 3;
    uint32_t l2 = mine & 2 ? (mine & 1 ? lo2[3] : lo2[2]) : (mine & 1 ? lo2[1] : lo2[0]);
    uint32_t h2 = mine & 2 ? (mine & 1 ? hi2[3] : hi2[2]) : (mine & 1 ? hi2[1] : hi2[0]);
    l2 = min_bf16x2(l2, __byte_perm(l2, l2, 0x1032));
    h2 = max_bf16x2(h2, __byte_perm(h2, h2, 0x1032));
    const GroupScale own = group_scale<ZERO>(bf16_lo(l2), bf16_lo(h2));
#pragma unroll
    for (int i = 0; i < kVectors; ++i) {
        const int from = (lane & 28) | i;
        GroupScale g;
        g.s = __shfl_sync(kFull, own.s, from);
        g.rs = __shfl_sync(kFull, own.rs, from);
        g.z = ZERO ? __shfl_sync(kFull, own.z, from) : 8.0f;
        const int64_t at = first + i * kThreads;
        if (at >= vectors)
            continue;
        if (threadIdx.x % kLanes == 0) {
            scale[at / kLanes] = __float2bfloat16_rn(g.s);
            if (ZERO)
                zero[at / kLanes] = (uint8_t)g.z;
        }
        const uint32_t p[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
        uint32_t out = 0;
        if (g.rs != 0.0f) {
            // codes as integers added to kRoundBits; only zero points can push one out of range (|w| / s <= 7.03)
            const float least = kRound - g.z, most = kRound + 15.0f - g.z;
#pragma unroll
            for (int j = 3; j >= 0; --j) {
                float2 t = round_quotients(make_float2(bf16_lo(p[j]), bf16_hi(p[j])), g.s, g.rs);
                if (ZERO)
                    t = make_float2(fminf(fmaxf(t.x, least), most), fminf(fmaxf(t.y, least), most));
                out = out * 16 + __float_as_uint(t.y);
                out = out * 16 + __float_as_uint(t.x);
            }
            // sum of (kRoundBits - z) * 16^j modulo 2^32; kRoundBits ends in 22 zeros
            out += (uint32_t)(int)g.z * 0x11111111u - kRoundBits * 0x11111111u;
        } else {   // no scale, or one out of the range of the above
            const bool plain = g.s > 0.0f && g.s < __int_as_float(0x7f800000);
#pragma unroll
            for (int j = 7; j >= 0; --j) {
                const float x = j & 1 ? bf16_hi(p[j >> 1]) : bf16_lo(p[j >> 1]);
                const float r = plain ? fminf(fmaxf(rintf(__fdiv_rn(x, g.s)), -64.0f), 64.0f) : 0.0f;
                out = out << 4 | (uint32_t)fminf(fmaxf(__fadd_rn(r, g.z), 0.0f), 15.0f);
            }
        }
        q[at] = out;
    }
}

template <int G, bool F32>
__global__ void __launch_bounds__(kThreads)
w4_dequantize_kernel(const uint32_t *q, const uint16_t *scale, const uint8_t *zero, int64_t vectors, void *out)
{
    const int64_t first = (int64_t)blockIdx.x * (kThreads * kVectors) + threadIdx.x;
    grid_dependency_wait();
    allow_dependents();
    uint32_t v[kVectors], zz[kVectors];
    float s[kVectors];
#pragma unroll
    for (int i = 0; i < kVectors; ++i) {
        const int64_t at = first + i * kThreads;
        if (at < vectors) {
            v[i] = ld_global(q + at);
            s[i] = __uint_as_float((uint32_t)ld_global(scale + at / (G / 8)) << 16);
            zz[i] = (0x4300u | (zero != nullptr ? ld_global(zero + at / (G / 8)) : 8u)) * 0x10001u;
        }
    }
#pragma unroll
    for (int i = 0; i < kVectors; ++i) {
        const int64_t at = first + i * kThreads;
        if (at >= vectors)
            return;
        float f[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {   // codes j and j + 4 as bf16 integers, less the zero point: exact
            const uint32_t c = sub_bf16x2(((v[i] >> (4 * j)) & 0x000f000fu) | kMagic, zz[i]);
            const float2 p = mul2_rn(make_float2(bf16_lo(c), bf16_hi(c)), make_float2(s[i], s[i]));
            f[j] = p.x;
            f[j + 4] = p.y;
        }
        if (F32) {
            float4 *o = static_cast<float4 *>(out) + 2 * at;
            o[0] = make_float4(f[0], f[1], f[2], f[3]);
            o[1] = make_float4(f[4], f[5], f[6], f[7]);
        } else {
            st_stream(static_cast<uint4 *>(out) + at, make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                                                 pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7])));
        }
    }
}

template <int G>
int quantize(const void *w, int64_t vectors, unsigned blocks, uint8_t *q, void *scale, uint8_t *zero,
             cudaStream_t stream)
{
    const auto *src = static_cast<const uint4 *>(w);
    auto *dst = reinterpret_cast<uint32_t *>(q);
    auto *s = static_cast<__nv_bfloat16 *>(scale);
    if (zero != nullptr)
        return launch_dependent(w4_quantize_kernel<G, true>, blocks, kThreads, 0, stream, src, vectors, dst, s, zero);
    return launch_dependent(w4_quantize_kernel<G, false>, blocks, kThreads, 0, stream, src, vectors, dst, s, zero);
}

template <int G>
int dequantize(const uint8_t *q, const void *scale, const uint8_t *zero, int64_t vectors, unsigned blocks, void *w,
               int out_dtype, cudaStream_t stream)
{
    const auto *src = reinterpret_cast<const uint32_t *>(q);
    const auto *s = static_cast<const uint16_t *>(scale);
    if (out_dtype == 1)
        return launch_dependent(w4_dequantize_kernel<G, true>, blocks, kThreads, 0, stream, src, s, zero, vectors, w);
    return launch_dependent(w4_dequantize_kernel<G, false>, blocks, kThreads, 0, stream, src, s, zero, vectors, w);
}

// ------------------------------------------------------------------ product --
// y[m,n]: each block owns an equal share of the rows of w, in groups of up to
// 16*RB, which its warps share evenly (ep_skinny.cuh); the passes over a group
// of rows (16 rows of x each, up to four of them in one block) follow one
// another.  (Running them side by side in different warps, which would find the
// codes in L2, changed nothing: the arithmetic on the codes takes the time.)
//
// Measured: one row with 50021x7168 in groups of 128, 42.1 us, 4.4 TB/s (0.65 of
// what a copy reaches); 16 rows 59 us, 64 rows 208 us; 24 rows with 7168x4096 in
// groups of 32, 16.5 us; one row with 2048x2048, 3.3 us, which is the launch,
// one trip to HBM and the join.
struct MatvecArgs {
    const uint8_t *x;
    int M, N, K;
    int each, rest;    // rows of a block; the first `rest` blocks have one more
    Weights w;
    void *y;
    int out_f32;
};

constexpr int kMaxPasses = 4;

template <int G, int RB>
struct MatvecItems {
    using F = FormatW4<G, false>;
    static constexpr int kStep = 16;
    const MatvecArgs &a;
    int row0, row1, m0, passes;
    float *side, *open;    // this warp's kept pieces: of an item begun by another, and of one it began

    __device__ __forceinline__ int group(int item) const { return passes == 1 ? item : quick_div(item, passes); }
    __device__ __forceinline__ int row(int item) const { return row0 + group(item) * (16 * RB); }
    __device__ __forceinline__ int col(int item) const { return m0 + (item - group(item) * passes) * kMaxCols; }

    __device__ __forceinline__ RowRange rows(int item) const
    {
        const int r = row(item), n = min(row1 - r, 16 * RB);
        return RowRange{r, r + 8, n, n - 8};
    }

    __device__ __forceinline__ int cols(int item) const { return min(a.M - col(item), kMaxCols); }

    template <int NT>
    __device__ __forceinline__ void columns(int item, Columns<NT, 1> &x) const
    {
        x.plane_bytes = 0;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int m = col(item) + nt * 8 + ((threadIdx.x & 31) >> 2);
            x.set(nt, m < a.M ? a.x + (int64_t)m * a.K * 2 : nullptr, a.K);
        }
    }

    __device__ __forceinline__ void store(int m, int n, float v) const
    {
        if (m < a.M && n < row1) {
            if (a.out_f32)
                static_cast<float *>(a.y)[(int64_t)m * a.N + n] = v;
            else
                static_cast<__nv_bfloat16 *>(a.y)[(int64_t)m * a.N + n] = __float2bfloat16_rn(v);
        }
    }

    template <int NT>
    __device__ __forceinline__ void done(int item, bool first, bool last, const float (&acc)[RB][NT][4]) const
    {
        if (!first || !last) {
            keep<RB, NT>(first ? open : side, acc);
            return;
        }
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
        const int n = row(item) + g, m = col(item) + 2 * t;
#pragma unroll
        for (int r = 0; r < RB; ++r)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    store(m + nt * 8 + (c & 1), n + r * 16 + (c >> 1) * 8, acc[r][nt][c]);
    }
};

template <int G, int RB>
__global__ void __launch_bounds__(32 * FormatW4<G, false>::kWarps, 1)
w4_matvec_kernel(MatvecArgs a)
{
    extern __shared__ __align__(128) uint8_t dynamic[];   // ring, then one side block per warp
    using F = FormatW4<G, false>;
    __shared__ int begins[F::kWarps + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint8_t *sides = dynamic + Room<F, RB>::kRing;
    MatvecItems<G, RB> items{a};
    items.row0 = a.each * blockIdx.x + min((int)blockIdx.x, a.rest);
    items.row1 = items.row0 + a.each + ((int)blockIdx.x < a.rest ? 1 : 0);
    items.m0 = blockIdx.y * (kMaxPasses * kMaxCols);
    items.passes = min((a.M - items.m0 + kMaxCols - 1) / kMaxCols, kMaxPasses);
    items.side = reinterpret_cast<float *>(sides + warp * Room<F, RB>::kSide);
    items.open = reinterpret_cast<float *>(dynamic + warp * Room<F, RB>::kWarpRing);   // the ring is idle by then
    const int n = (items.row1 - items.row0 + 16 * RB - 1) / (16 * RB) * items.passes;
    Stream<F, RB, 1, MatvecItems<G, RB>> stream(items, a.w, a.K, n, smem_u32(dynamic));
    grid_dependency_wait();
    allow_dependents();
    stream.start();
    stream.run();
    stream.meet(begins);
    const int item = stream.open_item;
    if (item >= 0) {
        if (items.cols(item) <= 8) {
            float acc[RB][1][4];
            stream.template join<1>(dynamic, acc);
            items.template done<1>(item, true, true, acc);
        } else {
            float acc[RB][2][4];
            stream.template join<2>(dynamic, acc);
            items.template done<2>(item, true, true, acc);
        }
    }
}

template <int G, int RB>
int launch_matvec(const MatvecArgs &a, int blocks, dim3 grid, cudaStream_t stream)
{
    if constexpr (RB > 1) {
        if (blocks < RB)
            return launch_matvec<G, RB - 1>(a, blocks, grid, stream);
    }
    using F = FormatW4<G, false>;
    static PerDevice set;
    const int rc = raise_smem(w4_matvec_kernel<G, RB>, Room<F, RB>::kFixed, set);
    if (rc != EP_OK)
        return rc;
    return launch_dependent(w4_matvec_kernel<G, RB>, grid, 32 * F::kWarps, Room<F, RB>::kFixed, stream, a);
}

template <int G>
int matvec(MatvecArgs a, cudaStream_t stream)
{
    constexpr int kMost = FormatW4<G, false>::kMaxBlocks;
    const int sms = std::min(device_sm_count(), a.N);
    a.each = a.N / sms;
    a.rest = a.N % sms;
    const dim3 grid(sms, (unsigned)ceil_div(a.M, kMaxPasses * kMaxCols));
    return launch_matvec<G, kMost>(a, blocks_at_once(ceil_div(ceil_div(a.N, sms), 16), kMost, true), grid, stream);
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
    if (N > kMostVectors / (K / 8))
        return EP_ERR_UNSUPPORTED;
    const int64_t vectors = N * (K / 8), blocks = ceil_div(vectors, kThreads * kVectors);
    switch (group) {
    case 32: return quantize<32>(w, vectors, (unsigned)blocks, q, scale, zero, stream);
    case 64: return quantize<64>(w, vectors, (unsigned)blocks, q, scale, zero, stream);
    default: return quantize<128>(w, vectors, (unsigned)blocks, q, scale, zero, stream);
    }
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
    if (N > kMostVectors / (K / 8))
        return EP_ERR_UNSUPPORTED;
    const int64_t vectors = N * (K / 8), blocks = ceil_div(vectors, kThreads * kVectors);
    switch (group) {
    case 32: return dequantize<32>(q, scale, zero, vectors, (unsigned)blocks, w, out_dtype, stream);
    case 64: return dequantize<64>(q, scale, zero, vectors, (unsigned)blocks, w, out_dtype, stream);
    default: return dequantize<128>(q, scale, zero, vectors, (unsigned)blocks, w, out_dtype, stream);
    }
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
    // rows are counted in 32 bits, and the last of a block's row blocks counts on past N before it is masked
    constexpr int64_t kMostRows = ((int64_t)1 << 31) - 16 * FormatW4<32, false>::kMaxBlocks;
    if (M >= ((int64_t)1 << 20) || N > kMostRows || K >= ((int64_t)1 << 25))
        return EP_ERR_UNSUPPORTED;
    // a block's units of work are counted in 32 bits
    const int64_t units = ceil_div(N, (int64_t)16 * device_sm_count()) * kMaxPasses * ceil_div(K, 256);
    if (units >= ((int64_t)1 << 28))
        return EP_ERR_UNSUPPORTED;
    const MatvecArgs a{static_cast<const uint8_t *>(x), (int)M, (int)N, (int)K, 0, 0,
                       Weights{q, static_cast<const uint16_t *>(scale), zero, kMagic}, y, out_dtype};
    switch (group) {
    case 32: return matvec<32>(a, stream);
    case 64: return matvec<64>(a, stream);
    default: return matvec<128>(a, stream);
    }
}
