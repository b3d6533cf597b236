// Low-rank adapters of many requests beside a shared projection:
//
//   out[m] = base[m] + s[a] * B[a] (A[a] x[m]),  a = the adapter of row m.
//
// Two kernels, the second launched while the first drains: `shrink` leaves
// v = A x in parts of K in the workspace, `expand` adds the parts, multiplies by
// B and adds to the base.  Both take 16 rows of x as the 16-row operand of
// m16n8k16 matrix steps, ranks or output columns as its 8 columns.
//
//   few rows (up to 1024): a tile is up to 16 rows of the batch that name the same
//   adapter, found by the block from the ids, so that each adapter's weights are
//   read once for 16 rows wherever they stand;
//   more rows: a tile is 16 neighbouring rows, gone over once for each adapter that
//   they name, which is one where requests are long.
//
// v is kept whole between the two products, as the sum of three bf16 terms (24
// bits), because the matrix step takes bf16.
#include <algorithm>
#include <type_traits>

#include "ep_device.cuh"
#include "ep_internal.h"
#include "ep_launch.cuh"
#include "ep_skinny.cuh"

namespace ep {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kUnit = 32;            // columns of a lane's 16-byte pieces: two k16 steps
constexpr int kBatch = 4;            // units loaded together, and summed by matrix steps alone
constexpr int kTile = 16;
constexpr int kGatherRows = 1024;
constexpr int kMaxRank = 128;
constexpr int kMaxSplits = 16;
constexpr int kBlocks = 2 * 152;     // that fill the GPU
constexpr int kPlanes = 3;

struct Lora {
    const uint8_t *x, *a, *b;
    const int64_t *ids;
    const float *scaling;
    const void *base;
    void *out;
    int64_t M;
    int K, N, R, L, splits, base_dtype, out_dtype;
    float *parts;                    // [splits][M][R]
    int32_t *err;
};

// The adapter of a row, or -1.
__device__ __forceinline__ int adapter_of(const Lora &p, int64_t m)
{
    const uint2 w = ld_global(reinterpret_cast<const uint2 *>(p.ids) + m);
    const int64_t id = (int64_t)((uint64_t)w.y << 32 | w.x);
    return id >= 0 && id < p.L ? (int)id : -1;
}

__device__ __forceinline__ bool bad_id(const Lora &p, int64_t m)
{
    const uint2 w = ld_global(reinterpret_cast<const uint2 *>(p.ids) + m);
    const int64_t id = (int64_t)((uint64_t)w.y << 32 | w.x);
    return id < -1 || id >= p.L;
}

// The tile that begins with row m: `mine` is the row index of this lane's slot (lane & 15), or -1; false if no tile
// does.  A tile begins with every 16th row of an adapter.  All threads of the block.
__device__ __forceinline__ bool gather_tile(const Lora &p, int m, int adapter, int &mine)
{
    __shared__ uint32_t same[kGatherRows / 32];
    for (int r = threadIdx.x; r < kGatherRows; r += kThreads) {
        const uint32_t bits = __ballot_sync(kFull, r < p.M && adapter_of(p, r) == adapter);
        if ((threadIdx.x & 31) == 0)
            same[r >> 5] = bits;
    }
    __syncthreads();
    int before = 0;
    for (int w = 0; w < (m >> 5); ++w)
        before += __popc(same[w]);
    before += __popc(same[m >> 5] & ((1u << (m & 31)) - 1u));
    if (before % kTile != 0)
        return false;
    // the slot-th row of the adapter from m on
    int left = threadIdx.x & (kTile - 1);
    mine = -1;
    uint32_t bits = same[m >> 5] & ~((1u << (m & 31)) - 1u);
    for (int w = m >> 5;;) {
        const int n = __popc(bits);
        if (left < n) {
            for (; left > 0; --left)
                bits &= bits - 1u;
            mine = w * 32 + __ffs(bits) - 1;
            break;
        }
        left -= n;
        if (++w >= kGatherRows / 32)
            break;
        bits = same[w];
    }
    return true;
}

__device__ __forceinline__ uint4 piece(const uint8_t *row, int k, int K)
{
    if (row == nullptr || k >= K)
        return make_uint4(0, 0, 0, 0);
    return ld_global(reinterpret_cast<const uint4 *>(row + (int64_t)k * 2));
}

// acc += x (two rows of this lane) times the adapter's ranks, over the units [u0, u1) of K.
template <int NT>
__device__ __forceinline__ void product(float (&acc)[NT][4], const uint8_t *x0, const uint8_t *x1, const uint8_t *a,
                                        int R, int K, int u0, int u1)
{
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    for (int u = u0; u < u1; u += kBatch) {
        uint4 xa[kBatch], xb[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int k = (u + i) * kUnit + 8 * t, end = u + i < u1 ? K : 0;
            xa[i] = piece(x0, k, end);
            xb[i] = piece(x1, k, end);
        }
        float sum[NT][4] = {};   // of at most 128 columns, then added with IEEE operations
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int k = (u + i) * kUnit + 8 * t, end = u + i < u1 ? K : 0;
            uint4 w[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n)
                w[n] = piece(8 * n + g < R ? a + (int64_t)(8 * n + g) * K * 2 : nullptr, k, end);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                mma_bf16(sum[n], xa[i].x, xb[i].x, xa[i].y, xb[i].y, w[n].x, w[n].y);
                mma_bf16(sum[n], xa[i].z, xb[i].z, xa[i].w, xb[i].w, w[n].z, w[n].w);
            }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c)
                acc[n][c] = __fadd_rn(acc[n][c], sum[n][c]);
    }
}

// Rows m0 and m1 of this lane (-1: none) to the workspace.
template <int NT>
__device__ __forceinline__ void leave(const Lora &p, const float (&acc)[NT][4], int64_t m0, int64_t m1, int split)
{
    const int t = threadIdx.x & 3;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int r = 8 * n + 2 * t;
        if (r < p.R && m0 >= 0)
            *reinterpret_cast<float2 *>(p.parts + ((int64_t)split * p.M + m0) * p.R + r) = make_float2(acc[n][0], acc[n][1]);
        if (r < p.R && m1 >= 0)
            *reinterpret_cast<float2 *>(p.parts + ((int64_t)split * p.M + m1) * p.R + r) = make_float2(acc[n][2], acc[n][3]);
    }
}

// Few rows: a block per row (where a tile begins) and part of K, its warps an eighth of that each.
template <int NT>
__global__ void __launch_bounds__(kThreads)
lora_shrink_few_kernel(Lora p)
{
    __shared__ __align__(16) float kept[kWarps / 2][NT * 32 * 4];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, m = blockIdx.x;
    grid_dependency_wait();
    allow_dependents();
    const int adapter = adapter_of(p, m);
    if (adapter < 0) {
        if (threadIdx.x == 0 && blockIdx.y == 0 && bad_id(p, m))
            raise(p.err, EP_ERR_INVALID_EXPERT);
        return;
    }
    int mine;
    if (!gather_tile(p, m, adapter, mine))
        return;
    const int m0 = __shfl_sync(kFull, mine, lane >> 2), m1 = __shfl_sync(kFull, mine, (lane >> 2) + 8);
    const int units = (p.K + kUnit - 1) / kUnit, all = p.splits * kWarps, part = blockIdx.y * kWarps + warp;
    float acc[NT][4] = {};
    product<NT>(acc, m0 < 0 ? nullptr : p.x + (int64_t)m0 * p.K * 2, m1 < 0 ? nullptr : p.x + (int64_t)m1 * p.K * 2,
                p.a + (int64_t)adapter * p.R * p.K * 2, p.R, p.K, (int)((int64_t)units * part / all),
                (int)((int64_t)units * (part + 1) / all));
#pragma unroll
    for (int half = kWarps / 2; half >= 1; half /= 2) {
        if (warp >= half && warp < 2 * half)
#pragma unroll
            for (int n = 0; n < NT; ++n)
                *reinterpret_cast<float4 *>(&kept[warp - half][(n * 32 + lane) * 4]) =
                    make_float4(acc[n][0], acc[n][1], acc[n][2], acc[n][3]);
        __syncthreads();
        if (warp < half)
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float4 v = *reinterpret_cast<const float4 *>(&kept[warp][(n * 32 + lane) * 4]);
                acc[n][0] = __fadd_rn(acc[n][0], v.x);
                acc[n][1] = __fadd_rn(acc[n][1], v.y);
                acc[n][2] = __fadd_rn(acc[n][2], v.z);
                acc[n][3] = __fadd_rn(acc[n][3], v.w);
            }
        __syncthreads();
    }
    if (warp == 0)
        leave<NT>(p, acc, m0, m1, blockIdx.y);
}

// Many rows: a warp per 16 neighbouring rows and part of K.
template <int NT>
__global__ void __launch_bounds__(kThreads)
lora_shrink_kernel(Lora p)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t first = ((int64_t)blockIdx.x * kWarps + warp) * kTile;
    grid_dependency_wait();
    allow_dependents();
    int adapter = -1;
    if (lane < kTile && first + lane < p.M) {
        adapter = adapter_of(p, first + lane);
        if (adapter < 0 && blockIdx.y == 0 && bad_id(p, first + lane))
            raise(p.err, EP_ERR_INVALID_EXPERT);
    }
    const int units = (p.K + kUnit - 1) / kUnit;
    const int u0 = (int)((int64_t)units * blockIdx.y / p.splits), u1 = (int)((int64_t)units * (blockIdx.y + 1) / p.splits);
    for (uint32_t left = __ballot_sync(kFull, adapter >= 0); left != 0;) {
        const int now = __shfl_sync(kFull, adapter, __ffs(left) - 1);
        const uint32_t rows = __ballot_sync(kFull, adapter == now);
        left &= ~rows;
        const int g = lane >> 2;
        const int64_t m0 = rows >> g & 1u ? first + g : -1, m1 = rows >> (g + 8) & 1u ? first + g + 8 : -1;
        float acc[NT][4] = {};
        product<NT>(acc, m0 < 0 ? nullptr : p.x + m0 * p.K * 2, m1 < 0 ? nullptr : p.x + m1 * p.K * 2,
                    p.a + (int64_t)now * p.R * p.K * 2, p.R, p.K, u0, u1);
        leave<NT>(p, acc, m0, m1, blockIdx.y);
    }
}

// ---------------------------------------------------------------- expand --
// Words of a lane's piece of a row of ranks: 16 bytes for each 32 ranks, or 8 for each 16.
template <int UNITS, int WORDS>
struct Ranks {
    uint32_t v[UNITS][WORDS];

    __device__ __forceinline__ void load(const uint8_t *row, int R)
    {
        const int t = threadIdx.x & 3;
#pragma unroll
        for (int u = 0; u < UNITS; ++u) {
            const int r = (u * 4 + t) * WORDS * 2;
#pragma unroll
            for (int w = 0; w < WORDS; ++w)
                v[u][w] = 0;
            if (row != nullptr && r < R) {
                if constexpr (WORDS == 4) {
                    const uint4 q = ld_global(reinterpret_cast<const uint4 *>(row + r * 2));
                    v[u][0] = q.x, v[u][1] = q.y, v[u][2] = q.z, v[u][3] = q.w;
                } else {
                    const uint2 q = ld_global(reinterpret_cast<const uint2 *>(row + r * 2));
                    v[u][0] = q.x, v[u][1] = q.y;
                }
            }
        }
    }
};

// v of a row (the parts in their order, scaled) as planes of bf16.
template <int UNITS, int WORDS>
__device__ __forceinline__ void load_v(Ranks<UNITS, WORDS> (&v)[kPlanes], const Lora &p, int64_t m, float scaling)
{
    const int t = threadIdx.x & 3;
#pragma unroll
    for (int u = 0; u < UNITS; ++u)
#pragma unroll
        for (int w = 0; w < WORDS; ++w) {
            const int r = (u * 4 + t) * WORDS * 2 + 2 * w;
            float a = 0.0f, b = 0.0f;
            if (m >= 0 && r < p.R)
                for (int z = 0; z < p.splits; ++z) {
                    const uint2 q = ld_global(reinterpret_cast<const uint2 *>(p.parts + ((int64_t)z * p.M + m) * p.R + r));
                    a = __fadd_rn(a, __uint_as_float(q.x));
                    b = __fadd_rn(b, __uint_as_float(q.y));
                }
            a = __fmul_rn(a, scaling);
            b = __fmul_rn(b, scaling);
#pragma unroll
            for (int i = 0; i < kPlanes; ++i) {
                v[i].v[u][w] = pack_bf16x2(a, b);
                // what is left of an infinity or NaN is nothing
                a = isfinite(a) ? __fsub_rn(a, bf16_lo(v[i].v[u][w])) : 0.0f;
                b = isfinite(b) ? __fsub_rn(b, bf16_hi(v[i].v[u][w])) : 0.0f;
            }
        }
}

// Eight columns of a row: base (or nothing) plus d, to out.
__device__ __forceinline__ void put(const Lora &p, int64_t m, int n, const float (&d)[8])
{
    const int64_t at = m * p.N + n;
    float f[8] = {};
    if (p.base != nullptr) {
        if (p.base_dtype == 0) {
            const uint4 q = ld_global(reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(p.base) + at * 2));
            const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[2 * i] = bf16_lo(w[i]);
                f[2 * i + 1] = bf16_hi(w[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint4 q = ld_global(reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(p.base) + at * 4) + i);
                f[4 * i] = __uint_as_float(q.x);
                f[4 * i + 1] = __uint_as_float(q.y);
                f[4 * i + 2] = __uint_as_float(q.z);
                f[4 * i + 3] = __uint_as_float(q.w);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        f[i] = __fadd_rn(f[i], d[i]);
    if (p.out_dtype == 0) {
        *reinterpret_cast<uint4 *>(static_cast<uint8_t *>(p.out) + at * 2) =
            make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
    } else {
        float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(p.out) + at);
        o[0] = make_float4(f[0], f[1], f[2], f[3]);
        o[1] = make_float4(f[4], f[5], f[6], f[7]);
    }
}

// 32 columns from n0 on of the tile's rows m0 and m1 (-1: none).  Column g of
// block j stands for column n0 + 8 (g / 2) + 2 j + g % 2, so that a lane ends up
// with eight neighbouring columns of each of its rows.
template <int UNITS, int WORDS>
__device__ __forceinline__ void columns(const Lora &p, const Ranks<UNITS, WORDS> (&v0)[kPlanes],
                                        const Ranks<UNITS, WORDS> (&v1)[kPlanes], int adapter, int64_t m0, int64_t m1,
                                        int n0)
{
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    float d[4][4];
    const float none = adapter >= 0 ? 0.0f : -0.0f;   // base + -0 is base
#pragma unroll
    for (int j = 0; j < 4; ++j)
        d[j][0] = d[j][1] = d[j][2] = d[j][3] = none;
    if (adapter >= 0) {
        Ranks<UNITS, WORDS> b[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int n = n0 + 8 * (g >> 1) + 2 * j + (g & 1);
            b[j].load(n < p.N ? p.b + ((int64_t)adapter * p.N + n) * p.R * 2 : nullptr, p.R);
        }
#pragma unroll
        for (int i = kPlanes - 1; i >= 0; --i)
#pragma unroll
            for (int u = 0; u < UNITS; ++u)
#pragma unroll
                for (int w = 0; w < WORDS; w += 2)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        mma_bf16(d[j], v0[i].v[u][w], v1[i].v[u][w], v0[i].v[u][w + 1], v1[i].v[u][w + 1], b[j].v[u][w],
                                 b[j].v[u][w + 1]);
    }
    const int n = n0 + 8 * t;
    if (n >= p.N)
        return;
    if (m0 >= 0)
        put(p, m0, n, {d[0][0], d[0][1], d[1][0], d[1][1], d[2][0], d[2][1], d[3][0], d[3][1]});
    if (m1 >= 0)
        put(p, m1, n, {d[0][2], d[0][3], d[1][2], d[1][3], d[2][2], d[2][3], d[3][2], d[3][3]});
}

__device__ __forceinline__ float scaling_of(const Lora &p, int adapter)
{
    return adapter < 0 || p.scaling == nullptr
               ? 1.0f : __uint_as_float(ld_global(reinterpret_cast<const uint32_t *>(p.scaling) + adapter));
}

// Few rows: a block per row (where a tile begins, or without an adapter) and 256 columns.
template <int UNITS, int WORDS>
__global__ void __launch_bounds__(kThreads)
lora_expand_few_kernel(Lora p)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, m = blockIdx.x;
    grid_dependency_wait();
    allow_dependents();
    const int adapter = adapter_of(p, m);
    int mine = (lane & (kTile - 1)) == 0 ? m : -1;
    if (adapter >= 0 && !gather_tile(p, m, adapter, mine))
        return;
    const int m0 = __shfl_sync(kFull, mine, lane >> 2), m1 = __shfl_sync(kFull, mine, (lane >> 2) + 8);
    const int n0 = (blockIdx.y * kWarps + warp) * 32;
    if (n0 >= p.N)
        return;
    Ranks<UNITS, WORDS> v0[kPlanes], v1[kPlanes];
    const float scaling = scaling_of(p, adapter);
    load_v(v0, p, adapter < 0 ? -1 : m0, scaling);
    load_v(v1, p, adapter < 0 ? -1 : m1, scaling);
    columns(p, v0, v1, adapter, m0, m1, n0);
}

// Many rows: a warp per 16 neighbouring rows and `chunk` columns.
template <int UNITS, int WORDS>
__global__ void __launch_bounds__(kThreads)
lora_expand_kernel(Lora p, int chunk)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2;
    const int64_t first = ((int64_t)blockIdx.x * kWarps + warp) * kTile;
    grid_dependency_wait();
    allow_dependents();
    const bool in = lane < kTile && first + lane < p.M;
    const int adapter = in ? adapter_of(p, first + lane) : -1;
    for (uint32_t left = __ballot_sync(kFull, in); left != 0;) {
        const int now = __shfl_sync(kFull, adapter, __ffs(left) - 1);
        const uint32_t rows = __ballot_sync(kFull, in && adapter == now);
        left &= ~rows;
        const int64_t m0 = rows >> g & 1u ? first + g : -1, m1 = rows >> (g + 8) & 1u ? first + g + 8 : -1;
        Ranks<UNITS, WORDS> v0[kPlanes], v1[kPlanes];
        const float scaling = scaling_of(p, now);
        load_v(v0, p, now < 0 ? -1 : m0, scaling);
        load_v(v1, p, now < 0 ? -1 : m1, scaling);
        const int from = blockIdx.y * chunk, to = min(from + chunk, p.N);
        for (int n0 = from; n0 < to; n0 += 32)
            columns(p, v0, v1, now, m0, m1, n0);
    }
}

// ---------------------------------------------------------------- launch --
// Parts of K: as many as fill the GPU, at least a unit to a warp of each.  Tiles are estimated from the sizes alone.
int splits_of(int64_t M, int K, int L)
{
    const bool few = M <= kGatherRows;
    const int64_t tiles = few ? std::min<int64_t>(M, L + M / kTile) : ceil_div(M, kTile * kWarps);
    const int64_t most = std::min<int64_t>(kMaxSplits, ceil_div(K, kUnit * (few ? kWarps : kBatch)));
    return (int)std::max<int64_t>(1, std::min<int64_t>(most, kBlocks / std::max<int64_t>(1, tiles)));
}

template <int NT>
int launch_shrink(const Lora &p, cudaStream_t stream)
{
    if (p.M <= kGatherRows)
        return launch_dependent(lora_shrink_few_kernel<NT>, dim3((unsigned)p.M, p.splits), kThreads, 0, stream, p);
    return launch_dependent(lora_shrink_kernel<NT>, dim3((unsigned)ceil_div(p.M, kTile * kWarps), p.splits), kThreads, 0,
                            stream, p);
}

template <int UNITS, int WORDS>
int launch_expand(const Lora &p, cudaStream_t stream)
{
    if (p.M <= kGatherRows)
        return launch_dependent(lora_expand_few_kernel<UNITS, WORDS>,
                                dim3((unsigned)p.M, (unsigned)ceil_div(p.N, 32 * kWarps)), kThreads, 0, stream, p);
    const int64_t tiles = ceil_div(p.M, kTile * kWarps);
    const int64_t pieces = std::max<int64_t>(1, std::min<int64_t>(ceil_div(p.N, 32), ceil_div(2 * kBlocks, tiles)));
    const int chunk = (int)(ceil_div(ceil_div(p.N, pieces), 32) * 32);
    return launch_dependent(lora_expand_kernel<UNITS, WORDS>, dim3((unsigned)tiles, (unsigned)ceil_div(p.N, chunk)),
                            kThreads, 0, stream, p, chunk);
}

}  // namespace
}  // namespace ep

using namespace ep;

extern "C" size_t ep_lora_workspace_size(int64_t M, int R)
{
    if (M < 0 || R < 1)
        return 0;
    // splits_of(m) * m is at most this for every m <= M, so that a workspace serves smaller batches too
    const int64_t rows = std::min<int64_t>(kMaxSplits * M, std::max<int64_t>(M, (int64_t)kBlocks * kTile * kWarps));
    return align_up((size_t)rows * R * sizeof(float), kWsAlign) + kWsAlign;
}

extern "C" int ep_lora(const void *x, int64_t M, int K, const int64_t *ids, const void *a, const void *b,
                       const float *scaling, int L, int R, int N, const void *base, int base_dtype, void *out,
                       int out_dtype, void *ws, size_t ws_bytes, int32_t *err, ep_stream_t stream_)
{
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    if (M < 0 || K < 8 || K % 8 != 0 || N < 8 || N % 8 != 0 || R < 8 || R % 8 != 0 || L < 1)
        return EP_ERR_INVALID_ARG;
    if ((out_dtype != 0 && out_dtype != 1) || (base != nullptr && base_dtype != 0 && base_dtype != 1) || R > kMaxRank ||
        K > (1 << 24) || N > (1 << 24) || M > (1 << 24))
        return EP_ERR_UNSUPPORTED;
    if (M == 0)
        return EP_OK;
    if (x == nullptr || ids == nullptr || a == nullptr || b == nullptr || out == nullptr || !aligned(x, 16) ||
        !aligned(a, 16) || !aligned(b, 16) || !aligned(base, 16) || !aligned(out, 16) || !aligned(ids, 8) ||
        !aligned(scaling, 4) || !aligned(err, 4) || (out == base && base_dtype != out_dtype) || ws == nullptr ||
        !aligned(ws, kWsAlign) || ws_bytes < ep_lora_workspace_size(M, R))
        return EP_ERR_INVALID_ARG;
    const Lora p{static_cast<const uint8_t *>(x), static_cast<const uint8_t *>(a), static_cast<const uint8_t *>(b), ids,
                 scaling, base, out, M, K, N, R, L, splits_of(M, K, L), base_dtype, out_dtype, static_cast<float *>(ws),
                 err};
    const int rc = R <= 8 ? launch_shrink<1>(p, stream) : R <= 16 ? launch_shrink<2>(p, stream)
                 : R <= 32 ? launch_shrink<4>(p, stream) : R <= 64 ? launch_shrink<8>(p, stream)
                                                                   : launch_shrink<16>(p, stream);
    if (rc != EP_OK)
        return rc;
    if (R <= 16)
        return launch_expand<1, 2>(p, stream);
    if (R <= 32)
        return launch_expand<1, 4>(p, stream);
    return R <= 64 ? launch_expand<2, 4>(p, stream) : launch_expand<4, 4>(p, stream);
}
