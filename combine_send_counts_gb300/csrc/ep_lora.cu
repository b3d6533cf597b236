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
//   more rows: a tile is 128 neighbouring rows, gone over once for each adapter that
//   they name, which is one or two where requests are long.
//
// v is kept whole between the two products, as the sum of three bf16 terms (24
// bits), because the matrix step takes bf16.
#include <algorithm>
#include <type_traits>

#include "ep_device.cuh"
#include "ep_internal.h"
#include "ep_launch.cuh"
#include "ep_lora.cuh"
#include "ep_skinny.cuh"

namespace ep {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kUnit = 32;            // columns of a lane's 16-byte pieces: two k16 steps
constexpr int kBatch = 4;            // units loaded together, and summed by matrix steps alone
constexpr int kTile = 16;

// The tile that begins with row m: `mine` is the row index of this lane's slot (lane & 15), or -1; false if no tile
// does.  A tile begins with every 16th row of an adapter.  All threads of the block.
__device__ __forceinline__ bool gather_tile(const Lora &p, int m, int adapter, int &mine)
{
    __shared__ uint32_t same[kLoraFewRows / 32];
    const int words = ((int)p.M + 31) / 32;
    for (int r = threadIdx.x; r < words * 32; r += kThreads) {
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
        if (++w >= words)
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

// Eight columns of a row of the base as they are loaded, bf16 (in lo) or fp32.
struct Base {
    uint4 lo, hi;

    __device__ __forceinline__ void load(const Lora &p, int64_t m, int n)
    {
        lo = hi = make_uint4(0, 0, 0, 0);
        if (m < 0 || n >= p.N || p.base == nullptr)
            return;
        const uint4 *at = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(p.base) +
                                                          (m * p.N + n) * (p.base_dtype == 0 ? 2 : 4));
        lo = ld_global(at);
        if (p.base_dtype != 0)
            hi = ld_global(at + 1);
    }
};

// Eight neighbouring columns: base plus d, to out.
__device__ __forceinline__ void put(void *out, bool bf16_base, bool bf16_out, const Base &base, const float (&d)[8])
{
    const uint32_t w[8] = {base.lo.x, base.lo.y, base.lo.z, base.lo.w, base.hi.x, base.hi.y, base.hi.z, base.hi.w};
    float f[8];
    if (bf16_base) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = bf16_lo(w[i]);
            f[2 * i + 1] = bf16_hi(w[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            f[i] = __uint_as_float(w[i]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        f[i] = __fadd_rn(f[i], d[i]);
    if (bf16_out) {
        *static_cast<uint4 *>(out) =
            make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
    } else {
        static_cast<float4 *>(out)[0] = make_float4(f[0], f[1], f[2], f[3]);
        static_cast<float4 *>(out)[1] = make_float4(f[4], f[5], f[6], f[7]);
    }
}

// Few rows: a block per row (where a tile begins, or without an adapter) and 256
// columns.  Column g of block j of a warp's 32 stands for column n0 + 8 (g / 2) + 2 j +
// g % 2, so that a lane ends up with eight neighbouring columns of each of its rows.
// The block makes v once, in shared memory.
template <int UNITS, int WORDS>
__global__ void __launch_bounds__(kThreads)
lora_expand_few_kernel(Lora p)
{
    constexpr int kRanks = UNITS * WORDS * 8, kVRow = kRanks * 2 + 16;   // bytes of a row of v
    __shared__ __align__(16) uint8_t v_room[kPlanes][kTile][kVRow];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, m = blockIdx.x;
    // Every block of shrink has waited for what was before it, so that only what shrink itself writes is waited for here.
    const int adapter = adapter_of(p, m);
    const int n0 = (blockIdx.y * kWarps + warp) * 32, n = n0 + 8 * t;
    Ranks<UNITS, WORDS> b[4];
    auto load_b = [&]() {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int row = n0 + 8 * (g >> 1) + 2 * j + (g & 1);
            b[j].load(adapter >= 0 && row < p.N ? p.b + ((int64_t)adapter * p.N + row) * p.R * 2 : nullptr, p.R);
        }
    };
    const bool early = p.M <= 64;   // most blocks have a tile, and nothing waits for the ids
    if (early)
        load_b();
    int mine = (lane & (kTile - 1)) == 0 ? m : -1;
    if (adapter >= 0 && !gather_tile(p, m, adapter, mine))
        return;
    const int m0 = __shfl_sync(kFull, mine, g), m1 = __shfl_sync(kFull, mine, g + 8);
    Base base0, base1;
    base0.load(p, m0, n);
    base1.load(p, m1, n);
    if (!early)
        load_b();
    const float none = adapter >= 0 ? 0.0f : -0.0f;   // base + -0 is base
    float d[4][4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        d[j][0] = d[j][1] = d[j][2] = d[j][3] = none;
    const float scaling = scaling_of(p, adapter);
    grid_dependency_wait();
    allow_dependents();
    if (adapter >= 0) {
        for (int i = warp; i < kTile; i += kWarps) {   // a warp to a row
            const int row = __shfl_sync(kFull, mine, i);
            for (int r = 2 * lane; r < kRanks; r += 64) {
                uint32_t terms[kPlanes];
                split(ranks_of(p, row, r, scaling), terms);
#pragma unroll
                for (int z = 0; z < kPlanes; ++z)
                    *reinterpret_cast<uint32_t *>(&v_room[z][i][r * 2]) = terms[z];
            }
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < UNITS; ++u)
#pragma unroll
            for (int z = kPlanes - 1; z >= 0; --z) {
                uint32_t v0[WORDS], v1[WORDS];
                const uint32_t *at0 = reinterpret_cast<const uint32_t *>(&v_room[z][g][(u * 4 + t) * WORDS * 4]);
                const uint32_t *at1 = reinterpret_cast<const uint32_t *>(&v_room[z][g + 8][(u * 4 + t) * WORDS * 4]);
#pragma unroll
                for (int w = 0; w < WORDS; ++w) {
                    v0[w] = at0[w];
                    v1[w] = at1[w];
                }
#pragma unroll
                for (int w = 0; w < WORDS; w += 2)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        mma_bf16(d[j], v0[w], v1[w], v0[w + 1], v1[w + 1], b[j].v[u][w], b[j].v[u][w + 1]);
            }
    }
    if (n >= p.N)
        return;
    const bool bf16_base = p.base_dtype == 0, bf16_out = p.out_dtype == 0;
    auto at = [&](int m) { return static_cast<uint8_t *>(p.out) + ((int64_t)m * p.N + n) * (bf16_out ? 2 : 4); };
    if (m0 >= 0)
        put(at(m0), bf16_base, bf16_out, base0, {d[0][0], d[0][1], d[1][0], d[1][1], d[2][0], d[2][1], d[3][0], d[3][1]});
    if (m1 >= 0)
        put(at(m1), bf16_base, bf16_out, base1, {d[0][2], d[0][3], d[1][2], d[1][3], d[2][2], d[2][3], d[3][2], d[3][3]});
}

// ---------------------------------------------------------------- launch --
// Parts of K: as many as fill the GPU, at least a unit to a warp of each, or 256
// columns of many rows.  Tiles are estimated from the sizes alone.
int splits_of(int64_t M, int K, int L)
{
    const bool few = M <= kLoraFewRows;
    const int64_t tiles = few ? std::min<int64_t>(M, L + M / kTile) : ceil_div(M, 128);
    const int64_t most = std::min<int64_t>(kLoraMaxSplits, ceil_div(K, 256));
    return (int)std::max<int64_t>(1, std::min<int64_t>(most, kLoraBlocks / std::max<int64_t>(1, tiles)));
}

template <int NT, int UNITS, int WORDS>
int launch_few(const Lora &p, cudaStream_t stream)
{
    const int rc = launch_dependent(lora_shrink_few_kernel<NT>, dim3((unsigned)p.M, p.splits), kThreads, 0, stream, p);
    if (rc != EP_OK)
        return rc;
    return launch_dependent(lora_expand_few_kernel<UNITS, WORDS>,
                            dim3((unsigned)p.M, (unsigned)ceil_div(p.N, 32 * kWarps)), kThreads, 0, stream, p);
}

int launch_few(const Lora &p, cudaStream_t stream)
{
    if (p.R <= 8)
        return launch_few<1, 1, 2>(p, stream);
    if (p.R <= 16)
        return launch_few<2, 1, 2>(p, stream);
    if (p.R <= 32)
        return launch_few<4, 1, 4>(p, stream);
    return p.R <= 64 ? launch_few<8, 2, 4>(p, stream) : launch_few<16, 4, 4>(p, stream);
}

}  // namespace
}  // namespace ep

using namespace ep;

extern "C" size_t ep_lora_workspace_size(int64_t M, int R)
{
    if (M < 0 || R < 1)
        return 0;
    // splits_of(m) * m is at most this for every m <= M, so that a workspace serves smaller batches too
    const int64_t rows = std::min<int64_t>(kLoraMaxSplits * M, std::max<int64_t>(M, (int64_t)kLoraBlocks * 128));
    return align_up((size_t)rows * R * sizeof(float), kWsAlign) + kWsAlign;
}

extern "C" int ep_lora(const void *x, int64_t M, int K, const int64_t *ids, const void *a, const void *b,
                       const float *scaling, int L, int R, int N, const void *base, int base_dtype, void *out,
                       int out_dtype, void *ws, size_t ws_bytes, int32_t *err, ep_stream_t stream_)
{
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    if (M < 0 || K < 8 || K % 8 != 0 || N < 8 || N % 8 != 0 || R < 8 || R % 8 != 0 || L < 1)
        return EP_ERR_INVALID_ARG;
    if ((out_dtype != 0 && out_dtype != 1) || (base != nullptr && base_dtype != 0 && base_dtype != 1) || R > kLoraMaxRank ||
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
    return M <= kLoraFewRows ? launch_few(p, stream) : launch_lora_many(p, stream);
}
