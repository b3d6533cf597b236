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

// Ranks r and r + 1 of v of row m: the parts in their order, scaled.
__device__ __forceinline__ float2 ranks_of(const Lora &p, int64_t m, int r, float scaling)
{
    float2 v = make_float2(0.0f, 0.0f);
    if (m < 0 || r >= p.R)
        return v;
    const float2 *part = reinterpret_cast<const float2 *>(p.parts + m * p.R + r);
    const int64_t next = p.M * p.R / 2;
    for (int z = 0; z < p.splits; z += 4) {
        float2 u[4];   // loaded together
#pragma unroll
        for (int i = 0; i < 4; ++i)
            u[i] = z + i < p.splits ? part[(z + i) * next] : make_float2(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v.x = __fadd_rn(v.x, u[i].x);
            v.y = __fadd_rn(v.y, u[i].y);
        }
    }
    return make_float2(__fmul_rn(v.x, scaling), __fmul_rn(v.y, scaling));
}

// Two values as sums of kPlanes bf16 terms each.
__device__ __forceinline__ void split(float2 v, uint32_t (&w)[kPlanes])
{
#pragma unroll
    for (int i = 0; i < kPlanes; ++i) {
        w[i] = pack_bf16x2(v.x, v.y);
        // what is left of an infinity or NaN is nothing
        v.x = isfinite(v.x) ? __fsub_rn(v.x, bf16_lo(w[i])) : 0.0f;
        v.y = isfinite(v.y) ? __fsub_rn(v.y, bf16_hi(w[i])) : 0.0f;
    }
}

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

__device__ __forceinline__ float scaling_of(const Lora &p, int adapter)
{
    return adapter < 0 || p.scaling == nullptr
               ? 1.0f : __uint_as_float(ld_global(reinterpret_cast<const uint32_t *>(p.scaling) + adapter));
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
    grid_dependency_wait();
    allow_dependents();
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
    if (adapter >= 0) {
        const float scaling = scaling_of(p, adapter);
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

// ------------------------------------------------------------- many rows --
// Tiles of 128 (or 64) neighbouring rows.  The adapters among a tile's rows, a few
// at a time in ascending order, have their weights in the same stage of a ring
// in shared memory (cp.async; rows 16 bytes apart from a multiple of 128, so that
// the eight rows of a matrix load meet no bank twice).  A warp takes those that its rows
// name, each for its own rows.
__device__ __forceinline__ void load_matrices(uint32_t (&r)[4], uint32_t at)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}

constexpr int kNoRow = 0x7fffffff;   // the adapter of a row past the end

// The least adapter above `last` among `rows` in shared memory, kNoRow if there is none.  The same in every lane.
__device__ __forceinline__ int adapter_after(const int *ids, int rows, int last)
{
    int least = kNoRow;
    for (int i = threadIdx.x & 31; i < rows; i += 32)
        least = ids[i] > last ? min(least, ids[i]) : least;
    return __reduce_min_sync(kFull, least);
}

constexpr int kChunk = 64;                       // columns of x a stage
constexpr int kRow = kChunk * 2 + 16;            // bytes of a row in shared memory

template <int NT, int MW, int SLOTS, int STAGES, int THREADS>
struct Shrink {
    static constexpr int kRows = THREADS / 32 * 16 * MW, kRanks = NT * 8, kStages = STAGES;
    static constexpr int kStage = (kRows + SLOTS * kRanks) * kRow;
    static constexpr int kBytes = kStages * kStage;
};

// v: a warp has MW blocks of 16 rows and all ranks.
template <int NT, int MW, int SLOTS, int STAGES, int THREADS>
__global__ void __launch_bounds__(THREADS)
lora_shrink_kernel(Lora p)
{
    using S = Shrink<NT, MW, SLOTS, STAGES, THREADS>;
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ int ids[S::kRows];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2;
    const int64_t first = (int64_t)blockIdx.x * S::kRows;
    grid_dependency_wait();
    allow_dependents();
    for (int r = threadIdx.x; r < S::kRows; r += THREADS) {
        ids[r] = first + r < p.M ? adapter_of(p, first + r) : -1;
        if (blockIdx.y == 0 && first + r < p.M && bad_id(p, first + r))
            raise(p.err, EP_ERR_INVALID_EXPERT);
    }
    __syncthreads();
    const int chunks = (p.K + kChunk - 1) / kChunk;
    const int c0 = (int)((int64_t)chunks * blockIdx.y / p.splits), c1 = (int)((int64_t)chunks * (blockIdx.y + 1) / p.splits);
    const uint32_t base = smem_u32(ring);
    // this thread's pieces: of 16 bytes, at `piece` of rows r0, r0 + kStep, ...
    const int r0 = threadIdx.x >> 3, piece = threadIdx.x & 7;
    constexpr int kStep = THREADS / 8, kXPieces = S::kRows / kStep, kAPieces = (S::kRanks + kStep - 1) / kStep;
    const int64_t x_row = (int64_t)p.K * 2 * kStep;   // from a piece to the next, in bytes
    for (int now = adapter_after(ids, S::kRows, -1); now != kNoRow;) {
        int slot_of[SLOTS];   // the adapters of this pass
        int slots = 0;
#pragma unroll
        for (int i = 0; i < SLOTS; ++i) {
            slot_of[i] = now;
            slots += now != kNoRow;
            if (now != kNoRow)
                now = adapter_after(ids, S::kRows, now);
        }
        uint32_t here = 0;   // rows of this thread's pieces that the pass is for
#pragma unroll
        for (int i = 0; i < kXPieces; ++i) {
            const int id = ids[r0 + kStep * i];
            here |= (id >= slot_of[0] && id < now && id != kNoRow ? 1u : 0u) << i;
        }
        uint32_t mine = 0;   // slots that this warp's rows name
#pragma unroll
        for (int i = 0; i < SLOTS; ++i) {
            bool any = false;
#pragma unroll
            for (int w = 0; w < MW; ++w)
                any |= lane < 16 && ids[(warp * MW + w) * 16 + (lane & 15)] == slot_of[i];
            if (__any_sync(kFull, any && slot_of[i] != kNoRow))
                mine |= 1u << i;
        }
        const bool mixed = (mine & (mine - 1u)) != 0;
        const uint8_t *x_at = p.x + ((first + r0) * p.K + piece * 8) * 2;
        auto fetch = [&](int c) {
            if (c < c1) {
                const uint32_t to = base + (c % STAGES) * S::kStage + r0 * kRow + piece * 16;
                const int64_t k = (int64_t)c * kChunk * 2;
                const bool in = c * kChunk + piece * 8 < p.K;
#pragma unroll
                for (int i = 0; i < kXPieces; ++i) {
                    const bool ok = in && (here >> i & 1u);
                    cp_async16(to + i * kStep * kRow, ok ? x_at + i * x_row + k : p.x, ok);
                }
#pragma unroll
                for (int i = 0; i < SLOTS; ++i) {
                    if (i >= slots)
                        break;
                    const uint8_t *a_at = p.a + (((int64_t)slot_of[i] * p.R + r0) * p.K + piece * 8) * 2;
#pragma unroll
                    for (int j = 0; j < kAPieces; ++j) {
                        const int r = r0 + kStep * j;
                        const bool ok = in && r < p.R;
                        if (r < S::kRanks)
                            cp_async16(to + (S::kRows + i * S::kRanks + j * kStep) * kRow, ok ? a_at + j * x_row + k : p.a, ok);
                    }
                }
            }
            cp_async_commit();
        };
#pragma unroll
        for (int i = 0; i < STAGES - 1; ++i)
            fetch(c0 + i);
        float acc[MW][NT][4] = {}, sum[MW][NT][4] = {};   // sums of at most 128 columns are added with IEEE operations
        for (int c = c0; c < c1; ++c) {
            cp_async_wait<STAGES - 2>();
            __syncthreads();
            fetch(c + STAGES - 1);
            const uint32_t stage = base + (c % STAGES) * S::kStage;
            for (uint32_t todo = mine; todo != 0; todo &= todo - 1u) {
                const int slot = __ffs(todo) - 1;
                int now_id = slot_of[0];
#pragma unroll
                for (int i = 1; i < SLOTS; ++i)
                    now_id = slot == i ? slot_of[i] : now_id;
#pragma unroll
                for (int k = 0; k < kChunk / 16; ++k) {
                    uint32_t x[MW][4];
#pragma unroll
                    for (int i = 0; i < MW; ++i)
                        load_matrices(x[i], stage + ((warp * MW + i) * 16 + (lane & 15)) * kRow + k * 32 + (lane >> 4) * 16);
#pragma unroll
                    for (int n = 0; n < NT; n += 2) {
                        uint32_t w[4];   // with one block of ranks the other half is not used
                        const int row = NT > 1 ? n * 8 + (lane >> 4) * 8 + (lane & 7) : lane & 7;
                        load_matrices(w, stage + (S::kRows + slot * S::kRanks + row) * kRow + k * 32 + (lane >> 3 & 1) * 16);
#pragma unroll
                        for (int i = 0; i < MW; ++i) {
                            mma_bf16(sum[i][n], x[i][0], x[i][1], x[i][2], x[i][3], w[0], w[1]);
                            if (NT > 1)
                                mma_bf16(sum[i][(n + 1) % NT], x[i][0], x[i][1], x[i][2], x[i][3], w[2], w[3]);
                        }
                    }
                }
                // sums of one adapter go to its own rows: another's weights, were they infinite, would make NaN of zeros
                if (mixed || (c - c0) % 2 == 1 || c + 1 == c1)
#pragma unroll
                    for (int i = 0; i < MW; ++i) {
                        const bool own0 = !mixed || ids[(warp * MW + i) * 16 + g] == now_id;
                        const bool own1 = !mixed || ids[(warp * MW + i) * 16 + g + 8] == now_id;
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int v = 0; v < 4; ++v) {
                                if (v < 2 ? own0 : own1)
                                    acc[i][n][v] = __fadd_rn(acc[i][n][v], sum[i][n][v]);
                                sum[i][n][v] = 0.0f;
                            }
                    }
            }
        }
        auto done = [&](int row) { return ids[row] >= slot_of[0] && ids[row] < now && ids[row] != kNoRow ? first + row : -1; };
#pragma unroll
        for (int i = 0; i < MW; ++i) {
            const int row = (warp * MW + i) * 16 + g;
            leave<NT>(p, acc[i], done(row), done(row + 8), blockIdx.y);
        }
        cp_async_wait<0>();
        __syncthreads();
    }
}

constexpr int kColumns = 64;     // of the output, a stage
constexpr int kExpandRows = kWarps * kTile;
constexpr int kExpandStages = 3;

// Adapters whose B a stage holds, for KS steps of 16 ranks.
__host__ __device__ constexpr int expand_slots(int ks) { return ks <= 2 ? 4 : 2; }

__host__ __device__ constexpr int expand_stage(int ks, int base_bytes)
{
    return expand_slots(ks) * kColumns * (ks * 32 + 16) + kThreads * base_bytes;
}

// out: a warp has 16 rows, whose v it holds in registers, and the block `span`
// columns.  A row of B's tile stands for a column as in the kernel for few rows; each
// thread fetches the part of the base that it will add to.  WIDE: 1 for a bf16 base, 2 for fp32.
template <int KS, int WIDE, bool BF16_OUT>
__global__ void __launch_bounds__(kThreads, KS <= 4 ? 2 : 1)
lora_expand_kernel(Lora p, int span)
{
    constexpr int kBRow = KS * 32 + 16, kSlots = expand_slots(KS), kBPieces = kColumns * KS * 2 / kThreads;
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ int ids[kExpandRows];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int64_t first = (int64_t)blockIdx.x * kExpandRows;
    grid_dependency_wait();
    allow_dependents();
    for (int r = threadIdx.x; r < kExpandRows; r += kThreads)
        ids[r] = first + r < p.M ? adapter_of(p, first + r) : kNoRow;
    __syncthreads();
    const int base_bytes = p.base == nullptr ? 0 : 64 * WIDE;
    const int b_bytes = kSlots * kColumns * kBRow, stage_bytes = b_bytes + kThreads * base_bytes;
    const int n_from = blockIdx.y * span, n_to = min(n_from + span, p.N);
    const uint32_t ring_at = smem_u32(ring);
    const int id0 = ids[warp * kTile + g], id1 = ids[warp * kTile + g + 8];
    // this thread's pieces of a tile of B: rows b_row, b_row + kThreads / (2 KS), ...
    const int b_piece = threadIdx.x % (KS * 2), b_row = threadIdx.x / (KS * 2);
    const bool b_in = b_piece * 8 < p.R && b_row < kColumns;
    for (int now = adapter_after(ids, kExpandRows, -2); now != kNoRow;) {
        // rows without an adapter are a pass of their own, of nothing but the base
        int slot_of[kSlots], slots = 0;
        const int least = now;
#pragma unroll
        for (int i = 0; i < kSlots; ++i) {
            slot_of[i] = now;
            if (now != kNoRow && (i == 0 || least >= 0)) {
                ++slots;
                now = adapter_after(ids, kExpandRows, now);
            }
        }
        const int64_t m0 = id0 >= least && id0 < now ? first + warp * kTile + g : -1;
        const int64_t m1 = id1 >= least && id1 < now ? first + warp * kTile + g + 8 : -1;
        const bool active = __any_sync(kFull, m0 >= 0 || m1 >= 0);
        uint32_t mine = 0;   // slots that this warp's rows name
        float scale0 = 1.0f, scale1 = 1.0f;
#pragma unroll
        for (int i = 0; i < kSlots; ++i)
            if (i < slots && least >= 0) {
                const bool in0 = id0 == slot_of[i], in1 = id1 == slot_of[i];
                if (__any_sync(kFull, in0 || in1)) {
                    mine |= 1u << i;
                    const float scaling = scaling_of(p, slot_of[i]);
                    scale0 = in0 ? scaling : scale0;
                    scale1 = in1 ? scaling : scale1;
                }
            }
        // 16 bytes of the base: row i (m0, m1), group of 32 columns j, part h of 32 bytes
        const uint32_t own = ring_at + b_bytes + threadIdx.x * 16;
        const uint8_t *base0 = static_cast<const uint8_t *>(p.base) + (m0 < 0 ? 0 : (m0 * p.N + 8 * t) * 2 * WIDE);
        const uint8_t *base1 = static_cast<const uint8_t *>(p.base) + (m1 < 0 ? 0 : (m1 * p.N + 8 * t) * 2 * WIDE);
        uint8_t *const out_at = static_cast<uint8_t *>(p.out) + (first + warp * kTile + g) * p.N * (BF16_OUT ? 2 : 4);
        const int64_t rows_apart = (int64_t)8 * p.N * (BF16_OUT ? 2 : 4);
        auto fetch = [&](int n0, int stage) {
            if (n0 < n_to) {
                const uint32_t to = ring_at + stage * stage_bytes;
                if (least >= 0)
#pragma unroll
                    for (int z = 0; z < kSlots; ++z) {
                        if (z >= slots)
                            break;
                        const uint8_t *b = p.b + (((int64_t)slot_of[z] * p.N + n0) * p.R + b_piece * 8) * 2;
#pragma unroll
                        for (int i = 0; i < (kBPieces > 0 ? kBPieces : 1); ++i) {
                            const int row = b_row + i * (kThreads / (KS * 2));
                            const int n = (row & 32) + 4 * (row & 6) + 2 * (row >> 3 & 3) + (row & 1);
                            const bool ok = b_in && n0 + n < p.N;
                            if (row < kColumns)
                                cp_async16(to + (z * kColumns + row) * kBRow + b_piece * 16, ok ? b + n * p.R * 2 : p.b, ok);
                        }
                    }
                if (p.base != nullptr) {
                    const uint32_t slot = own + stage * stage_bytes;
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int n = n0 + 32 * j;
                        const bool in = n + 8 * t < p.N;
#pragma unroll
                        for (int h = 0; h < WIDE; ++h) {
                            cp_async16(slot + (j * WIDE + h) * kThreads * 16, in ? base0 + n * 2 * WIDE + 16 * h : base0, in && m0 >= 0);
                            cp_async16(slot + ((2 + j) * WIDE + h) * kThreads * 16, in ? base1 + n * 2 * WIDE + 16 * h : base1,
                                       in && m1 >= 0);
                        }
                    }
                }
            }
            cp_async_commit();
        };
#pragma unroll
        for (int i = 0; i < kExpandStages - 1; ++i)
            fetch(n_from + i * kColumns, i);
        uint32_t v[kPlanes][KS][4];
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                uint32_t terms[kPlanes];
                split(ranks_of(p, least < 0 ? -1 : w % 2 == 0 ? m0 : m1, k * 16 + (w / 2) * 8 + 2 * t, w % 2 == 0 ? scale0 : scale1),
                      terms);
#pragma unroll
                for (int i = 0; i < kPlanes; ++i)
                    v[i][k][w] = terms[i];
            }
        int stage = 0;
        for (int n0 = n_from; n0 < n_to; n0 += kColumns) {
            cp_async_wait<kExpandStages - 2>();
            __syncthreads();
            fetch(n0 + (kExpandStages - 1) * kColumns, stage == 0 ? kExpandStages - 1 : stage - 1);
            if (active) {
                // one adapter after the other, each for its own rows; without adapters, once for the base
                for (uint32_t todo = least < 0 ? 1u : mine; todo != 0; todo &= todo - 1u) {
                    const int slot = __ffs(todo) - 1;
                    int id = slot_of[0];
#pragma unroll
                    for (int i = 1; i < kSlots; ++i)
                        id = slot == i ? slot_of[i] : id;
                    const float none = least >= 0 ? 0.0f : -0.0f;   // base + -0 is base
                    float d[8][4];
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        d[c][0] = d[c][1] = d[c][2] = d[c][3] = none;
                    const uint32_t tile = ring_at + stage * stage_bytes +
                                          (slot * kColumns + (lane >> 4) * 8 + (lane & 7)) * kBRow + (lane >> 3 & 1) * 16;
                    if (least >= 0)
#pragma unroll
                        for (int k = 0; k < KS; ++k) {
                            uint32_t w[4][4];
#pragma unroll
                            for (int c = 0; c < 4; ++c)
                                load_matrices(w[c], tile + c * 16 * kBRow + k * 32);
#pragma unroll
                            for (int i = kPlanes - 1; i >= 0; --i)
#pragma unroll
                                for (int c = 0; c < 8; ++c)
                                    mma_bf16(d[c], v[i][k][0], v[i][k][1], v[i][k][2], v[i][k][3], w[c / 2][c % 2 * 2],
                                             w[c / 2][c % 2 * 2 + 1]);
                        }
                    const uint32_t at = own + stage * stage_bytes;
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int n = n0 + 32 * j + 8 * t;
                        if (n >= p.N)
                            continue;
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            if ((i == 0 ? id0 : id1) != id)
                                continue;
                            Base base{make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
                            if (p.base != nullptr) {
                                base.lo = ld_shared16(at + (2 * i + j) * WIDE * kThreads * 16);
                                if (WIDE == 2)
                                    base.hi = ld_shared16(at + ((2 * i + j) * WIDE + 1) * kThreads * 16);
                            }
                            put(out_at + (i == 0 ? 0 : rows_apart) + (int64_t)n * (BF16_OUT ? 2 : 4), WIDE == 1, BF16_OUT, base,
                                {d[4 * j][2 * i], d[4 * j][2 * i + 1], d[4 * j + 1][2 * i], d[4 * j + 1][2 * i + 1],
                                 d[4 * j + 2][2 * i], d[4 * j + 2][2 * i + 1], d[4 * j + 3][2 * i], d[4 * j + 3][2 * i + 1]});
                        }
                    }
                }
            }
            stage = stage + 1 == kExpandStages ? 0 : stage + 1;
        }
        cp_async_wait<0>();
        __syncthreads();
    }
}

// ---------------------------------------------------------------- launch --
// Rows of a tile of many rows, 16 or 32 to a warp by what its registers hold.
int tile_rows(int R) { return R <= 64 ? 128 : 64; }

// Parts of K: as many as fill the GPU, at least a unit to a warp of each, or four
// stages.  Tiles are estimated from the sizes alone.
int splits_of(int64_t M, int K, int L, int R)
{
    const bool few = M <= kGatherRows;
    const int64_t tiles = few ? std::min<int64_t>(M, L + M / kTile) : ceil_div(M, tile_rows(R));
    const int64_t most = std::min<int64_t>(kMaxSplits, ceil_div(K, few ? kUnit * kWarps : 4 * kChunk));
    return (int)std::max<int64_t>(1, std::min<int64_t>(most, kBlocks / std::max<int64_t>(1, tiles)));
}

template <int NT, int MW, int SLOTS, int STAGES, int THREADS>
int launch_shrink(const Lora &p, cudaStream_t stream)
{
    if (p.M <= kGatherRows)
        return launch_dependent(lora_shrink_few_kernel<NT>, dim3((unsigned)p.M, p.splits), kThreads, 0, stream, p);
    using S = Shrink<NT, MW, SLOTS, STAGES, THREADS>;
    static PerDevice set;
    const int rc = raise_smem(lora_shrink_kernel<NT, MW, SLOTS, STAGES, THREADS>, S::kBytes, set);
    if (rc != EP_OK)
        return rc;
    return launch_dependent(lora_shrink_kernel<NT, MW, SLOTS, STAGES, THREADS>,
                            dim3((unsigned)ceil_div(p.M, S::kRows), p.splits), THREADS, S::kBytes, stream, p);
}

template <int KS, int WIDE, bool BF16_OUT>
int launch_expand_many(const Lora &p, cudaStream_t stream)
{
    static PerDevice set;
    const int rc = raise_smem(lora_expand_kernel<KS, WIDE, BF16_OUT>, kExpandStages * expand_stage(KS, 64 * WIDE), set);
    if (rc != EP_OK)
        return rc;
    const int64_t tiles = ceil_div(p.M, kExpandRows);
    const int64_t pieces = std::max<int64_t>(1, std::min<int64_t>(ceil_div(p.N, kColumns), kBlocks / tiles));
    const int span = (int)(ceil_div(ceil_div(p.N, pieces), kColumns) * kColumns);
    return launch_dependent(lora_expand_kernel<KS, WIDE, BF16_OUT>, dim3((unsigned)tiles, (unsigned)ceil_div(p.N, span)),
                            kThreads, (size_t)kExpandStages * expand_stage(KS, p.base == nullptr ? 0 : 64 * WIDE), stream, p,
                            span);
}

template <int KS>
int launch_expand_many(const Lora &p, cudaStream_t stream)
{
    if (p.base != nullptr && p.base_dtype != 0)
        return p.out_dtype == 0 ? launch_expand_many<KS, 2, true>(p, stream) : launch_expand_many<KS, 2, false>(p, stream);
    return p.out_dtype == 0 ? launch_expand_many<KS, 1, true>(p, stream) : launch_expand_many<KS, 1, false>(p, stream);
}

template <int UNITS, int WORDS>
int launch_expand(const Lora &p, cudaStream_t stream)
{
    if (p.M > kGatherRows)
        return launch_expand_many<UNITS * WORDS / 2>(p, stream);
    return launch_dependent(lora_expand_few_kernel<UNITS, WORDS>,
                            dim3((unsigned)p.M, (unsigned)ceil_div(p.N, 32 * kWarps)), kThreads, 0, stream, p);
}

}  // namespace
}  // namespace ep

using namespace ep;

extern "C" size_t ep_lora_workspace_size(int64_t M, int R)
{
    if (M < 0 || R < 1)
        return 0;
    // splits_of(m) * m is at most this for every m <= M, so that a workspace serves smaller batches too
    const int64_t rows = std::min<int64_t>(kMaxSplits * M, std::max<int64_t>(M, (int64_t)kBlocks * 128));
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
                 scaling, base, out, M, K, N, R, L, splits_of(M, K, L, R), base_dtype, out_dtype, static_cast<float *>(ws),
                 err};
    const int rc = R <= 8 ? launch_shrink<1, 1, 4, 4, 256>(p, stream) : R <= 16 ? launch_shrink<2, 1, 4, 4, 256>(p, stream)
                 : R <= 32 ? launch_shrink<4, 1, 4, 3, 256>(p, stream) : R <= 64 ? launch_shrink<8, 1, 2, 3, 256>(p, stream)
                                                                                 : launch_shrink<16, 1, 1, 4, 128>(p, stream);
    if (rc != EP_OK)
        return rc;
    if (R <= 16)
        return launch_expand<1, 2>(p, stream);
    if (R <= 32)
        return launch_expand<1, 4>(p, stream);
    return R <= 64 ? launch_expand<2, 4>(p, stream) : launch_expand<4, 4>(p, stream);
}
