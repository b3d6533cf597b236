// Low-rank adapters of many requests beside a shared projection:
//
//   out[m] = base[m] + s[a] * B[a] (A[a] x[m]),  a = the adapter of row m.
//
// Two kernels, the second launched while the first drains: `shrink` leaves
// v = A x in parts of K in the workspace, `expand` adds the parts, multiplies by
// B and adds to the base.  v is kept whole between the two products, as the sum of
// three bf16 terms (24 bits), because the matrix step takes bf16.
//
// Rows come in one of three ways, by the sizes (Way):
//   few: a tile is up to 16 rows that name the same adapter, wherever they stand, so that
//     each adapter's weights are read once for 16 rows.  Up to 64 rows each block finds
//     its tile by itself; with more, a block makes a list of them first.
//   many (ep_lora_many.cu): a tile is 128 neighbouring rows, gone over once for each two or
//     four adapters that they name.
//   mixed: each 128 rows that name more than eight adapters by the list, the rest as many; 8192 rows
//     at a time.
//
// What bounds them: few rows, the chain of two dependent launches (24 rows, rank 16,
// 4096 x 4096: 5.4 us, of which the bytes are 0.7); 1024 rows of 64 adapters 21 us;
// many rows, HBM and the start of expand (8192 rows, rank 64, 7168 x 4096: 61 us, 4.1 TB/s).
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
constexpr int kTile = kLoraTile;
// Most rows of which each block finds its tile by itself.  (Of 256 rows of 64 adapters of rank 16, 17.5 us so and 13.2 with a
// list; of 1024, 55 and 23, most of it for the blocks that look at all ids to find that they have no tile.  The list is a
// launch more: 64 rows of 64 adapters 9.0 us without, 96 rows 10.3 with one.)
constexpr int kSearchRows = 64;

// The tile that begins with row m: `mine` is the row index of this lane's slot (lane & 15), or -1; false if no tile
// does.  A tile begins with every 16th row of an adapter.  All threads of the block.
__device__ __forceinline__ bool gather_tile(const Lora &p, int m, int adapter, int &mine)
{
    __shared__ uint32_t same[kSearchRows / 32];
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

// ------------------------------------------------------------------ list --
// The tiles of more rows, by one block: the rows of an adapter (or of none) are counted in
// a table of twice as many places as there are rows, which gives each row its place
// among them, and each adapter its tiles.  The order of tiles, and of rows in them, is as
// it comes: a row's sums do not depend on where it stands.
constexpr int kListThreads = 1024;
constexpr uint32_t kNowhere = 0xffffffffu;

struct Entry {
    int key, count;   // adapter, or -1 for none; -2: a free entry.  Rows, and then the first tile
};

__global__ void __launch_bounds__(kListThreads)
lora_list_kernel(Lora p, int places)
{
    extern __shared__ __align__(16) uint8_t list_room[];
    Entry *const table = reinterpret_cast<Entry *>(list_room);                      // [places]
    uint32_t *const where = reinterpret_cast<uint32_t *>(list_room + places * sizeof(Entry));   // [M]: place, and rank above it
    __shared__ int tiles;
    const int M = (int)p.M, lane = threadIdx.x & 31;
    for (int i = threadIdx.x; i < places; i += kListThreads)
        table[i] = Entry{-2, 0};
    if (threadIdx.x == 0)
        tiles = 0;
    grid_dependency_wait();
    allow_dependents();
    __syncthreads();
    auto add = [&](int r, int key) {   // a whole warp; -2: not in the list
        const uint32_t same = __match_any_sync(kFull, key);
        const int leader = __ffs(same) - 1;
        int at = 0, rank = 0;
        if (lane == leader && key != -2) {
            at = (int)((uint32_t)key * 2654435761u >> 16) & (places - 1);
            for (int i = 0; i < places; ++i) {   // at most half of them are taken
                const int was = atomicCAS(&table[at].key, -2, key);
                if (was == -2 || was == key)
                    break;
                at = (at + 1) & (places - 1);
            }
            rank = atomicAdd(&table[at].count, __popc(same));
        }
        at = __shfl_sync(kFull, at, leader);
        rank = __shfl_sync(kFull, rank, leader) + __popc(same & lanemask_lt());
        if (r < M)
            where[r] = key == -2 ? kNowhere : (uint32_t)rank << 14 | (uint32_t)at;
    };
    // a warp takes 32 rows, or the 128 of a tile of the other kernels, which it may leave to them
    constexpr int kEach = kLoraWide / 32;
    const int warp = threadIdx.x >> 5, each = p.mixed ? kEach : 1;
    bool some = false;
    for (int m = warp * each * 32; m < M; m += kListThreads * each) {
        int keys[kEach];
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int r = m + i * 32 + lane;
            keys[i] = i < each && r < M ? adapter_of(p, r) : -2;
            if (i < each && r < M && bad_id(p, r))
                raise(p.err, EP_ERR_INVALID_EXPERT);
        }
        const bool theirs = p.mixed && !many_adapters(keys);
        some |= !theirs;
#pragma unroll
        for (int i = 0; i < kEach; ++i)
            if (i < each)
                add(m + i * 32 + lane, theirs ? -2 : keys[i]);
    }
    if (!__syncthreads_or(some)) {
        if (threadIdx.x == 0)
            *p.list = 0;
        return;
    }
    int *const adapters = p.list + 1, *const rows = adapters + M;
    for (int i = threadIdx.x; i < places; i += kListThreads) {
        const Entry e = table[i];
        if (e.key == -2)
            continue;
        const int n = (e.count + kTile - 1) / kTile, from = atomicAdd(&tiles, n);
        for (int t = 0; t < n; ++t)
            adapters[from + t] = e.key;
        for (int j = e.count; j < n * kTile; ++j)
            rows[from * kTile + j] = -1;
        table[i].count = from;
    }
    __syncthreads();
    for (int r = threadIdx.x; r < M; r += kListThreads)
        if (where[r] != kNowhere)
            rows[table[where[r] & 0x3fffu].count * kTile + (int)(where[r] >> 14)] = r;
    if (threadIdx.x == 0)
        *p.list = tiles;
}

// Where a block of the kernels for few rows has its tiles from: each row that begins one, a list of which it takes one, or
// one of which it takes several.
enum Source { kSearch, kList, kLists };

// This lane's row (lane & 15) of tile m, or -1; false if there is none.  With a list it is its tile m; without, that
// which begins with row m.
template <int FROM>
__device__ __forceinline__ bool tile_of(const Lora &p, int m, int adapter, int &mine)
{
    if (FROM != kSearch) {
        mine = p.list[1 + p.M + m * kTile + (threadIdx.x & (kTile - 1))];
        return true;
    }
    mine = (threadIdx.x & (kTile - 1)) == 0 ? m : -1;
    return adapter < 0 || gather_tile(p, m, adapter, mine);
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
    // Units whose x is loaded together, and which are summed by matrix steps alone: as many as leave registers for the
    // ranks' loads ahead (24 rows of rank 64 8.8 us with one, 9.4 with two and 10.5 with four; of rank 128 13.0 with two, 13.4
    // with one and 14.5 with four).
    constexpr int kBatch = NT == 16 ? 2 : NT == 8 ? 1 : 4;
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

// A block takes tiles of a list (or one, without) and a part of K, its warps an eighth of that each.
// Registers for two blocks to an SM up to rank 64, which fill it with loads: 2048 rows of 64 adapters of rank 64 in 53 us
// instead of 76, as the compiler by itself left room for one, and 24 of rank 16 in 5.6 instead of 6.8, where it left
// some for four.  Lists of long batches, of rank 16, are faster with four: 8192 rows 106 us, with two 131.
template <int NT, int FROM>
__global__ void __launch_bounds__(kThreads, FROM == kLists && NT <= 2 ? 4 : NT <= 8 ? 2 : 1)
lora_shrink_few_kernel(Lora p)
{
    __shared__ __align__(16) float kept[kWarps / 2][NT * 32 * 4];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    grid_dependency_wait();
    allow_dependents();
    const int units = (p.K + kUnit - 1) / kUnit, all = p.splits * kWarps, part = blockIdx.y * kWarps + warp;
    const int u0 = (int)((int64_t)units * part / all), u1 = (int)((int64_t)units * (part + 1) / all);
    const int tiles = FROM != kSearch ? *p.list : (int)p.M;
    for (int m = blockIdx.x; m < tiles; m = FROM == kLists ? m + gridDim.x : tiles) {
        const int adapter = FROM != kSearch ? p.list[1 + m] : adapter_of(p, m);
        if (adapter < 0) {
            if (FROM == kSearch && threadIdx.x == 0 && blockIdx.y == 0 && bad_id(p, m))
                raise(p.err, EP_ERR_INVALID_EXPERT);
            continue;
        }
        int mine;
        if (!tile_of<FROM>(p, m, adapter, mine))
            continue;
        const int m0 = __shfl_sync(kFull, mine, lane >> 2), m1 = __shfl_sync(kFull, mine, (lane >> 2) + 8);
        float acc[NT][4] = {};
        product<NT>(acc, m0 < 0 ? nullptr : p.x + (int64_t)m0 * p.K * 2, m1 < 0 ? nullptr : p.x + (int64_t)m1 * p.K * 2,
                    p.a + (int64_t)adapter * p.R * p.K * 2, p.R, p.K, u0, u1);
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

// A block takes tiles of a list (or, without, one, or a row without an adapter) and 256 columns.
// Column g of block j of a warp's 32 stands for column n0 + 8 (g / 2) + 2 j + g % 2, so that a
// lane ends up with eight neighbouring columns of each of its rows.  The block makes v once, in
// shared memory.
// Registers for three blocks to an SM up to rank 32, two of more: 2048 rows of 9 adapters of rank 16 in 25 us with three and 29
// with as many as the compiler takes, of rank 128 66 with two and 87; of rank 64 41 either way.
template <int UNITS, int WORDS, int FROM>
__global__ void __launch_bounds__(kThreads, UNITS == 1 ? (FROM == kLists ? 4 : 3) : UNITS == 2 ? 1 : 2)
lora_expand_few_kernel(Lora p)
{
    constexpr int kRanks = UNITS * WORDS * 8, kVRow = kRanks * 2 + 16;   // bytes of a row of v
    __shared__ __align__(16) uint8_t v_room[kPlanes][kTile][kVRow];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    // Every block of shrink has waited for what was before it, so that only what shrink itself writes is waited for here.
    const int n0 = (blockIdx.y * kWarps + warp) * 32, n = n0 + 8 * t;
    const bool bf16_base = p.base_dtype == 0, bf16_out = p.out_dtype == 0;
    const int tiles = FROM != kSearch ? *p.list : (int)p.M;
    for (int m = blockIdx.x; m < tiles; m = FROM == kLists ? m + gridDim.x : tiles) {
        const int adapter = FROM != kSearch ? p.list[1 + m] : adapter_of(p, m);
        Ranks<UNITS, WORDS> b[4];
        auto load_b = [&]() {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int row = n0 + 8 * (g >> 1) + 2 * j + (g & 1);
                b[j].load(adapter >= 0 && row < p.N ? p.b + ((int64_t)adapter * p.N + row) * p.R * 2 : nullptr, p.R);
            }
        };
        load_b();   // nothing waits for the tile's rows
        int mine;
        if (!tile_of<FROM>(p, m, adapter, mine))
            continue;
        const int m0 = __shfl_sync(kFull, mine, g), m1 = __shfl_sync(kFull, mine, g + 8);
        Base base0, base1;
        base0.load(p, m0, n);
        base1.load(p, m1, n);
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
        auto at = [&](int m) { return static_cast<uint8_t *>(p.out) + ((int64_t)m * p.N + n) * (bf16_out ? 2 : 4); };
        if (m0 >= 0 && n < p.N)
            put(at(m0), bf16_base, bf16_out, base0, {d[0][0], d[0][1], d[1][0], d[1][1], d[2][0], d[2][1], d[3][0], d[3][1]});
        if (m1 >= 0 && n < p.N)
            put(at(m1), bf16_base, bf16_out, base1, {d[0][2], d[0][3], d[1][2], d[1][3], d[2][2], d[2][3], d[3][2], d[3][3]});
        if (FROM == kLists)
            __syncthreads();   // before v is made again
    }
    grid_dependency_wait();   // also without a tile: what follows waits for all before it through this kernel
}

// ---------------------------------------------------------------- launch --
// Kernels for few rows alone, for many alone, or both: each tile of 128 rows by the one or the other.  Measured with
// 4096 x 4096 in us, few / many / both:
//                        rank 16                          rank 64
//   rows    1 adapter      64 at random        1 adapter      64 at random
//   512     11 / 11 / 18   15 / 128 / 22       15 / 15 / 22   29 / 197 / 42
//   768     12 / 12 / 19   18 / 165 / 24       19 / 17 / 24   33 / 238 / 45
//   1024    15 / 13 / 19   21 / 164 / 32       23 / 18 / 25   36 / 236 / 55
//   2048    25 / 18 / 27   31 / 259 / 45       40 / 23 / 32   57 / 333 / 76
//   8192    82 / 44 / 55   93 / 875 / 106      141 / 50 / 63  156 / 1033 / 189
// Many alone where no tile can name more than eight (8192 rows of 8 at random: 84 / 165 and 142 / 187).
enum Way { kFew, kMany, kMixed };

Way way_of(int64_t M, int L)
{
    if (M <= 768 || (M <= 2048 && L > kLoraMostAdapters))
        return kFew;
    return L <= kLoraMostAdapters ? kMany : kMixed;
}

// Parts of K: as many as fill the GPU, at least a unit to a warp of each, or 256
// columns of many rows, and no more than are worth reading again by each block of expand:
// 1 row of rank 16 takes 4.8 us with up to 8 and 5.2 with 16, 1024 rows of rank 64 18.6 and 20.3
// (20.1 with 4); 4096 rows of rank 128 47 with 4 and 55 with 8.  Tiles are estimated from the sizes alone.
int splits_of(int64_t M, int K, int L, int R)
{
    const int64_t tiles = way_of(M, L) == kFew ? std::min<int64_t>(M, L + M / kTile) : ceil_div(M, 128);
    const int64_t most = std::min<int64_t>(way_of(M, L) != kFew && R > 64 ? 4 : kLoraMaxSplits, ceil_div(K, 256));
    return (int)std::max<int64_t>(1, std::min<int64_t>(most, kLoraBlocks / std::max<int64_t>(1, tiles)));
}

size_t list_bytes(int64_t M)
{
    return align_up((1 + (size_t)std::min<int64_t>(M, kLoraListRows) * (1 + kTile)) * sizeof(int), kWsAlign);
}

// f with the kernels' shapes of a rank as constants: eights of ranks, and units and words of B's.
template <class F>
int with_rank(int R, F &&f)
{
    using std::integral_constant;
    if (R <= 8)
        return f(integral_constant<int, 1>(), integral_constant<int, 1>(), integral_constant<int, 2>());
    if (R <= 16)
        return f(integral_constant<int, 2>(), integral_constant<int, 1>(), integral_constant<int, 2>());
    if (R <= 32)
        return f(integral_constant<int, 4>(), integral_constant<int, 1>(), integral_constant<int, 4>());
    if (R <= 64)
        return f(integral_constant<int, 8>(), integral_constant<int, 2>(), integral_constant<int, 4>());
    return f(integral_constant<int, 16>(), integral_constant<int, 4>(), integral_constant<int, 4>());
}

// Blocks for a list's tiles, in `pieces` each: as many as it may have; where it may as well have none, no more than
// run at a time.
unsigned blocks_of(const Lora &p, int64_t pieces)
{
    const int64_t most = std::min<int64_t>(p.M, (int64_t)p.L + 1 + p.M / kTile);
    return (unsigned)(p.mixed ? std::min<int64_t>(most, ceil_div(2 * kLoraBlocks, pieces)) : most);
}

int launch_list(const Lora &p, cudaStream_t stream)
{
    static PerDevice set;
    int places = 2 * kSearchRows;
    while (places < 2 * p.M)
        places *= 2;
    const int rc = raise_smem(lora_list_kernel, kLoraListRows * (2 * sizeof(Entry) + sizeof(int)), set);
    if (rc != EP_OK)
        return rc;
    return launch_dependent(lora_list_kernel, dim3(1), kListThreads, places * sizeof(Entry) + p.M * sizeof(int), stream, p,
                            places);
}

int launch_shrink_few(const Lora &p, bool list, cudaStream_t stream)
{
    return with_rank(p.R, [&](auto nt, auto, auto) {
        constexpr int NT = decltype(nt)::value;
        const dim3 grid(list ? blocks_of(p, p.splits) : (unsigned)p.M, p.splits);
        return launch_dependent(p.mixed ? lora_shrink_few_kernel<NT, kLists> : list ? lora_shrink_few_kernel<NT, kList>
                                                                                    : lora_shrink_few_kernel<NT, kSearch>,
                                grid, kThreads, 0, stream, p);
    });
}

int launch_expand_few(const Lora &p, bool list, cudaStream_t stream)
{
    return with_rank(p.R, [&](auto, auto units, auto words) {
        constexpr int U = decltype(units)::value, W = decltype(words)::value;
        const int64_t pieces = ceil_div(p.N, 32 * kWarps);
        const dim3 grid(list ? blocks_of(p, pieces) : (unsigned)p.M, (unsigned)pieces);
        return launch_dependent(p.mixed ? lora_expand_few_kernel<U, W, kLists> : list ? lora_expand_few_kernel<U, W, kList>
                                                                                      : lora_expand_few_kernel<U, W, kSearch>,
                                grid, kThreads, 0, stream, p);
    });
}

int launch_lora(const Lora &p, Way way, cudaStream_t stream)
{
    const bool list = p.M > kSearchRows;
    int rc = way != kMany && list ? launch_list(p, stream) : EP_OK;
    if (rc == EP_OK && way != kMany)
        rc = launch_shrink_few(p, list, stream);
    if (rc == EP_OK && way != kFew)
        rc = launch_lora_shrink_many(p, stream);
    if (rc == EP_OK && way != kMany)
        rc = launch_expand_few(p, list, stream);
    if (rc == EP_OK && way != kFew)
        rc = launch_lora_expand_many(p, stream);
    return rc;
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
    return list_bytes(M) + align_up((size_t)rows * R * sizeof(float), kWsAlign) + kWsAlign;
}

extern "C" int ep_lora(const void *x, int64_t M, int K, const int64_t *ids, const void *a, const void *b,
                       const float *scaling, int L, int R, int N, const void *base, int base_dtype, void *out,
                       int out_dtype, void *ws, size_t ws_bytes, int32_t *err, ep_stream_t stream_)
{
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    if (M < 0 || K < 8 || K % 8 != 0 || N < 8 || N % 8 != 0 || R < 8 || R % 8 != 0 || L < 1)
        return EP_ERR_INVALID_ARG;
    if ((out_dtype != 0 && out_dtype != 1) || (base != nullptr && base_dtype != 0 && base_dtype != 1) || R > kLoraMaxRank ||
        K > (1 << 23) || N > (1 << 23) || M > (1 << 24))
        return EP_ERR_UNSUPPORTED;
    if (M == 0)
        return EP_OK;
    if (x == nullptr || ids == nullptr || a == nullptr || b == nullptr || out == nullptr || !aligned(x, 16) ||
        !aligned(a, 16) || !aligned(b, 16) || !aligned(base, 16) || !aligned(out, 16) || !aligned(ids, 8) ||
        !aligned(scaling, 4) || !aligned(err, 4) || (out == base && base_dtype != out_dtype) || ws == nullptr ||
        !aligned(ws, kWsAlign) || ws_bytes < ep_lora_workspace_size(M, R))
        return EP_ERR_INVALID_ARG;
    // the longest list at a time; what is in the workspace is of one piece, as the next waits for its end
    const int64_t step = L <= kLoraMostAdapters ? M : kLoraListRows;
    for (int64_t m = 0; m < M; m += step) {
        const int64_t rows = std::min(step, M - m);
        const Way way = way_of(rows, L);
        const Lora p{static_cast<const uint8_t *>(x) + m * K * 2, static_cast<const uint8_t *>(a),
                     static_cast<const uint8_t *>(b), ids + m, scaling,
                     base == nullptr ? nullptr : static_cast<const uint8_t *>(base) + m * N * (base_dtype == 0 ? 2 : 4),
                     static_cast<uint8_t *>(out) + m * N * (out_dtype == 0 ? 2 : 4), rows, K, N, R, L,
                     splits_of(rows, K, L, R), base_dtype, out_dtype,
                     reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + list_bytes(rows)), static_cast<int *>(ws),
                     way == kMixed, err};
        const int rc = launch_lora(p, way, stream);
        if (rc != EP_OK)
            return rc;
    }
    return EP_OK;
}
