// Low-rank adapters for many rows.
//
// Tiles of 128 neighbouring rows, on tcgen05 matrix steps of 128 x N.  A tile's rows may
// name several adapters: they are taken a few at a time (a pass), side by side as N, so that
// every row has a product with each of them, and each row keeps its own.  (One
// adapter's infinities never meet another's rows.)  What a pass does not need is
// not loaded.
//
//   shrink: x and the adapters' A come 64 columns at a time through a ring; the tensor
//     memory's sums are taken into registers after every 128 columns and added there
//     with IEEE operations, as a long chain of matrix steps loses bits.
//   expand: v is made once for a tile, as three bf16 terms, and stays in shared
//     memory; B comes 64 or 128 columns at a time, up to three chunks ahead; the base comes
//     in boxes of 32 rows and 32 columns through a ring of each warp's own, where the sums
//     are added to it and from where they leave as such a box (by tensor maps), or in pieces
//     of rows where some of the 32 are another pass's.
//
// Measured with 8192 rows of 8 adapters of rank 64, 7168 x 4096, bf16: shrink 25 us (the bytes
// of x alone: 17), expand 37 (base and result: 20), of which making v from its parts takes 4.
// With the base copied by cp.async and the results stored by the lanes, expand took 42 us:
// the copies alone took each warp 1300 to 1700 cycles of a chunk's 4000 to issue.  With two
// stages of B instead of four for one adapter's tiles, a chunk took 3300 cycles instead of
// 2500.  Eight warps of 64 columns instead of 16 of 32: 66 us in all instead of 62.
//
// x, A and B come by TMA (tensor maps of x [M,K], A [L,R,K] and B [L,N,R], whose
// edges read as zeros) with the 128-byte swizzle that the matrix steps take.  Copied by
// cp.async instead, with a proxy fence by the threads that copied, both kernels waited
// at that fence for the copies still in flight.  Waits on barriers give up after a
// second or so (EP_ERR_TIMEOUT).
#include <algorithm>
#include <atomic>

#include <cuda.h>
#include <cudaTypedefs.h>

#include "ep_device.cuh"
#include "ep_internal.h"
#include "ep_launch.cuh"
#include "ep_lora.cuh"
#include "ep_skinny.cuh"
#include "ep_tensor.cuh"

namespace ep {
namespace {

constexpr int kRows = kLoraWide;     // of a tile
constexpr int kTries = 1 << 16;      // of a wait, each of which may sleep for 20 us

__device__ __forceinline__ int adapter_after(const int *ids, int last)
{
    int mine[kRows / 32];
#pragma unroll
    for (int i = 0; i < kRows / 32; ++i)
        mine[i] = ids[i * 32 + (threadIdx.x & 31)];
    return next_adapter(mine, last);
}

// Whether the kernels for few rows have this tile.  The same in every warp.
__device__ __forceinline__ bool left_to_few(const Lora &p, const int *ids)
{
    if (!p.mixed)
        return false;
    int mine[kRows / 32];
#pragma unroll
    for (int i = 0; i < kRows / 32; ++i)
        mine[i] = ids[i * 32 + (threadIdx.x & 31)];
    return many_adapters(mine);
}

// The adapters of a pass: up to SLOTS in ascending order, and the first that is left for the next pass.
template <int SLOTS>
struct Pass {
    int slot[SLOTS], slots, next;

    __device__ __forceinline__ void set(const int *ids, int first)
    {
        next = first;
        slots = 0;
#pragma unroll
        for (int i = 0; i < SLOTS; ++i) {
            slot[i] = next;
            if (next != kNoRow) {
                ++slots;
                next = adapter_after(ids, next);
            }
        }
    }

    __device__ __forceinline__ bool has(int id) const { return id >= slot[0] && id < next; }

    // the slots that the lanes' adapters name
    __device__ __forceinline__ uint32_t mask(int id) const
    {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < SLOTS; ++i)
            m |= (i < slots && id == slot[i] ? 1u : 0u) << i;
        return __reduce_or_sync(kFull, m);
    }

    __device__ __forceinline__ int id_of(int i) const
    {
        int id = slot[0];
#pragma unroll
        for (int j = 1; j < SLOTS; ++j)
            id = i == j ? slot[j] : id;
        return id;
    }
};

// One thread waits for the n-th use of a barrier that is completed once a use; false (once and for all) after kTries.
// It sleeps while it waits: spinning warps take the issue slots of those that they wait for.
__device__ __forceinline__ bool wait_alone(uint64_t *bar, int n, volatile int *failed)
{
    for (int i = 0; i < kTries; ++i) {
        uint32_t ok;
        asm volatile("{\n\t.reg .pred p;\n\t"
                     "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
                     "selp.u32 %0, 1, 0, p;\n\t}"
                     : "=r"(ok)
                     : "r"(smem_u32(bar)), "r"((uint32_t)n & 1u), "r"(20000u)
                     : "memory");
        if (ok != 0)
            return true;
    }
    *failed = 1;
    return false;
}

// A whole warp waits, by one lane.  The way out of a wait that failed leaves the caller's loop, so that lanes which got
// through at different times would meet again only behind it: the vote brings them together for the .aligned
// instructions here.
__device__ __forceinline__ bool wait_for(uint64_t *bar, int n, volatile int *failed)
{
    const bool ok = (threadIdx.x & 31) != 0 || wait_alone(bar, n, failed);
    return __all_sync(kFull, ok);
}

// After a wait that failed: what this thread has on its way, copies of the last `stages` of `copied` uses and steps of as
// many of `stepped` ones, ends before the block does, within the waits' limits.
__device__ __forceinline__ void drain(uint64_t *full, uint64_t *empty, int stages, int copied, int stepped,
                                      volatile int *failed)
{
    for (int use = max(0, copied - stages); use < copied; ++use)
        wait_alone(&full[use % stages], use / stages, failed);
    for (int use = max(0, stepped - stages); use < stepped; ++use)
        wait_alone(&empty[use % stages], use / stages, failed);
}

// ---------------------------------------------------------------- shrink --
constexpr int kFlushWarps = 4, kShrinkThreads = kFlushWarps * 32 + 64;
constexpr int kChunk = 64;      // columns of x a stage
constexpr int kGroup = 2;       // stages of a sum

template <int RP, int SLOTS, int STAGES>
struct Shrink {
    static constexpr int kX = kRows * 128, kN = SLOTS * RP, kStage = kX + kN * 128;
    static constexpr int kColumns = 2 * kN;                      // of tensor memory
    static constexpr int kBytes = STAGES * kStage + 1024;        // and room to align
};

template <int RP, int SLOTS, int STAGES>
__global__ void __launch_bounds__(kShrinkThreads, RP <= 64 ? 2 : 1)
lora_shrink_many_kernel(Lora p, const __grid_constant__ CUtensorMap x_map, const __grid_constant__ CUtensorMap a_map)
{
    using S = Shrink<RP, SLOTS, STAGES>;
    constexpr int kLoad = RP < 32 ? RP : 32;   // columns of tensor memory a load
    extern __shared__ uint8_t dynamic[];
    __shared__ int ids[kRows];
    __shared__ uint64_t full[STAGES], empty[STAGES], done[2], taken[2];
    __shared__ uint32_t tensor;
    __shared__ int failed;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t first = (int64_t)blockIdx.x * kRows;
    const uint32_t ring = (smem_u32(dynamic) + 1023u) & ~1023u;
    grid_dependency_wait();
    if (threadIdx.x < kRows) {
        const int64_t m = first + threadIdx.x;
        ids[threadIdx.x] = m < p.M ? adapter_of(p, m) : -1;
        if (blockIdx.y == 0 && m < p.M && bad_id(p, m))
            raise(p.err, EP_ERR_INVALID_EXPERT);
    }
    if (threadIdx.x == 0) {
        failed = 0;
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&done[i], 1);
            mbar_init(&taken[i], kFlushWarps);
        }
        fence_mbar_init();
    }
    __syncthreads();
    if (left_to_few(p, ids))
        return;
    if (warp == kFlushWarps + 1)
        tensor_alloc(&tensor, S::kColumns);
    tensor_fence_before();
    __syncthreads();
    tensor_fence_after();
    allow_dependents();   // with its tensor memory in hand
    const int chunks = (p.K + kChunk - 1) / kChunk;
    const int c0 = (int)((int64_t)chunks * blockIdx.y / p.splits), c1 = (int)((int64_t)chunks * (blockIdx.y + 1) / p.splits);
    int used = 0, summed = 0;   // stages and sums so far
    Pass<SLOTS> pass;
    if (warp < kFlushWarps) {
        // a row to a thread
        const int id = ids[threadIdx.x];
        const int64_t m = first + threadIdx.x;
        for (int now = adapter_after(ids, -1); now != kNoRow; now = pass.next) {
            pass.set(ids, now);
            const uint32_t mine = pass.mask(id);
            float acc[RP] = {};
            for (int c = c0; c < c1; c += kGroup, ++summed) {
                const int buf = summed & 1;
                if (!wait_for(&done[buf], summed >> 1, &failed))
                    break;
                tensor_fence_after();
                for (uint32_t todo = mine; todo != 0; todo &= todo - 1u) {
                    const int slot = __ffs(todo) - 1;
                    const bool own = id == pass.id_of(slot);
                    const uint32_t at = tensor + ((uint32_t)(warp * 32) << 16) + buf * S::kN + slot * RP;
#pragma unroll
                    for (int j = 0; j < RP; j += kLoad) {
                        float f[kLoad];
                        tensor_load<kLoad>(f, at + j);
                        if (own)
#pragma unroll
                            for (int i = 0; i < kLoad; ++i)
                                acc[j + i] = __fadd_rn(acc[j + i], f[i]);
                    }
                }
                tensor_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&taken[buf]);
            }
            if (__any_sync(kFull, failed))
                break;
            if (pass.has(id)) {
                float *to = p.parts + ((int64_t)blockIdx.y * p.M + m) * p.R;
#pragma unroll
                for (int r = 0; r < RP; r += 4)
                    if (r < p.R)
                        *reinterpret_cast<float4 *>(to + r) = make_float4(acc[r], acc[r + 1], acc[r + 2], acc[r + 3]);
            }
        }
    } else if (warp == kFlushWarps) {
        for (int now = adapter_after(ids, -1); now != kNoRow; now = pass.next) {
            pass.set(ids, now);
            if (lane == 0)
                for (int c = c0; c < c1; ++c, ++used) {
                    const int at = used % STAGES;
                    if (used >= STAGES && !wait_alone(&empty[at], used / STAGES - 1, &failed))
                        break;
                    const uint32_t to = ring + at * S::kStage;
                    mbar_arrive_expect_tx(&full[at], S::kX + pass.slots * RP * 128);
                    tensor_copy(to, &x_map, c * kChunk, (int)first, 0, &full[at]);
#pragma unroll
                    for (int i = 0; i < SLOTS; ++i)
                        if (i < pass.slots)
                            tensor_copy(to + S::kX + i * RP * 128, &a_map, c * kChunk, 0, pass.slot[i], &full[at]);
                }
            __syncwarp();
            if (__any_sync(kFull, failed))
                break;
        }
        if (lane == 0 && failed)
            drain(full, empty, STAGES, used, 0, &failed);
    } else {
        for (int now = adapter_after(ids, -1); now != kNoRow; now = pass.next) {
            pass.set(ids, now);
            const uint32_t kind = step_kind(pass.slots * RP);
            if (lane == 0)
                for (int c = c0; c < c1; ++c, ++used) {
                    const int at = (c - c0) % kGroup, buf = summed & 1;
                    if ((at == 0 && summed >= 2 && !wait_alone(&taken[buf], (summed >> 1) - 1, &failed)) ||
                        !wait_alone(&full[used % STAGES], used / STAGES, &failed))
                        break;
                    tensor_fence_after();
                    const uint32_t stage = ring + (used % STAGES) * S::kStage;
                    const uint64_t x = tile_descriptor(stage), a = tile_descriptor(stage + S::kX);
#pragma unroll
                    for (int k = 0; k < kChunk / 16; ++k)
                        tensor_step(tensor + buf * S::kN, x + 2 * k, a + 2 * k, kind, at != 0 || k != 0);
                    tensor_commit(&empty[used % STAGES]);
                    if (at == kGroup - 1 || c + 1 == c1) {
                        tensor_commit(&done[buf]);
                        ++summed;
                    }
                }
            __syncwarp();
            if (__any_sync(kFull, failed))
                break;
        }
        if (lane == 0 && failed)
            drain(full, empty, STAGES, 0, used, &failed);
    }
    __syncthreads();
    if (failed && threadIdx.x == 0)
        raise(p.err, EP_ERR_TIMEOUT);
    __syncwarp();
    if (warp == kFlushWarps + 1)
        tensor_free(tensor, S::kColumns);
}

// ---------------------------------------------------------------- expand --
constexpr int kExpandSlots = 2, kBStages = 4;   // stages of B, each of one adapter

// STEPS: of 16 ranks, 8 of them in two runs of 64.  BASE, OUT: bytes of an element.
//
// A step reads the 128 rows of v, which takes it some 70 cycles whatever its N: chunks are as wide as there is room
// for.  (Of 32 columns, with two blocks to an SM, the steps alone took 1700 of the 1350 cycles that a pair of
// chunks' bytes take.)
template <int STEPS, int BASE, int OUT>
struct Expand {
    static constexpr int kRuns = STEPS > 4 ? 2 : 1;
    static constexpr int kN = kRuns == 1 && BASE == 2 && OUT == 2 ? 128 : 64;  // columns of a chunk
    static constexpr int kSumWarps = kN / 8, kThreads = kSumWarps * 32 + 32;   // 32 rows and 32 columns to a warp
    static constexpr int kV = kRows * 128;                                     // a term of v, 64 ranks
    static constexpr int kB = kN * 128;                                        // a stage of B, 64 ranks
    static constexpr int kBaseRow = 32 * BASE, kOutRow = 32 * OUT;             // bytes
    static constexpr int kRoom = 32 * (BASE > OUT ? kBaseRow : kOutRow);       // a warp's stage
    static constexpr int kFixed = kPlanes * kRuns * kV + kBStages * kRuns * kB + 1024;
    static constexpr int kFit = (225 * 1024 - kFixed) / (kSumWarps * kRoom);
    static constexpr int kRowStages = kFit < 4 ? kFit : 4;
    // chunks of the base ahead; results that may still be on their way when a stage is filled again
    static constexpr int kAhead = kRowStages > 3 ? 2 : 1, kLeaving = kRowStages - 1 - kAhead;
    static constexpr int kBytes = kFixed + kRowStages * kSumWarps * kRoom;
    static constexpr int kTensor = 2 * kExpandSlots * kN;                      // columns of tensor memory
};

// Where a tensor map of rows of ROW bytes (swizzled in as many) leaves a row's 16-byte piece.
template <int ROW>
__device__ __forceinline__ uint32_t piece_at(int row, int i)
{
    static_assert(ROW == 128 || ROW == 64, "bytes of a row");
    return row * ROW + ((i ^ (ROW == 128 ? row & 7 : row >> 1 & 3)) << 4);
}

// Each of the warps but the last takes 32 rows and 32 columns of every chunk's sums; the last copies B and issues the
// matrix steps.
template <int STEPS, int BASE, int OUT>
__global__ void __launch_bounds__((Expand<STEPS, BASE, OUT>::kThreads), 1)
lora_expand_many_kernel(Lora p, const __grid_constant__ CUtensorMap b_map, const __grid_constant__ CUtensorMap base_map,
                        const __grid_constant__ CUtensorMap out_map, int span)
{
    using S = Expand<STEPS, BASE, OUT>;
    constexpr int kRuns = S::kRuns, kN = S::kN, kSumWarps = S::kSumWarps, kStages = S::kRowStages;
    extern __shared__ uint8_t dynamic[];
    __shared__ int ids[kRows];
    __shared__ float scales[kRows];
    __shared__ uint64_t full[kBStages], empty[kBStages], done[2], taken[2], here[kSumWarps][kStages];
    __shared__ uint32_t tensor;
    __shared__ int failed;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t first = (int64_t)blockIdx.x * kRows;
    const uint32_t v_at = (smem_u32(dynamic) + 1023u) & ~1023u, b_at = v_at + kPlanes * kRuns * S::kV;
    const uint32_t rows_at = b_at + kBStages * kRuns * S::kB;
    const int n_from = blockIdx.y * span, n_to = min(n_from + span, p.N);
    const int chunks = (n_to - n_from + kN - 1) / kN;
    // Every block of shrink has waited for what was before it, so that only what shrink itself writes is waited for here.
    if (threadIdx.x < kRows) {
        const int id = first + threadIdx.x < p.M ? adapter_of(p, first + threadIdx.x) : kNoRow;
        ids[threadIdx.x] = id;
        scales[threadIdx.x] = id == kNoRow ? 1.0f : scaling_of(p, id);
    }
    if (threadIdx.x == 0) {
        failed = 0;
        for (int i = 0; i < kBStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&done[i], 1);
            mbar_init(&taken[i], kSumWarps);
        }
        for (int i = 0; i < kSumWarps * kStages; ++i)
            mbar_init(&here[0][0] + i, 1);
        fence_mbar_init();
    }
    __syncthreads();
    if (left_to_few(p, ids)) {
        grid_dependency_wait();   // what follows waits for all that is before it through this kernel
        return;
    }
    Pass<kExpandSlots> pass;
    // a row to a thread; the columns from column0 on of each chunk
    const int column0 = (warp >> 2) * 32, mine0 = (warp & 3) * 32, id = ids[mine0 + lane];
    const uint32_t room = rows_at + warp * kStages * S::kRoom;
    uint32_t rows = 0, mine = 0;   // of the pass: rows of these 32, and the slots that they name
    bool one = false;              // they name one, and each does
    bool whole = false;            // no other row of the batch is among the 32
    int taken_in = 0, fetched = 0; // stages of the rows so far; of the base copied, by the one lane
    auto fetch = [&](int c, int use) {   // one lane
        if (p.base != nullptr && c < chunks) {
            uint64_t *bar = &here[warp][use % kStages];
            mbar_arrive_expect_tx(bar, 32 * S::kBaseRow);
            tensor_copy(room + use % kStages * S::kRoom, &base_map, n_from + c * kN + column0, (int)first + mine0, 0, bar);
            fetched = use + 1;
        }
    };
    auto begin = [&](int now, bool start) {
        pass.set(ids, now);
        if (warp >= kSumWarps)
            return;
        // rows without an adapter go along with the first pass
        const bool in = pass.has(id) || (start && id == -1);
        rows = __ballot_sync(kFull, in);
        whole = __all_sync(kFull, in || id == kNoRow);
        mine = pass.mask(id);
        one = mine != 0 && (mine & (mine - 1u)) == 0 && !__any_sync(kFull, in && id == -1);
        if (lane == 0 && rows != 0) {
            bulk_wait_read<0>();
            for (int i = 0; i < S::kAhead; ++i)
                fetch(i, taken_in + i);
        }
    };
    // One thread copies B, ahead by all stages but one that the pass's adapters leave: four, or two of two adapters each.
    int used = 0, copied = 0, stepped = 0;   // chunks: of passes before; of B copied, and with their steps issued
    auto copy = [&](int c) {
        const int use = used + c, stages = kBStages / pass.slots;
        const int last = c < stages ? used - 1 : use - stages;   // whose steps have to be done
        if (last >= 0 && !wait_alone(&empty[last % kBStages], last / kBStages, &failed))
            return false;
        uint64_t *const bar = &full[use % kBStages];
        mbar_arrive_expect_tx(bar, pass.slots * kRuns * kN * 128);
        copied = use + 1;
        const uint32_t to = b_at + c % stages * pass.slots * (kRuns * S::kB);
#pragma unroll
        for (int b = 0; b < kRuns; ++b)
#pragma unroll
            for (int i = 0; i < kExpandSlots; ++i)
                if (i < pass.slots)
                    tensor_copy(to + (b * pass.slots + i) * S::kB, &b_map, b * 64, n_from + c * kN, pass.slot[i], bar);
        return true;
    };
    auto copy_first = [&]() {
        for (int c = 0; c < min(chunks, kBStages / pass.slots - 1); ++c)
            if (!copy(c))
                return false;
        return true;
    };
    begin(adapter_after(ids, -1), true);
    if (warp == kSumWarps && lane == 0 && pass.slots > 0)
        copy_first();
    __syncwarp();
    grid_dependency_wait();
    // not before: a block that held tensor memory while it waits for shrink could keep it from shrink
    if (warp == kSumWarps)
        tensor_alloc(&tensor, S::kTensor);
    allow_dependents();
    if (warp < kSumWarps) {   // v of every row: a thread has four ranks of several rows, whose parts are loaded together
        constexpr int kFours = STEPS * 4, kApart = kSumWarps * 32 / kFours;
        constexpr int kEach = kRows / kApart, kBatch = kEach < 4 ? kEach : kSumWarps > 8 ? 2 : 4;
        const int r = threadIdx.x % kFours * 4, row0 = threadIdx.x / kFours;
        const int64_t next = p.M * p.R / 4;
#pragma unroll 1
        for (int i = 0; i < kEach; i += kBatch) {
            const float4 *part[kBatch];
            float4 f[kBatch];
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const int row = row0 + (i + j) * kApart, a = ids[row];
                part[j] = a >= 0 && a != kNoRow && r < p.R
                              ? reinterpret_cast<const float4 *>(p.parts + (first + row) * p.R + r) : nullptr;
                f[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            }
#pragma unroll 1
            for (int z = 0; z < p.splits; z += 4) {
                float4 u[kBatch][4];
#pragma unroll
                for (int j = 0; j < kBatch; ++j)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        u[j][k] = part[j] != nullptr && z + k < p.splits ? part[j][(z + k) * next]
                                                                        : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                for (int j = 0; j < kBatch; ++j)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        f[j] = make_float4(__fadd_rn(f[j].x, u[j][k].x), __fadd_rn(f[j].y, u[j][k].y),
                                           __fadd_rn(f[j].z, u[j][k].z), __fadd_rn(f[j].w, u[j][k].w));
            }
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const int row = row0 + (i + j) * kApart;
                const float by = scales[row];
                uint32_t lo[kPlanes], hi[kPlanes];
                split(make_float2(__fmul_rn(f[j].x, by), __fmul_rn(f[j].y, by)), lo);
                split(make_float2(__fmul_rn(f[j].z, by), __fmul_rn(f[j].w, by)), hi);
                const uint32_t to = v_at + (r >> 6) * S::kV + tile_offset(row, (r & 63) >> 3) + (r & 7) * 2;
#pragma unroll
                for (int z = 0; z < kPlanes; ++z)
                    asm volatile("st.shared.v2.u32 [%0], {%1,%2};" ::"r"(to + z * kRuns * S::kV), "r"(lo[z]), "r"(hi[z])
                                 : "memory");
            }
        }
    }
    fence_async_shared();
    tensor_fence_before();
    __syncthreads();
    tensor_fence_after();
    if (warp < kSumWarps) {
        constexpr int kBasePieces = 32 * BASE / 16, kOutPieces = 32 * OUT / 16;   // of 32 columns
        const uint32_t sums = tensor + ((uint32_t)mine0 << 16) + column0;
        int summed = 0;
        for (;;) {
            for (int c = 0; c < chunks; ++c) {
                const int buf = summed & 1, n0 = n_from + c * kN + column0;
                const uint32_t at = room + taken_in % kStages * S::kRoom;
                if (lane == 0 && rows != 0) {
                    bulk_wait_read<S::kLeaving>();
                    fetch(c + S::kAhead, taken_in + S::kAhead);
                }
                if (pass.slots > 0) {
                    if (!wait_for(&done[buf], summed >> 1, &failed))
                        break;
                    ++summed;
                    tensor_fence_after();
                }
                __syncwarp();
                if (rows != 0 && p.base != nullptr &&
                    !wait_for(&here[warp][taken_in % kStages], taken_in / kStages, &failed))
                    break;
                if (rows != 0) {
                    float d[32];
                    const uint32_t from = sums + buf * kExpandSlots * kN;
                    if (one) {
                        tensor_load<32>(d, from + (__ffs(mine) - 1) * kN);
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            d[i] = -0.0f;   // base + -0 is base
                        for (uint32_t todo = mine; todo != 0; todo &= todo - 1u) {
                            const int slot = __ffs(todo) - 1;
                            float f[32];
                            tensor_load<32>(f, from + slot * kN);
                            if (id == pass.id_of(slot))
#pragma unroll
                                for (int i = 0; i < 32; ++i)
                                    d[i] = f[i];
                        }
                    }
                    if (p.base != nullptr) {
#pragma unroll
                        for (int i = 0; i < kBasePieces; ++i) {
                            const uint4 v = ld_shared16(at + piece_at<S::kBaseRow>(lane, i));
                            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                if (BASE == 4) {
                                    d[(i * 4 + j) % 32] = __fadd_rn(__uint_as_float(w[j]), d[(i * 4 + j) % 32]);
                                } else {
                                    const int k = (i * 8 + j * 2) % 32;
                                    d[k] = __fadd_rn(bf16_lo(w[j]), d[k]);
                                    d[k + 1] = __fadd_rn(bf16_hi(w[j]), d[k + 1]);
                                }
                            }
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            d[i] = __fadd_rn(0.0f, d[i]);
                    }
                    if (BASE != OUT)
                        __syncwarp();   // the result's rows lie over other rows of the base
#pragma unroll
                    for (int i = 0; i < kOutPieces; ++i) {
                        uint4 v;
                        if (OUT == 2)
                            v = make_uint4(pack_bf16x2(d[i * 8 % 32], d[(i * 8 + 1) % 32]),
                                           pack_bf16x2(d[(i * 8 + 2) % 32], d[(i * 8 + 3) % 32]),
                                           pack_bf16x2(d[(i * 8 + 4) % 32], d[(i * 8 + 5) % 32]),
                                           pack_bf16x2(d[(i * 8 + 6) % 32], d[(i * 8 + 7) % 32]));
                        else
                            v = make_uint4(__float_as_uint(d[i * 4 % 32]), __float_as_uint(d[(i * 4 + 1) % 32]),
                                           __float_as_uint(d[(i * 4 + 2) % 32]), __float_as_uint(d[(i * 4 + 3) % 32]));
                        asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};"
                                     ::"r"(at + piece_at<S::kOutRow>(lane, i)), "r"(v.x), "r"(v.y),
                                     "r"(v.z), "r"(v.w)
                                     : "memory");
                    }
                }
                if (pass.slots > 0) {
                    tensor_fence_before();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(&taken[buf]);
                }
                if (rows == 0)
                    continue;
                ++taken_in;
                fence_async_shared();
                __syncwarp();
                if (whole) {
                    if (lane == 0 && n0 < p.N)
                        tensor_store(&out_map, at, n0, (int)first + mine0, 0);
                } else {   // pieces of the rows that are this pass's, neighbours by neighbouring lanes
                    constexpr int kPieces = S::kOutRow / 16;
                    const int piece = lane % kPieces;
                    uint8_t *const to = static_cast<uint8_t *>(p.out) + ((first + mine0) * p.N + n0) * OUT + piece * 16;
                    if (n0 + piece * (16 / OUT) < p.N)
#pragma unroll
                        for (int row = lane / kPieces; row < 32; row += 32 / kPieces)
                            if (rows >> row & 1u)
                                *reinterpret_cast<uint4 *>(to + (int64_t)row * p.N * OUT) =
                                    ld_shared16(at + piece_at<S::kOutRow>(row, piece));
                    __syncwarp();   // before the stage is filled again
                }
                if (lane == 0)
                    bulk_commit();
            }
            if (__any_sync(kFull, failed) || pass.next == kNoRow)
                break;
            begin(pass.next, false);
        }
        if (lane == 0) {
            for (; failed && taken_in < fetched; ++taken_in)   // what is still on its way
                wait_alone(&here[warp][taken_in % kStages], taken_in / kStages, &failed);
            bulk_wait<0>();
        }
    } else {
        uint64_t terms[kPlanes];
#pragma unroll
        for (int z = 0; z < kPlanes; ++z)
            terms[z] = tile_descriptor(v_at + z * kRuns * S::kV);
        while (pass.slots > 0) {
            const uint32_t kind = step_kind(pass.slots * kN);
            const int stages = kBStages / pass.slots, run = pass.slots * S::kB;
            // With four stages the steps of a chunk are issued before the next copy waits for those of the chunk before
            // it, so that the matrix pipe always has some ahead; with two, whose copies are what is waited for, after.
            if (lane == 0) {
                if (used == 0 || copy_first())   // the first pass's are on their way
                    for (int c = 0; c < chunks; ++c) {
                        const int use = used + c, buf = use & 1;
                        if (failed || (use >= 2 && !wait_alone(&taken[buf], (use >> 1) - 1, &failed)) ||
                            !wait_alone(&full[use % kBStages], use / kBStages, &failed))
                            break;
                        if (stages == 2 && c + 1 < chunks && !copy(c + 1))
                            break;
                        tensor_fence_after();
                        const uint32_t d = tensor + buf * kExpandSlots * kN, stage = b_at + c % stages * (kRuns * run);
                        const uint64_t b = tile_descriptor(stage);
#pragma unroll
                        for (int z = kPlanes - 1; z >= 0; --z)
#pragma unroll
                            for (int k = 0; k < STEPS; ++k)
                                tensor_step(d, terms[z] + ((k >> 2) * S::kV >> 4) + 2 * (k & 3),
                                            b + ((k >> 2) * run >> 4) + 2 * (k & 3), kind, z != kPlanes - 1 || k != 0);
                        tensor_commit(&empty[use % kBStages]);
                        tensor_commit(&done[buf]);
                        stepped = use + 1;
                        if (stages != 2 && c + stages - 1 < chunks && !copy(c + stages - 1))
                            break;
                    }
                used += chunks;
            }
            __syncwarp();
            if (__any_sync(kFull, failed) || pass.next == kNoRow)
                break;
            begin(pass.next, false);
        }
        if (lane == 0 && failed)
            drain(full, empty, kBStages, copied, stepped, &failed);
    }
    __syncthreads();
    if (failed && threadIdx.x == 0)
        raise(p.err, EP_ERR_TIMEOUT);
    __syncwarp();
    if (warp == kSumWarps)
        tensor_free(tensor, S::kTensor);
}

// ---------------------------------------------------------------- launch --
// A tensor map of [z, y, x] of elements of `bytes` bytes (2: bf16, 4: fp32) in boxes of `columns` columns, 64 or 128 bytes,
// and `rows` rows, swizzled in as many bytes.
int make_map(CUtensorMap *map, const void *at, int bytes, int64_t x, int64_t y, int64_t z, int columns, int rows)
{
    static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> found;
    PFN_cuTensorMapEncodeTiled_v12000 encode = found.load(std::memory_order_relaxed);
    if (encode == nullptr) {
        void *entry = nullptr;
        cudaDriverEntryPointQueryResult how;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &entry, 12000, cudaEnableDefault, &how) != cudaSuccess ||
            how != cudaDriverEntryPointSuccess || entry == nullptr) {
            cudaGetLastError();
            return EP_ERR_CUDA;
        }
        encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(entry);
        found.store(encode, std::memory_order_relaxed);
    }
    const cuuint64_t dims[3] = {(cuuint64_t)x, (cuuint64_t)y, (cuuint64_t)z};
    const cuuint64_t strides[2] = {(cuuint64_t)x * bytes, (cuuint64_t)(x * y) * bytes};
    const cuuint32_t box[3] = {(cuuint32_t)columns, (cuuint32_t)rows, 1}, step[3] = {1, 1, 1};
    return encode(map, bytes == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3,
                  const_cast<void *>(at), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  columns * bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS ? EP_OK : EP_ERR_CUDA;
}

template <int RP, int SLOTS, int STAGES>
int launch_shrink(const Lora &p, cudaStream_t stream)
{
    using S = Shrink<RP, SLOTS, STAGES>;
    static PerDevice set;
    CUtensorMap x, a;
    int rc = raise_smem(lora_shrink_many_kernel<RP, SLOTS, STAGES>, S::kBytes, set);
    if (rc == EP_OK)
        rc = make_map(&x, p.x, 2, p.K, p.M, 1, kChunk, kRows);
    if (rc == EP_OK)
        rc = make_map(&a, p.a, 2, p.K, p.R, p.L, kChunk, RP);
    if (rc != EP_OK)
        return rc;
    return launch_dependent(lora_shrink_many_kernel<RP, SLOTS, STAGES>, dim3((unsigned)ceil_div(p.M, kRows), p.splits),
                            kShrinkThreads, S::kBytes, stream, p, x, a);
}

template <int STEPS, int BASE, int OUT>
int launch_expand(const Lora &p, cudaStream_t stream)
{
    using S = Expand<STEPS, BASE, OUT>;
    static PerDevice set;
    CUtensorMap b, base, out;
    int rc = raise_smem(lora_expand_many_kernel<STEPS, BASE, OUT>, S::kBytes, set);
    if (rc == EP_OK)
        rc = make_map(&b, p.b, 2, p.R, p.N, p.L, 64, S::kN);
    if (rc == EP_OK)
        rc = make_map(&out, p.out, OUT, p.N, p.M, 1, 32, 32);
    if (rc == EP_OK && p.base != nullptr)
        rc = make_map(&base, p.base, BASE, p.N, p.M, 1, 32, 32);
    else
        base = out;   // never read
    if (rc != EP_OK)
        return rc;
    // a block to an SM, with as few columns as that leaves
    const int64_t tiles = ceil_div(p.M, kRows);
    const int64_t pieces = std::max<int64_t>(1, std::min<int64_t>(ceil_div(p.N, S::kN), kLoraBlocks / 2 / tiles));
    const int span = (int)(ceil_div(ceil_div(p.N, pieces), S::kN) * S::kN);
    return launch_dependent(lora_expand_many_kernel<STEPS, BASE, OUT>, dim3((unsigned)tiles, (unsigned)ceil_div(p.N, span)),
                            S::kThreads, S::kBytes, stream, p, b, base, out, span);
}

template <int STEPS>
int launch_expand(const Lora &p, cudaStream_t stream)
{
    if (p.base != nullptr && p.base_dtype != 0)
        return p.out_dtype == 0 ? launch_expand<STEPS, 4, 2>(p, stream) : launch_expand<STEPS, 4, 4>(p, stream);
    return p.out_dtype == 0 ? launch_expand<STEPS, 2, 2>(p, stream) : launch_expand<STEPS, 2, 4>(p, stream);
}

}  // namespace

int launch_lora_shrink_many(const Lora &p, cudaStream_t stream)
{
    return p.R <= 16 ? launch_shrink<16, 4, 4>(p, stream) : p.R <= 32 ? launch_shrink<32, 4, 3>(p, stream)
                   : p.R <= 64 ? launch_shrink<64, 2, 3>(p, stream) : launch_shrink<128, 2, 3>(p, stream);
}

int launch_lora_expand_many(const Lora &p, cudaStream_t stream)
{
    if (p.R <= 16)
        return launch_expand<1>(p, stream);
    if (p.R <= 32)
        return launch_expand<2>(p, stream);
    return p.R <= 64 ? launch_expand<4>(p, stream) : launch_expand<8>(p, stream);
}

}  // namespace ep
