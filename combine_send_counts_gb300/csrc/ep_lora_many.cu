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
//     memory; B comes 32 columns at a time; the base comes through a ring of each warp's
//     own, where the sums are added to it and from where they leave in whole rows.
//
// x, A and B come by TMA (tensor maps of x [M,K], A [L,R,K] and B [L,N,R], whose
// edges read as zeros) with the 128-byte swizzle that the matrix steps take.  Copied by
// cp.async instead, with a proxy fence by the threads that copied, both kernels waited
// at that fence for the copies still in flight.  Waits on barriers give up after a
// second (EP_ERR_TIMEOUT).
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

constexpr int kRows = 128;           // of a tile
constexpr int kNoRow = 0x7fffffff;   // the adapter of a row past the end
constexpr uint64_t kLimitNs = 1000000000;

// The least adapter above `last` among a tile's rows, kNoRow if there is none.  The same in every lane.
__device__ __forceinline__ int adapter_after(const int *ids, int last)
{
    int least = kNoRow;
#pragma unroll
    for (int i = 0; i < kRows / 32; ++i) {
        const int id = ids[i * 32 + (threadIdx.x & 31)];
        least = id > last ? min(least, id) : least;
    }
    return __reduce_min_sync(kFull, least);
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

// One thread waits for the n-th use of a barrier that is completed once a use; false (once and for all) after a second.
__device__ __forceinline__ bool wait_alone(uint64_t *bar, int n, volatile int *failed)
{
    if (mbar_wait(bar, n & 1, kLimitNs))
        return true;
    *failed = 1;
    return false;
}

// A whole warp waits.  Lanes may leave the spin one by one, and the way out of a wait that failed leaves the caller's
// loop, so that they would meet again only behind it: the vote brings them together for the .aligned instructions here.
__device__ __forceinline__ bool wait_for(uint64_t *bar, int n, volatile int *failed)
{
    const bool ok = wait_alone(bar, n, failed);
    return __all_sync(kFull, ok);
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
    allow_dependents();
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
    __syncwarp();
    if (warp == kFlushWarps + 1)
        tensor_alloc(&tensor, S::kColumns);
    tensor_fence_before();
    __syncthreads();
    tensor_fence_after();
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
            if (failed)
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
            if (failed)
                break;
        }
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
            if (failed)
                break;
        }
    }
    __syncthreads();
    if (failed && threadIdx.x == 0)
        raise(p.err, EP_ERR_TIMEOUT);
    __syncwarp();
    if (warp == kFlushWarps + 1)
        tensor_free(tensor, S::kColumns);
}

// ---------------------------------------------------------------- expand --
constexpr int kSumWarps = 8, kExpandThreads = kSumWarps * 32 + 32;
constexpr int kColumns = 32;        // of the output, a chunk
constexpr int kExpandSlots = 2, kBStages = 3, kRowStages = 2;

// KB: runs of 64 ranks.  BASE, OUT: bytes of an element.
template <int KB, int BASE, int OUT>
struct Expand {
    static constexpr int kV = kRows * 128;                                     // a term of v, 64 ranks
    static constexpr int kB = kExpandSlots * kColumns * 128;                   // a stage of B, 64 ranks
    static constexpr int kRowBytes = kColumns * (BASE > OUT ? BASE : OUT);
    static constexpr int kRoom = 32 * kRowBytes;                               // a warp's stage
    static constexpr int kBytes = kPlanes * KB * kV + kBStages * KB * kB + kSumWarps * kRowStages * kRoom + 1024;
    static constexpr int kTensor = 2 * kExpandSlots * kColumns;                // columns of tensor memory
    static constexpr int kPerSM = KB == 1 && kBytes <= 112 * 1024 ? 2 : 1;     // blocks

    // a 16-byte piece of a row, so that eight rows' meet no bank twice
    __device__ __forceinline__ static uint32_t piece(int row, int i)
    {
        return row * kRowBytes + ((kRowBytes == 64 ? i ^ (row >> 1 & 3) : i ^ (row & 7)) << 4);
    }
};

// Warps 0-3 take the even chunks, 4-7 the odd ones, each its own buffer of tensor memory; warp 8 copies B and issues the
// matrix steps.
template <int KB, int BASE, int OUT>
__global__ void __launch_bounds__(kExpandThreads, (Expand<KB, BASE, OUT>::kPerSM))
lora_expand_many_kernel(Lora p, const __grid_constant__ CUtensorMap b_map, int span)
{
    using S = Expand<KB, BASE, OUT>;
    extern __shared__ uint8_t dynamic[];
    __shared__ int ids[kRows];
    __shared__ float scales[kRows];
    __shared__ uint64_t full[kBStages], empty[kBStages], done[2], taken[2];
    __shared__ uint32_t tensor;
    __shared__ int failed;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t first = (int64_t)blockIdx.x * kRows;
    const uint32_t v_at = (smem_u32(dynamic) + 1023u) & ~1023u, b_at = v_at + kPlanes * KB * S::kV;
    const uint32_t rows_at = b_at + kBStages * KB * S::kB;
    const int n_from = blockIdx.y * span, n_to = min(n_from + span, p.N);
    const int chunks = (n_to - n_from + kColumns - 1) / kColumns;
    const int steps = (p.R + 15) / 16;   // of 16 ranks
    grid_dependency_wait();
    allow_dependents();
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
            mbar_init(&taken[i], kSumWarps / 2);
        }
        fence_mbar_init();
    }
    __syncwarp();
    if (warp == kSumWarps)
        tensor_alloc(&tensor, S::kTensor);
    __syncthreads();
    if (warp < kSumWarps) {   // v of every row: a thread has a pair of ranks of several rows, kBatch of them at a time
        constexpr int kBatch = 4;
        const int log_pairs = p.R <= 16 ? 3 : p.R <= 32 ? 4 : p.R <= 64 ? 5 : 6;
        const int r = (threadIdx.x & ((1 << log_pairs) - 1)) * 2, apart = kSumWarps * 32 >> log_pairs;
        for (int row = threadIdx.x >> log_pairs; row < kRows; row += kBatch * apart) {
            float2 f[kBatch];
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const int at = row + j * apart, id = at < kRows ? ids[at] : -1;
                f[j] = ranks_of(p, id >= 0 && id != kNoRow ? first + at : -1, r, id >= 0 ? scales[at] : 1.0f);
            }
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const int at = row + j * apart;
                if (at >= kRows || r >= steps * 16)
                    break;
                uint32_t terms[kPlanes];
                split(f[j], terms);
                const uint32_t to = v_at + (r >> 6) * S::kV + tile_offset(at, (r & 63) >> 3) + (r & 7) * 2;
#pragma unroll
                for (int z = 0; z < kPlanes; ++z)
                    asm volatile("st.shared.u32 [%0], %1;" ::"r"(to + z * KB * S::kV), "r"(terms[z]) : "memory");
            }
        }
    }
    fence_async_shared();
    tensor_fence_before();
    __syncthreads();
    tensor_fence_after();
    Pass<kExpandSlots> pass;
    const int begin = adapter_after(ids, -1);
    if (warp < kSumWarps) {
        // a row to a thread for the sums; whole rows by neighbouring lanes for the base and the result
        constexpr int kBasePieces = kColumns * BASE / 16, kOutPieces = kColumns * OUT / 16;
        const int group = warp >> 2, mine0 = (warp & 3) * 32, id = ids[mine0 + lane];
        const uint32_t room = rows_at + warp * kRowStages * S::kRoom;
        const uint32_t sums = tensor + ((uint32_t)mine0 << 16) + group * kExpandSlots * kColumns;
        // this lane's pieces: of rows lane / pieces, and so many further
        const int base_row = lane / kBasePieces, base_piece = lane % kBasePieces;
        const int out_row = lane / kOutPieces, out_piece = lane % kOutPieces;
        const uint8_t *const base_at = static_cast<const uint8_t *>(p.base) + (first + mine0 + base_row) * p.N * BASE + base_piece * 16;
        uint8_t *const out_at = static_cast<uint8_t *>(p.out) + (first + mine0 + out_row) * p.N * OUT + out_piece * 16;
        const int64_t base_apart = (int64_t)(32 / kBasePieces) * p.N * BASE, out_apart = (int64_t)(32 / kOutPieces) * p.N * OUT;
        int used = 0;       // sums of this group so far
        int before = 0;     // chunks of the passes so far
        bool start = true;
        for (int now = begin; start || now != kNoRow; now = pass.next) {
            pass.set(ids, now);
            // rows without an adapter go along with the first pass
            const bool row_in = pass.has(id) || (start && id == -1);
            const uint32_t rows = __ballot_sync(kFull, row_in), mine = pass.mask(id);
            start = false;
            // the group of a chunk goes on counting through the passes, as the buffers do
            const int c0 = (before & 1) == group ? 0 : 1;
            if (pass.slots > 0)
                before += chunks;
            auto fetch = [&](int c, int stage) {
                if (p.base != nullptr && c < chunks) {
                    const int n0 = n_from + c * kColumns;
                    const bool in = n0 + base_piece * (16 / BASE) < p.N;
#pragma unroll
                    for (int i = 0; i < kBasePieces; ++i) {
                        const int row = base_row + i * (32 / kBasePieces);
                        const bool ok = in && (rows >> row & 1u);
                        cp_async16(room + stage * S::kRoom + S::piece(row, base_piece),
                                   ok ? base_at + i * base_apart + (int64_t)n0 * BASE : p.x, ok);
                    }
                }
                cp_async_commit();
            };
            fetch(c0, 0);
            int stage = 0;
            for (int c = c0; c < chunks; c += 2, stage ^= 1) {
                fetch(c + 2, stage ^ 1);
                const int n0 = n_from + c * kColumns;
                float d[kColumns];
#pragma unroll
                for (int i = 0; i < kColumns; ++i)
                    d[i] = -0.0f;   // base + -0 is base
                if (pass.slots > 0) {
                    if (!wait_for(&done[group], used++, &failed))
                        break;
                    tensor_fence_after();
                    if (mine != 0 && (mine & (mine - 1u)) == 0) {   // rows of one adapter, or of none here
                        tensor_load<kColumns>(d, sums + (__ffs(mine) - 1) * kColumns);
                        if (id == -1)
#pragma unroll
                            for (int i = 0; i < kColumns; ++i)
                                d[i] = -0.0f;
                    } else {
                        for (uint32_t todo = mine; todo != 0; todo &= todo - 1u) {
                            const int slot = __ffs(todo) - 1;
                            float f[kColumns];
                            tensor_load<kColumns>(f, sums + slot * kColumns);
                            if (id == pass.id_of(slot))
#pragma unroll
                                for (int i = 0; i < kColumns; ++i)
                                    d[i] = f[i];
                        }
                    }
                    tensor_fence_before();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(&taken[group]);
                }
                cp_async_wait<1>();
                __syncwarp();
                const uint32_t at = room + stage * S::kRoom;
                if (p.base != nullptr) {
#pragma unroll
                    for (int i = 0; i < kBasePieces; ++i) {
                        const uint4 v = ld_shared16(at + S::piece(lane, i));
                        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            if (BASE == 4) {
                                d[(i * 4 + j) % kColumns] = __fadd_rn(__uint_as_float(w[j]), d[(i * 4 + j) % kColumns]);
                            } else {
                                const int k = (i * 8 + j * 2) % kColumns;
                                d[k] = __fadd_rn(bf16_lo(w[j]), d[k]);
                                d[k + 1] = __fadd_rn(bf16_hi(w[j]), d[k + 1]);
                            }
                        }
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < kColumns; ++i)
                        d[i] = __fadd_rn(0.0f, d[i]);
                }
#pragma unroll
                for (int i = 0; i < kOutPieces; ++i) {
                    uint4 v;
                    if (OUT == 2)
                        v = make_uint4(pack_bf16x2(d[i * 8 % kColumns], d[(i * 8 + 1) % kColumns]),
                                       pack_bf16x2(d[(i * 8 + 2) % kColumns], d[(i * 8 + 3) % kColumns]),
                                       pack_bf16x2(d[(i * 8 + 4) % kColumns], d[(i * 8 + 5) % kColumns]),
                                       pack_bf16x2(d[(i * 8 + 6) % kColumns], d[(i * 8 + 7) % kColumns]));
                    else
                        v = make_uint4(__float_as_uint(d[i * 4 % kColumns]), __float_as_uint(d[(i * 4 + 1) % kColumns]),
                                       __float_as_uint(d[(i * 4 + 2) % kColumns]), __float_as_uint(d[(i * 4 + 3) % kColumns]));
                    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at + S::piece(lane, i)), "r"(v.x), "r"(v.y),
                                 "r"(v.z), "r"(v.w)
                                 : "memory");
                }
                __syncwarp();
                const bool in = n0 + out_piece * (16 / OUT) < p.N;
#pragma unroll
                for (int i = 0; i < kOutPieces; ++i) {
                    const int row = out_row + i * (32 / kOutPieces);
                    if (in && (rows >> row & 1u))
                        *reinterpret_cast<uint4 *>(out_at + i * out_apart + (int64_t)n0 * OUT) =
                            ld_shared16(at + S::piece(row, out_piece));
                }
                __syncwarp();   // before the stage is filled again
            }
            cp_async_wait<0>();
            __syncwarp();
            if (failed)
                break;
        }
    } else {
        int used = 0;   // chunks so far: stages of B, and sums
        uint64_t terms[kPlanes];
#pragma unroll
        for (int z = 0; z < kPlanes; ++z)
            terms[z] = tile_descriptor(v_at + z * KB * S::kV);
        for (int now = begin; now != kNoRow; now = pass.next) {
            pass.set(ids, now);
            const uint32_t kind = step_kind(pass.slots * kColumns);
            // one thread: chunk c is copied, and the steps of the chunk before those in flight issued
            if (lane == 0)
                for (int c = 0; c < chunks + kBStages - 1; ++c) {
                    if (c < chunks) {
                        const int use = used + c, at = use % kBStages;
                        if (use >= kBStages && !wait_alone(&empty[at], use / kBStages - 1, &failed))
                            break;
                        const uint32_t to = b_at + at * (KB * S::kB);
                        mbar_arrive_expect_tx(&full[at], pass.slots * KB * kColumns * 128);
#pragma unroll
                        for (int i = 0; i < kExpandSlots; ++i)
                            if (i < pass.slots)
#pragma unroll
                                for (int b = 0; b < KB; ++b)
                                    tensor_copy(to + b * S::kB + i * kColumns * 128, &b_map, b * 64, n_from + c * kColumns,
                                                pass.slot[i], &full[at]);
                    }
                    if (c < kBStages - 1)
                        continue;
                    const int use = used + c - (kBStages - 1), buf = use & 1;
                    if ((use >= 2 && !wait_alone(&taken[buf], (use >> 1) - 1, &failed)) ||
                        !wait_alone(&full[use % kBStages], use / kBStages, &failed))
                        break;
                    tensor_fence_after();
                    const uint32_t d = tensor + buf * kExpandSlots * kColumns, stage = b_at + use % kBStages * (KB * S::kB);
                    if constexpr (KB == 1) {
                        // few instructions to a step: one thread issues them all
                        const uint64_t b = tile_descriptor(stage);
#pragma unroll
                        for (int z = kPlanes - 1; z >= 0; --z)
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                if (k < steps)
                                    tensor_step(d, terms[z] + 2 * k, b + 2 * k, kind, z != kPlanes - 1 || k != 0);
                    } else {
                        bool add = false;
#pragma unroll
                        for (int z = kPlanes - 1; z >= 0; --z)
                            for (int k = 0; k < steps; ++k) {
                                const uint64_t a = tile_descriptor(v_at + (z * KB + (k >> 2)) * S::kV) + 2 * (k & 3);
                                const uint64_t b = tile_descriptor(stage + (k >> 2) * S::kB) + 2 * (k & 3);
                                tensor_step(d, a, b, kind, add);
                                add = true;
                            }
                    }
                    tensor_commit(&empty[use % kBStages]);
                    tensor_commit(&done[buf]);
                }
            __syncwarp();
            if (failed)
                break;
            used += chunks;
        }
    }
    __syncthreads();
    if (failed && threadIdx.x == 0)
        raise(p.err, EP_ERR_TIMEOUT);
    __syncwarp();
    if (warp == kSumWarps)
        tensor_free(tensor, S::kTensor);
}

// ---------------------------------------------------------------- launch --
// A tensor map of bf16 [z, y, x] read in boxes of 64 columns and `rows` rows.
int make_map(CUtensorMap *map, const void *at, int64_t x, int64_t y, int64_t z, int rows)
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
    const cuuint64_t strides[2] = {(cuuint64_t)x * 2, (cuuint64_t)(x * y) * 2};
    const cuuint32_t box[3] = {kChunk, (cuuint32_t)rows, 1}, step[3] = {1, 1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(at), dims, strides, box, step,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS ? EP_OK : EP_ERR_CUDA;
}

template <int RP, int SLOTS, int STAGES>
int launch_shrink(const Lora &p, cudaStream_t stream)
{
    using S = Shrink<RP, SLOTS, STAGES>;
    static PerDevice set;
    CUtensorMap x, a;
    int rc = raise_smem(lora_shrink_many_kernel<RP, SLOTS, STAGES>, S::kBytes, set);
    if (rc == EP_OK)
        rc = make_map(&x, p.x, p.K, p.M, 1, kRows);
    if (rc == EP_OK)
        rc = make_map(&a, p.a, p.K, p.R, p.L, RP);
    if (rc != EP_OK)
        return rc;
    return launch_dependent(lora_shrink_many_kernel<RP, SLOTS, STAGES>, dim3((unsigned)ceil_div(p.M, kRows), p.splits),
                            kShrinkThreads, S::kBytes, stream, p, x, a);
}

template <int KB, int BASE, int OUT>
int launch_expand(const Lora &p, cudaStream_t stream)
{
    using S = Expand<KB, BASE, OUT>;
    static PerDevice set;
    CUtensorMap b;
    int rc = raise_smem(lora_expand_many_kernel<KB, BASE, OUT>, S::kBytes, set);
    if (rc == EP_OK)
        rc = make_map(&b, p.b, p.R, p.N, p.L, kColumns);
    if (rc != EP_OK)
        return rc;
    const int64_t tiles = ceil_div(p.M, kRows);
    const int64_t pieces = std::max<int64_t>(1, std::min<int64_t>(ceil_div(p.N, kColumns), kLoraBlocks / 2 * S::kPerSM / tiles));
    const int span = (int)(ceil_div(ceil_div(p.N, pieces), kColumns) * kColumns);
    return launch_dependent(lora_expand_many_kernel<KB, BASE, OUT>, dim3((unsigned)tiles, (unsigned)ceil_div(p.N, span)),
                            kExpandThreads, S::kBytes, stream, p, b, span);
}

template <int KB>
int launch_expand(const Lora &p, cudaStream_t stream)
{
    if (p.base != nullptr && p.base_dtype != 0)
        return p.out_dtype == 0 ? launch_expand<KB, 4, 2>(p, stream) : launch_expand<KB, 4, 4>(p, stream);
    return p.out_dtype == 0 ? launch_expand<KB, 2, 2>(p, stream) : launch_expand<KB, 2, 4>(p, stream);
}

}  // namespace

int launch_lora_many(const Lora &p, cudaStream_t stream)
{
    const int rc = p.R <= 16 ? launch_shrink<16, 4, 4>(p, stream) : p.R <= 32 ? launch_shrink<32, 4, 3>(p, stream)
                   : p.R <= 64 ? launch_shrink<64, 2, 3>(p, stream) : launch_shrink<128, 2, 3>(p, stream);
    if (rc != EP_OK)
        return rc;
    return p.R <= 64 ? launch_expand<1>(p, stream) : launch_expand<2>(p, stream);
}

}  // namespace ep
