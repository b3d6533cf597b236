// The experts of a mixture-of-experts layer for a few tokens, in two kernels.
//
//   up:    h[s] = silu(Wg x) * (Wu x) for every slot s = (t, k) that names a
//          local expert;
//   down:  out[t] = sum over k of w[t,k] * (W2 h[t,k]).
//
// Each expert that some token names has its matrices read once for all its
// slots (32 at a time), by products of 16 weight rows with the slots as columns
// (ep_skinny.cuh).  No row of x is copied to an expert and no list is made on
// the host: every block derives the experts in use and their slots from
// topk_idx, which a graph replay may have changed.
//
// up: the elements of h of all experts in use, laid end to end, are dealt to
// one block per SM in equal runs.  An item is 8 elements: their 8 gate rows and
// 8 up rows are the 16 rows of a matrix step, whose accumulators hold gate and
// up of an element in the same lane.
//
// down: each block owns an equal share of the output's rows and adds up all
// experts for them.  An item is up to 16 of its rows of one expert.  Every
// slot's results stay in shared memory and are weighted and added from there in
// ascending k, so nothing but out is written.
//
// In both the block's items are shared evenly by its warps, whose runs may stop
// inside an item; the pieces of a divided item are added in the order of their
// columns.  Nothing depends on the order of arrival.
//
// h is kept as the bf16 terms of a sum (two terms, or three for fp32 results:
// 16 or 24 significant bits), which is what the matrix step takes; one bf16
// would add an error as large as the rounding of the result itself.
#include <algorithm>

#include "ep_device.cuh"
#include "ep_internal.h"
#include "ep_skinny.cuh"

namespace ep {
namespace {

constexpr int kThreads = kSkinnyThreads;
constexpr int kWarps = kSkinnyWarps;
constexpr int kMaxSlots = EP_MOE_MAX_SLOTS;
constexpr int kMaxDim = 65536;   // H and I: a block's units are counted in 32 bits
constexpr int kRow = 17;   // floats between slots in shared memory, for 16 rows

struct Routing {
    const int64_t *idx;
    int n;           // slots: T * K
    int K, E, E_local;
    int64_t first;   // first local expert

    // local expert of slot s, or -1
    __device__ __forceinline__ int local(int s, int32_t *err) const
    {
        const int64_t v = idx[s];
        if (v < -1 || v >= E) {
            raise(err, EP_ERR_INVALID_EXPERT);
            return -1;
        }
        const int64_t l = v - first;
        return v >= 0 && l >= 0 && l < E_local ? (int)l : -1;
    }
};

// The experts in use, in entries of up to 32 slots each, in shared memory.
struct Lists {
    int entries, big;
    int scan[3][kWarps];
    uint16_t big_expert[kMaxSlots / kMaxCols];   // experts of more than one entry
    int cost[kMaxSlots + 1];          // exclusive sums of the entries' costs per weight row
    uint16_t expert[kMaxSlots];
    uint16_t begin[kMaxSlots + 1];    // slots of entry q: slot[begin[q] .. begin[q+1])
    uint16_t slot[kMaxSlots];
    int16_t use[kMaxSlots];           // slot -> its entry, or -1
    uint16_t place[kMaxSlots];        // slot -> its place among its expert's slots
};

__device__ __forceinline__ int blocks_of(int cols) { return (cols + 7) >> 3; }

// All threads of the block; count: E_local ints of shared memory.  An entry of
// nb column blocks costs item_cost + nb for each row.
__device__ __forceinline__ void build_lists(const Routing &r, Lists &l, int *count, int item_cost, int32_t *err)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int e = tid; e < r.E_local; e += kThreads)
        count[e] = 0;
    if (tid == 0)
        l.big = 0;
    __syncthreads();
    for (int s = tid; s < r.n; s += kThreads) {
        const int e = r.local(s, err);
        l.use[s] = (int16_t)e;
        if (e >= 0)
            l.place[s] = (uint16_t)atomicAdd(&count[e], 1);
    }
    __syncthreads();
    // each thread owns a run of experts; scan of (entries, slots, cost)
    const int per = (r.E_local + kThreads - 1) / kThreads;
    const int e0 = min(tid * per, r.E_local), e1 = min(e0 + per, r.E_local);
    int own[3] = {0, 0, 0};
    for (int e = e0; e < e1; ++e) {
        const int c = count[e], full = c / kMaxCols, rest = c % kMaxCols;
        own[0] += full + (rest > 0);
        own[1] += c;
        own[2] += full * (item_cost + kMaxCols / 8) + (rest > 0 ? item_cost + blocks_of(rest) : 0);
    }
    int sum[3] = {own[0], own[1], own[2]};
    for (int o = 1; o < 32; o <<= 1)
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            const int v = __shfl_up_sync(kFull, sum[i], o);
            if (lane >= o)
                sum[i] += v;
        }
    if (lane == 31)
        for (int i = 0; i < 3; ++i)
            l.scan[i][warp] = sum[i];
    __syncthreads();
    for (int i = 0; i < 3; ++i) {
        sum[i] -= own[i];
        for (int w = 0; w < warp; ++w)
            sum[i] += l.scan[i][w];
    }
    int q = sum[0], at = sum[1], cost = sum[2];
    for (int e = e0; e < e1; ++e) {
        const int c = count[e];
        count[e] = q;
        if (c > kMaxCols)
            l.big_expert[atomicAdd(&l.big, 1)] = (uint16_t)e;
        for (int b = 0; b < c; b += kMaxCols) {
            const int cols = min(c - b, kMaxCols);
            l.expert[q] = (uint16_t)e;
            l.begin[q] = (uint16_t)(at + b);
            l.cost[q] = cost;
            cost += item_cost + blocks_of(cols);
            ++q;
        }
        at += c;
    }
    if (tid == kThreads - 1) {
        l.entries = q;
        l.begin[q] = (uint16_t)at;
        l.cost[q] = cost;
    }
    __syncthreads();
    // The order of slots within an entry moves no result, but every block must put the same slots into an
    // entry: where an expert has several, its slots take their places in ascending order.
    if (l.big > 0) {
        for (int b = warp; b < l.big; b += kWarps) {
            const int e = l.big_expert[b];
            int before = 0;
            for (int s0 = 0; s0 < r.n; s0 += 32) {
                const int s = s0 + lane;
                const bool hit = s < r.n && l.use[s] == e;
                const unsigned m = __ballot_sync(kFull, hit);
                if (hit)
                    l.place[s] = (uint16_t)(before + __popc(m & lanemask_lt()));
                before += __popc(m);
            }
        }
        __syncthreads();
    }
    for (int s = tid; s < r.n; s += kThreads) {
        const int e = l.use[s];
        if (e >= 0) {
            const int p = l.place[s], f = count[e];
            l.slot[l.begin[f] + p] = (uint16_t)s;
            l.use[s] = (int16_t)(f + p / kMaxCols);
        }
    }
    __syncthreads();
}

struct Planes {
    uint8_t *h;            // [PLANES][n][I] bf16
    int64_t plane_bytes;
    int I;
};

// h as a sum of bf16 terms; an infinity or NaN is its own first term
template <int PLANES, bool PERMUTED>
__device__ __forceinline__ void store_planes(const Planes &p, int slot, int i, float h)
{
    const int place = (i & ~7) | column_place<PERMUTED>(i & 7);
    uint8_t *at = p.h + ((int64_t)slot * p.I + place) * 2;
    float rest = h;
#pragma unroll
    for (int q = 0; q < PLANES; ++q) {
        // toward zero, so that a term never rounds up to infinity; the last to nearest
        const bool last = q == PLANES - 1;
        const float term = last ? __bfloat162float(__float2bfloat16_rn(rest))
                                : __uint_as_float(__float_as_uint(rest) & 0xffff0000u);
        *reinterpret_cast<uint16_t *>(at + q * p.plane_bytes) = (uint16_t)(__float_as_uint(term) >> 16);
        const float left = __fsub_rn(rest, term);
        rest = isfinite(h) ? left : 0.0f;
    }
}

// silu(gate) * up; a NaN keeps its set bits in the upper half, where the terms above look
__device__ __forceinline__ float activate(float gate, float up)
{
    const float h = __fmul_rn(__fdiv_rn(gate, __fadd_rn(1.0f, expf(-gate))), up);
    return isnan(h) ? __int_as_float(0x7fffffff) : h;
}

template <int NT, int PLANES>
__device__ __forceinline__ void set_columns(const Lists &l, int q, const uint8_t *rows, int64_t row_bytes,
                                            int slots_per_row, Columns<NT, PLANES> &x)
{
    const int g = (threadIdx.x & 31) >> 2, first = l.begin[q], end = l.begin[q + 1];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int s = first + nt * 8 + g;
        x.p[nt] = s < end ? rows + (int64_t)(l.slot[s] / slots_per_row) * row_bytes : nullptr;
    }
}

// ------------------------------------------------------------------------ up --
struct UpArgs {
    const uint8_t *x;
    Routing r;
    int H, I;
    Weights w;
    Planes out;
    int32_t *err;
};

// A block's elements: from element i0 of entry q0 to element i1 of entry q1
// (exclusive), in items of 8 elements that do not cross entries.
template <int G, int PLANES>
struct UpItems {
    using F = typename FormatOf<G, false>::F;
    const UpArgs &a;
    const Lists &l;
    int q0, i0, q1, i1;
    int head, body;        // items of the first entry, items of each further one
    float *side;           // this warp's kept piece of an item that another warp began
    float *open;           // its kept piece of an item that it began and another goes on with

    __device__ __forceinline__ int count() const
    {
        return q1 > q0 ? head + (q1 - q0 - 1) * body + (i1 + 7) / 8 : head;
    }

    __device__ __forceinline__ void where(int item, int &q, int &i, int &end) const
    {
        if (item < head) {
            q = q0;
            i = i0 + item * 8;
        } else {
            const int v = item - head;
            q = q0 + 1 + v / body;
            i = v % body * 8;
        }
        end = min(i + 8, q == q1 ? i1 : a.I);
    }

    __device__ __forceinline__ RowPtrs rows(int item) const
    {
        int q, i, end;
        where(item, q, i, end);
        i += (threadIdx.x & 31) >> 2;
        const int64_t row = (int64_t)l.expert[q] * 2 * a.I + i;
        return F::rows(a.w, row, row + a.I, i < end, i < end, a.H);
    }

    __device__ __forceinline__ int blocks(int item) const
    {
        int q, i, end;
        where(item, q, i, end);
        return blocks_of(l.begin[q + 1] - l.begin[q]);
    }

    template <int NT>
    __device__ __forceinline__ void columns(int item, Columns<NT, 1> &x) const
    {
        int q, i, end;
        where(item, q, i, end);
        x.plane_bytes = 0;
        set_columns<NT, 1>(l, q, a.x, (int64_t)a.H * 2, a.r.K, x);
    }

    template <int NT>
    __device__ __forceinline__ void done(int item, bool first, bool last, float (&acc)[NT][4]) const
    {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
        if (!first || !last) {
            float *keep = first ? open : side;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                *reinterpret_cast<float4 *>(keep + (nt * 32 + lane) * 4) =
                    make_float4(acc[nt][0], acc[nt][1], acc[nt][2], acc[nt][3]);
            return;
        }
        int q, i, end;
        where(item, q, i, end);
        if (i + g >= end)
            return;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int s = l.begin[q] + nt * 8 + 2 * t + c;
                if (s < l.begin[q + 1])
                    store_planes<PLANES, (G > 0)>(a.out, l.slot[s], i + g, activate(acc[nt][c], acc[nt][2 + c]));
            }
    }
};

// the entry and element at position pos of the costs laid end to end
__device__ __forceinline__ void find(const Lists &l, int I, int64_t pos, int &q, int &i)
{
    int lo = 0, hi = l.entries;   // cost[lo] * I <= pos < cost[hi] * I
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if ((int64_t)l.cost[mid] * I <= pos)
            lo = mid;
        else
            hi = mid;
    }
    q = lo;
    i = (int)((pos - (int64_t)l.cost[lo] * I) / (l.cost[lo + 1] - l.cost[lo]));
}

template <int G, int PLANES>
__global__ void __launch_bounds__(kThreads, 1)
moe_up_kernel(UpArgs a)
{
    extern __shared__ __align__(16) uint8_t dynamic[];   // ring, then one side block per warp
    __shared__ Lists l;
    using F = typename FormatOf<G, false>::F;
    grid_dependency_wait();
    allow_dependents();
    build_lists(a.r, l, reinterpret_cast<int *>(dynamic), F::kItemCost, blockIdx.x == 0 ? a.err : nullptr);
    if (l.entries == 0)
        return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint8_t *sides = dynamic + kRingBytes;
    UpItems<G, PLANES> items{a, l};
    const int64_t total = (int64_t)l.cost[l.entries] * a.I;
    find(l, a.I, total * blockIdx.x / gridDim.x, items.q0, items.i0);
    if (blockIdx.x + 1 < gridDim.x) {
        find(l, a.I, total * (blockIdx.x + 1) / gridDim.x, items.q1, items.i1);
    } else {
        items.q1 = l.entries;
        items.i1 = 0;
    }
    items.head = ((items.q1 > items.q0 ? a.I : items.i1) - items.i0 + 7) / 8;
    items.body = (a.I + 7) / 8;
    items.side = reinterpret_cast<float *>(sides + warp * kSideBytes);
    items.open = reinterpret_cast<float *>(dynamic + warp * (kStages * kStageBytes));   // the ring is idle by then
    const int n = items.count();
    if (n == 0)
        return;
    Stream<F, 1, UpItems<G, PLANES>> stream(items, a.H, n, smem_u32(dynamic));
    stream.start();
    stream.run();
    __syncthreads();
    // the warp that began an item which others went on with adds up its pieces
    const int per = (a.H + F::kUnit - 1) / F::kUnit;
    const int begin = run_begin(n, per, warp), end = run_begin(n, per, warp + 1);
    const int item = (end - 1) / per;
    if (begin == end || end % per == 0 || item * per < begin)
        return;
    int q, i, stop;
    items.where(item, q, i, stop);
    const int first = l.begin[q], cols = l.begin[q + 1] - first;
    for (int v = lane; v < 8 * cols; v += 32) {
        const int g = v & 7, c = v >> 3;
        if (i + g >= stop)
            continue;
        float gate = items.open[side_index(g, c)], up = items.open[side_index(g + 8, c)];
        for (int w = warp + 1; w < kWarps && run_begin(n, per, w) < (item + 1) * per; ++w) {
            if (run_begin(n, per, w) == run_begin(n, per, w + 1))
                continue;
            const float *p = reinterpret_cast<const float *>(sides + w * kSideBytes);
            gate = __fadd_rn(gate, p[side_index(g, c)]);
            up = __fadd_rn(up, p[side_index(g + 8, c)]);
        }
        store_planes<PLANES, (G > 0)>(a.out, l.slot[first + c], i + g, activate(gate, up));
    }
}

// ---------------------------------------------------------------------- down --
struct DownArgs {
    Routing r;
    const float *weights;
    int T, H, I;
    Weights w;
    Planes h;
    void *out;
    int out_f32;
    int blocks;        // row blocks that the shared memory has room for at a time
};

// Row blocks [0, nb) of `rows` rows each from row0 on, times all entries.
template <int G, int PLANES>
struct DownItems {
    using F = typename FormatOf<G, (G > 0)>::F;
    const DownArgs &a;
    const Lists &l;
    int row0, row1, rows_per;
    float *y;              // [nb][n][kRow]
    float *side;

    __device__ __forceinline__ RowPtrs rows(int item) const
    {
        const int b = item / l.entries, q = item - b * l.entries, g = (threadIdx.x & 31) >> 2;
        const int r = row0 + b * rows_per, end = min(r + rows_per, row1);
        const int64_t row = (int64_t)l.expert[q] * a.H + r + g;
        return F::rows(a.w, row, row + 8, r + g < end, r + g + 8 < end, a.I);
    }

    __device__ __forceinline__ int blocks(int item) const
    {
        const int q = item % l.entries;
        return blocks_of(l.begin[q + 1] - l.begin[q]);
    }

    template <int NT>
    __device__ __forceinline__ void columns(int item, Columns<NT, PLANES> &x) const
    {
        x.plane_bytes = a.h.plane_bytes;
        set_columns<NT, PLANES>(l, item % l.entries, a.h.h, (int64_t)a.I * 2, 1, x);
    }

    template <int NT>
    __device__ __forceinline__ void done(int item, bool first, bool, float (&acc)[NT][4]) const
    {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
        const int b = item / l.entries, q = item - b * l.entries;
        if (!first) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                *reinterpret_cast<float4 *>(side + (nt * 32 + lane) * 4) =
                    make_float4(acc[nt][0], acc[nt][1], acc[nt][2], acc[nt][3]);
            return;
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int s = l.begin[q] + nt * 8 + 2 * t + c;
                if (s < l.begin[q + 1]) {
                    float *p = y + ((size_t)b * a.r.n + l.slot[s]) * kRow + g;
                    p[0] = acc[nt][c];
                    p[8] = acc[nt][2 + c];
                }
            }
    }
};

template <int G, int PLANES>
__global__ void __launch_bounds__(kThreads, 1)
moe_down_kernel(DownArgs a)
{
    extern __shared__ __align__(16) uint8_t dynamic[];   // ring, one side block per warp, y
    __shared__ Lists l;
    using F = typename FormatOf<G, (G > 0)>::F;
    // topk_idx was complete before the up kernel began; h is complete after the wait
    build_lists(a.r, l, reinterpret_cast<int *>(dynamic), F::kItemCost, nullptr);
    const int warp = threadIdx.x >> 5;
    uint8_t *sides = dynamic + kRingBytes;
    const int row0 = (int)((int64_t)a.H * blockIdx.x / gridDim.x);
    const int row1 = (int)((int64_t)a.H * (blockIdx.x + 1) / gridDim.x);
    const int all = (row1 - row0 + 15) / 16;       // row blocks, of equal size up to one row
    const int per = (a.I + F::kUnit - 1) / F::kUnit, K = a.r.K;
    DownItems<G, PLANES> items{a, l};
    items.rows_per = (row1 - row0 + all - 1) / all;
    items.row1 = row1;
    items.y = reinterpret_cast<float *>(sides + kWarps * kSideBytes);
    items.side = reinterpret_cast<float *>(sides + warp * kSideBytes);
    for (int b0 = 0; b0 < all; b0 += a.blocks) {
        const int nb = min(a.blocks, all - b0);
        const int n = nb * l.entries;
        items.row0 = row0 + b0 * items.rows_per;
        Stream<F, PLANES, DownItems<G, PLANES>> stream(items, a.I, n, smem_u32(dynamic));
        if (n > 0)
            stream.start();
        if (b0 == 0) {
            grid_dependency_wait();
            allow_dependents();
        }
        if (n > 0)
            stream.run();
        __syncthreads();
        // weighted sums over k; a slot's divided items are added in the order of their columns
        const int rows = min(nb * items.rows_per, row1 - items.row0);
        for (int v = threadIdx.x; v < a.T * rows; v += kThreads) {
            const int tok = v / rows, rr = v - tok * rows;
            const int b = rr / items.rows_per, i = rr - b * items.rows_per;
            float sum = 0.0f;
            for (int k = 0; k < K; ++k) {
                const int slot = tok * K + k;
                const int q = l.use[slot];
                if (q < 0)
                    continue;
                float p = items.y[((size_t)b * a.r.n + slot) * kRow + i];
                const int item = b * l.entries + q;
                // warps whose run begins inside the item
                int w = (int)((int64_t)item * per * kWarps / ((int64_t)n * per));
                const int col = l.place[slot] % kMaxCols;
                for (; w < kWarps; ++w) {
                    const int at = run_begin(n, per, w);
                    if (at >= (item + 1) * per)
                        break;
                    if (at > item * per && at < run_begin(n, per, w + 1))
                        p = __fadd_rn(p, reinterpret_cast<const float *>(sides + w * kSideBytes)[side_index(i, col)]);
                }
                sum = __fmaf_rn(a.weights[slot], p, sum);
            }
            const int64_t o = (int64_t)tok * a.H + items.row0 + rr;
            if (a.out_f32)
                static_cast<float *>(a.out)[o] = sum;
            else
                static_cast<__nv_bfloat16 *>(a.out)[o] = __float2bfloat16_rn(sum);
        }
        __syncthreads();   // y and the sides are read before the next row blocks overwrite them
    }
}

// ------------------------------------------------------------ launch policy --
constexpr size_t kMaxSmem = 227 * 1024 - sizeof(Lists) - 64;   // dynamic shared memory of a block that owns an SM
static_assert(kRingBytes + kWarps * kSideBytes + (size_t)kMaxSlots * kRow * sizeof(float) <= kMaxSmem, "one row block fits");

template <class Kernel>
int raise_smem(Kernel kernel, size_t smem, PerDevice &set)
{
    const int dev = current_device();
    if ((int)smem > set.get(dev)) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess) {
            cudaGetLastError();
            return EP_ERR_CUDA;
        }
        set.put(dev, (int)smem);
    }
    return EP_OK;
}

template <class Kernel, class Args>
int launch_dependent(Kernel kernel, unsigned grid, size_t smem, cudaStream_t stream, const Args &a)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kernel, a) != cudaSuccess) {
        cudaGetLastError();
        return EP_ERR_CUDA;
    }
    return launch_status();
}

template <int G, int PLANES>
int launch(const UpArgs &up, DownArgs down, cudaStream_t stream)
{
    const int sms = device_sm_count();
    const size_t fixed = kRingBytes + kWarps * kSideBytes;
    static_assert(EP_MAX_EXPERTS * sizeof(int) <= kRingBytes, "the experts' counters use the ring before it starts");
    {
        static PerDevice set;
        int rc = raise_smem(moe_up_kernel<G, PLANES>, fixed, set);
        if (rc != EP_OK)
            return rc;
        // one block per SM, or one per element where there are fewer
        const int64_t elements = (int64_t)std::min(up.r.n, up.r.E_local) * up.I;
        rc = launch_dependent(moe_up_kernel<G, PLANES>, (unsigned)std::min<int64_t>(elements, sms), fixed, stream, up);
        if (rc != EP_OK)
            return rc;
    }
    static PerDevice set;
    const int grid = std::min(sms, up.H);
    const size_t block = (size_t)up.r.n * kRow * sizeof(float);   // results of 16 rows
    const int all = (int)ceil_div(ceil_div(up.H, grid), 16);
    down.blocks = (int)std::min<size_t>(all, std::max<size_t>(1, (kMaxSmem - fixed) / block));
    const size_t smem = fixed + down.blocks * block;
    const int rc = raise_smem(moe_down_kernel<G, PLANES>, smem, set);
    if (rc != EP_OK)
        return rc;
    return launch_dependent(moe_down_kernel<G, PLANES>, (unsigned)grid, smem, stream, down);
}

bool matrix_ok(const ep_matrix *m)
{
    return m->data != nullptr && aligned(m->data, 16) &&
           (m->format == EP_W_BF16 ? m->scale == nullptr && m->zero == nullptr && m->group == 0
                                   : m->scale != nullptr && aligned(m->scale, 2));
}

Weights weights_of(const ep_matrix *m)
{
    return Weights{static_cast<const uint8_t *>(m->data), static_cast<const uint16_t *>(m->scale), m->zero};
}

}  // namespace
}  // namespace ep

using namespace ep;

extern "C" size_t ep_moe_workspace_size(int64_t T, int K, int I)
{
    if (T < 0 || K < 1 || I < 1)
        return 0;
    return std::max<size_t>(3 * align_up((size_t)T * K * I * 2, kWsAlign), kWsAlign);
}

extern "C" int ep_moe_decode(const void *x, const int64_t *topk_idx, const float *topk_weights, int64_t T, int K,
                             int H, int I, int E, int E_local, int rank, const ep_matrix *w13, const ep_matrix *w2,
                             void *out, int out_dtype, void *ws, size_t ws_bytes, int32_t *err, ep_stream_t stream_)
{
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    if (T < 0 || K < 1 || K > EP_MAX_TOPK || H < 8 || H % 8 != 0 || I < 8 || I % 8 != 0 || E < 1 ||
        E > EP_MAX_EXPERTS || E_local < 1 || E % E_local != 0 || rank < 0 || rank >= E / E_local || w13 == nullptr ||
        w2 == nullptr)
        return EP_ERR_INVALID_ARG;
    if ((out_dtype != 0 && out_dtype != 1) || (w13->format != EP_W_BF16 && w13->format != EP_W_INT4) ||
        w2->format != w13->format || w2->group != w13->group)
        return EP_ERR_UNSUPPORTED;
    if (w13->format == EP_W_INT4) {
        const int g = w13->group;
        if ((g != 32 && g != 64 && g != 128) || H % g != 0 || I % g != 0)
            return EP_ERR_INVALID_ARG;
    }
    if (T > kMaxSlots || T * K > kMaxSlots || H > kMaxDim || I > kMaxDim)
        return EP_ERR_UNSUPPORTED;
    if (T == 0)
        return EP_OK;
    if (x == nullptr || topk_idx == nullptr || topk_weights == nullptr || out == nullptr || !aligned(x, 16) ||
        !aligned(out, 16) || !matrix_ok(w13) || !matrix_ok(w2) || ws == nullptr || !aligned(ws, kWsAlign) ||
        ws_bytes < ep_moe_workspace_size(T, K, I))
        return EP_ERR_INVALID_ARG;
    const int n = (int)T * K;
    const Routing r{topk_idx, n, K, E, E_local, (int64_t)rank * E_local};
    const Planes h{static_cast<uint8_t *>(ws), (int64_t)align_up((size_t)n * I * 2, kWsAlign), I};
    const UpArgs up{static_cast<const uint8_t *>(x), r, H, I, weights_of(w13), h, err};
    const DownArgs down{r, topk_weights, (int)T, H, I, weights_of(w2), h, out, out_dtype, 1};
    switch (w13->group + out_dtype) {   // group: 0, 32, 64 or 128
    case 0: return launch<0, 2>(up, down, stream);
    case 1: return launch<0, 3>(up, down, stream);
    case 32: return launch<32, 2>(up, down, stream);
    case 33: return launch<32, 3>(up, down, stream);
    case 64: return launch<64, 2>(up, down, stream);
    case 65: return launch<64, 3>(up, down, stream);
    case 128: return launch<128, 2>(up, down, stream);
    default: return launch<128, 3>(up, down, stream);
    }
}
