// The experts of a mixture-of-experts layer for a few tokens, in two kernels
// (internal; the entry point is in ep_moe.cu).
//
//   up:    h[s] = silu(Wg x) * (Wu x) for every slot s = (t, k) that names a
//          local expert;
//   down:  out[t] = sum over k of w[t,k] * (W2 h[t,k]).
//
// Each expert that some token names has its matrices read once for every 16 of
// its slots, by products of blocks of 16 weight rows with the slots as columns
// (ep_skinny.cuh).  (Passes of 32 slots, tried twice, lost more to their
// registers than the reads of the second pass take.)  No row of x is copied to
// an expert and no list is made on the host: every block derives the experts in
// use and their slots from topk_idx, which a graph replay may have changed.
//
// up: the elements of h of all experts in use, laid end to end, are dealt to
// one block per SM in equal runs.  An item is up to 32 elements: 8 gate rows and
// the 8 up rows of the same elements are the 16 rows of a matrix step, whose
// accumulators hold gate and up of an element in the same lane.
//
// down: each block owns an equal share of the output's rows and adds up all
// experts for them.  An item is up to 48 of its rows of one expert.  Every
// slot's results stay in shared memory (in the workspace, which means in L2,
// when there are too many) and are weighted and added by the same block in
// ascending k.
//
// In both the block's items are shared evenly by its warps, whose runs may stop
// inside an item; the pieces of a divided item are added in the order of their
// columns.  Nothing depends on the order of arrival.
//
// h is kept whole: as the three bf16 terms of a sum (24 significant bits), which
// is what the matrix step takes.  One bf16 would add an error as large as the
// rounding of the result itself, and with two (16 bits) about one bf16 result
// in 270 rounded the other way.
//
// Measured (up + down, of the bytes of the experts in use at 6.79 TB/s): one
// token, 6 of 64 bf16 experts 2048x1024, 20.9 us (0.53); 128 tokens, 128 bf16
// experts 4096x1536, 814 us (0.87); 64 tokens, 31 of 32 bf16 experts 7168x2048
// with 44 passes, 588 us (0.70); one token, 8 4-bit experts 7168x2048 in groups
// of 128, 59.3 us (0.45); 13 tokens, 32 4-bit experts 4160x1472 in groups of 64,
// 68.3 us (0.38).  (With two terms of h these were 20.4, 781, 585 and 54.5 us;
// the last had an fp32 result and three.)  4-bit down holds x of a unit in up to
// 192 registers and spills in its loop.
#pragma once

#include <algorithm>

#include "ep_device.cuh"
#include "ep_internal.h"
#include "ep_launch.cuh"
#include "ep_skinny.cuh"

namespace ep {

constexpr int kMostWarps = 8;    // of a block, in either format
constexpr int kMaxSlots = EP_MOE_MAX_SLOTS;
constexpr int kMaxDim = 65536;   // H and I: a block's units are counted in 32 bits

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

__device__ __forceinline__ int passes_of(int slots) { return (slots + kMaxCols - 1) / kMaxCols; }

// The experts in use and their slots, in shared memory.  An expert has an entry
// for each pass over its weights, of up to 16 slots.
struct Lists {
    int experts, entries, big;
    int scan[3][kMostWarps];
    uint16_t id[kMaxSlots];           // expert j's local id
    uint16_t entry[kMaxSlots + 1];    // its first entry: it has entry[j] .. entry[j+1]
    uint16_t owner[kMaxSlots];        // entry -> j
    uint16_t begin[kMaxSlots + 1];    // slots of entry q: slot[begin[q] .. begin[q+1])
    uint16_t slot[kMaxSlots];
    int16_t use[kMaxSlots];           // slot -> its entry, or -1
    uint16_t place[kMaxSlots];        // slot -> its place among its expert's slots
    float weight[kMaxSlots];          // down: the slots' weights
    uint16_t big_expert[kMaxSlots / kMaxCols];   // experts of more than one entry
};

// build_lists for up to 32 slots, by the first warp: one slot to a lane.  The
// experts come in the order of their first slots.  (One token of 6 bf16 experts
// 2048x1024: 20.9 us, with the general lists 22.0; of 8 4-bit experts
// 7168x2048: 59.3 and 62.9.)
__device__ __forceinline__ void build_few(const Routing &r, Lists &l, int32_t *err)
{
    if (threadIdx.x < 32) {
        const int s = threadIdx.x;
        const int e = s < r.n ? r.local(s, err) : -1;
        const unsigned lt = lanemask_lt(), peers = __match_any_sync(kFull, e), before = peers & lt;
        const int c = __popc(peers);
        const unsigned leaders = __ballot_sync(kFull, e >= 0 && before == 0);
        // 32 slots are two passes at most
        const unsigned twice = __ballot_sync(kFull, e >= 0 && before == 0 && c > kMaxCols);
        const int leader = __ffs(peers) - 1;
        const unsigned earlier = e >= 0 ? (1u << leader) - 1 : 0;   // lanes below this expert's first
        const int j = __popc(leaders & earlier), q = j + __popc(twice & earlier);
        int at = 0;   // slots of the experts before
        for (unsigned m = leaders; m != 0; m &= m - 1) {
            const int o = __ffs(m) - 1, n = __shfl_sync(kFull, c, o);
            if (earlier >> o & 1)
                at += n;
        }
        const int place = __popc(before);
        if (s < r.n) {
            l.use[s] = e >= 0 ? (int16_t)(q + place / kMaxCols) : (int16_t)-1;
            l.place[s] = (uint16_t)place;
        }
        if (e >= 0) {
            l.slot[at + place] = (uint16_t)s;
            if (before == 0) {
                l.id[j] = (uint16_t)e;
                l.entry[j] = (uint16_t)q;
                for (int p = 0; p < passes_of(c); ++p) {
                    l.owner[q + p] = (uint16_t)j;
                    l.begin[q + p] = (uint16_t)(at + p * kMaxCols);
                }
            }
        }
        if (s == 0) {
            const int experts = __popc(leaders), entries = experts + __popc(twice);
            l.experts = experts;
            l.entries = entries;
            l.entry[experts] = (uint16_t)entries;
        }
        const int slots = __popc(__ballot_sync(kFull, e >= 0));
        if (s == 0)
            l.begin[__popc(leaders) + __popc(twice)] = (uint16_t)slots;
    }
    __syncthreads();
}

// All threads of the block, WARPS warps; count: E_local ints of shared memory.
template <int WARPS>
__device__ __forceinline__ void build_lists(const Routing &r, Lists &l, int *count, int32_t *err)
{
    if (r.n <= 32) {
        build_few(r, l, err);
        return;
    }
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int e = tid; e < r.E_local; e += (32 * WARPS))
        count[e] = 0;
    if (tid == 0)
        l.big = 0;
    __syncthreads();
    for (int s = tid; s < r.n; s += (32 * WARPS)) {
        const int e = r.local(s, err);
        l.use[s] = (int16_t)e;
        if (e >= 0)
            l.place[s] = (uint16_t)atomicAdd(&count[e], 1);
    }
    __syncthreads();
    // each thread owns a run of experts; scans of (experts in use, entries, slots)
    const int per = (r.E_local + (32 * WARPS) - 1) / (32 * WARPS);
    const int e0 = min(tid * per, r.E_local), e1 = min(e0 + per, r.E_local);
    int own[3] = {0, 0, 0};
    for (int e = e0; e < e1; ++e) {
        const int c = count[e];
        own[0] += c > 0;
        own[1] += passes_of(c);
        own[2] += c;
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
    int j = sum[0], q = sum[1], at = sum[2];
    for (int e = e0; e < e1; ++e) {
        const int c = count[e];
        count[e] = q;
        if (c == 0)
            continue;
        if (c > kMaxCols)
            l.big_expert[atomicAdd(&l.big, 1)] = (uint16_t)e;
        l.id[j] = (uint16_t)e;
        l.entry[j] = (uint16_t)q;
        for (int b = 0; b < c; b += kMaxCols) {
            l.owner[q] = (uint16_t)j;
            l.begin[q++] = (uint16_t)(at + b);
        }
        ++j;
        at += c;
    }
    if (tid == (32 * WARPS) - 1) {
        l.experts = j;
        l.entries = q;
        l.entry[j] = (uint16_t)q;
        l.begin[q] = (uint16_t)at;
    }
    __syncthreads();
    // The order of slots within an entry moves no result, but every block must put the same slots into an
    // entry: where an expert has several, its slots take their places in ascending order.
    if (l.big > 0) {
        for (int b = warp; b < l.big; b += WARPS) {
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
    for (int s = tid; s < r.n; s += (32 * WARPS)) {
        const int e = l.use[s];
        if (e >= 0) {
            const int p = l.place[s], f = count[e];
            l.slot[l.begin[f] + p] = (uint16_t)s;
            l.use[s] = (int16_t)(f + p / kMaxCols);
        }
    }
    __syncthreads();
}

constexpr int kPlanes = 3;   // bf16 terms of h

struct Planes {
    uint8_t *h;            // [kPlanes][n][I] bf16
    int64_t plane_bytes;
    int I;
};

// h as a sum of bf16 terms, each the next 8 of its 24 bits and toward zero, so
// that a term never rounds up to infinity; an infinity or NaN is its own first
// term
template <bool PERMUTED>
__device__ __forceinline__ void store_planes(const Planes &p, int slot, int i, float h)
{
    const int place = (i & ~7) | column_place<PERMUTED>(i & 7);
    uint8_t *at = p.h + ((int64_t)slot * p.I + place) * 2;
    float rest = h;
#pragma unroll
    for (int q = 0; q < kPlanes; ++q) {
        const float term = __uint_as_float(__float_as_uint(rest) & 0xffff0000u);
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
        x.set(nt, s < end ? rows + (int64_t)(l.slot[s] / slots_per_row) * row_bytes : nullptr, (int)(row_bytes / 2));
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

// A block's elements: from element i0 of expert j0 to element i1 of expert j1
// (exclusive), in items that do not cross experts.  An expert's passes follow
// one another over all of its elements in the block, so that two passes read
// the same rows at about the same time, in different warps, and the second
// finds them in L2 (64 tokens, 44 passes for 31 experts: 585 us; with the passes
// of each item in turn, an item of 900 KB apart in every warp, 624).
template <int G, int RB>
struct UpItems {
    using F = typename FormatOf<G, false>::F;
    static constexpr int kStep = 8;
    const UpArgs &a;
    const Lists &l;
    int j0, i0, j1, i1;
    int head, body;        // items of the first expert, all passes; of a whole expert in one pass
    float *side;           // this warp's kept piece of an item that another warp began
    float *open;           // its kept piece of an item that it began and another goes on with

    __device__ __forceinline__ int passes(int j) const { return l.entry[j + 1] - l.entry[j]; }

    mutable int open_q, open_i, open_end;   // the item that it began: its entry and elements

    static __device__ __forceinline__ int cut(int elements) { return (elements + 8 * RB - 1) / (8 * RB); }

    __device__ __forceinline__ UpItems(const UpArgs &args, const Lists &lists, int ja, int ia, int jb, int ib)
        : a(args), l(lists), j0(ja), i0(ia), j1(jb), i1(ib)
    {
        const int first = (j1 > j0 ? a.I : i1) - i0;
        head = first > 0 ? cut(first) * passes(j0) : 0;
        body = cut(a.I);
    }

    __device__ __forceinline__ int count() const
    {
        int n = head;
        if (j1 > j0) {
            n += body * (l.entry[j1] - l.entry[j0 + 1]);
            if (i1 > 0)
                n += cut(i1) * passes(j1);
        }
        return n;
    }

    // item -> its entry, expert, and elements [i, end)
    __device__ __forceinline__ void where(int item, int &q, int &j, int &i, int &end) const
    {
        int v = item;
        j = j0;
        i = i0;
        if (item >= head) {
            const int q1 = l.entry[j0 + 1];
            v -= head;
            j = l.owner[q1 + quick_div(v, body)];
            v -= body * (l.entry[j] - q1);
            i = 0;
        }
        const int stop = j == j1 ? i1 : a.I;
        int pass = 0, block = v;
        if (passes(j) > 1) {
            const int blocks = cut(stop - i);
            pass = quick_div(v, blocks);
            block = v - pass * blocks;
        }
        i += block * (8 * RB);
        q = l.entry[j] + pass;
        end = min(i + 8 * RB, stop);
    }

    __device__ __forceinline__ RowRange rows(int item) const
    {
        int q, j, i, end;
        where(item, q, j, i, end);
        const int64_t row = (int64_t)l.id[j] * 2 * a.I + i;
        return RowRange{row, row + a.I, end - i, end - i};
    }

    __device__ __forceinline__ int cols(int item) const
    {
        int q, j, i, end;
        where(item, q, j, i, end);
        return l.begin[q + 1] - l.begin[q];
    }

    template <int NT>
    __device__ __forceinline__ void columns(int item, Columns<NT, 1> &x) const
    {
        int q, j, i, end;
        where(item, q, j, i, end);
        x.plane_bytes = 0;
        set_columns<NT, 1>(l, q, a.x, (int64_t)a.H * 2, a.r.K, x);
    }

    template <int NT>
    __device__ __forceinline__ void done(int item, bool first, bool last, const float (&acc)[RB][NT][4]) const
    {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
        int q, j, i, end;
        where(item, q, j, i, end);
        if (!first || !last) {
            keep<RB, NT>(first ? open : side, acc);
            if (first) {
                open_q = q;
                open_i = i;
                open_end = end;
            }
            return;
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int s = l.begin[q] + nt * 8 + 2 * t + c;
                if (s < l.begin[q + 1])
#pragma unroll
                    for (int r = 0; r < RB; ++r)
                        if (i + 8 * r + g < end)
                            store_planes<(G > 0)>(a.out, l.slot[s], i + 8 * r + g,
                                                  activate(acc[r][nt][c], acc[r][nt][2 + c]));
            }
    }
};

// The expert and element where the shares of blocks b and b + 1 begin, by lanes 0
// and 1 of every warp: an element costs its expert's passes, each of which reads
// its rows again.  (At most kMaxSlots * kMaxDim = 2^26 in all.)
__device__ __forceinline__ void share(const Lists &l, int I, int b, int blocks, int &j0, int &i0, int &j1, int &i1)
{
    const int total = l.entry[l.experts] * I, each = quick_div(total, blocks), rest = total - each * blocks;
    b += threadIdx.x & 1;
    const int pos = each * b + min(b, rest);
    int lo = 0, hi = l.experts;   // entry[lo] * I <= pos < entry[hi] * I
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (l.entry[mid] * I <= pos)
            lo = mid;
        else
            hi = mid;
    }
    const int at = l.entry[lo], cost = l.entry[lo + 1] - at;
    int i = quick_div(pos - at * I, cost);
    if (b == blocks) {
        lo = l.experts;
        i = 0;
    }
    j0 = __shfl_sync(kFull, lo, 0);
    i0 = __shfl_sync(kFull, i, 0);
    j1 = __shfl_sync(kFull, lo, 1);
    i1 = __shfl_sync(kFull, i, 1);
}

template <int G, int RB>
__global__ void __launch_bounds__(32 * FormatOf<G, false>::F::kWarps, 1)
moe_up_kernel(UpArgs a)
{
    extern __shared__ __align__(128) uint8_t dynamic[];   // ring, then one side block per warp
    __shared__ Lists l;
    using F = typename FormatOf<G, false>::F;
    __shared__ int begins[F::kWarps + 1];
    grid_dependency_wait();
    allow_dependents();
    build_lists<F::kWarps>(a.r, l, reinterpret_cast<int *>(dynamic), blockIdx.x == 0 ? a.err : nullptr);
    if (l.experts == 0)
        return;
    const int warp = threadIdx.x >> 5;
    uint8_t *sides = dynamic + Room<F, RB>::kRing;
    int j0, i0, j1, i1;
    share(l, a.I, blockIdx.x, gridDim.x, j0, i0, j1, i1);
    UpItems<G, RB> items(a, l, j0, i0, j1, i1);
    items.side = reinterpret_cast<float *>(sides + warp * Room<F, RB>::kSide);
    items.open = reinterpret_cast<float *>(dynamic + warp * Room<F, RB>::kWarpRing);   // the ring is idle by then
    const int n = items.count();
    if (n == 0)
        return;
    Stream<F, RB, 1, UpItems<G, RB>> stream(items, a.w, a.H, n, smem_u32(dynamic));
    stream.start();
    stream.run();
    stream.meet(begins);
    if (stream.open_item >= 0) {
        const int first = l.begin[items.open_q], cols = l.begin[items.open_q + 1] - first, nb = cols <= 8 ? 1 : 2;
        for (int v = threadIdx.x & 31; v < 8 * RB * cols; v += 32) {
            const int e = v % (8 * RB), c = v / (8 * RB), i = items.open_i + e;
            const int at[2] = {side_index(e >> 3, e & 7, nb, c), side_index(e >> 3, (e & 7) + 8, nb, c)};
            float sum[2];
            stream.template add_pieces<2>(dynamic, at, sum);
            if (i < items.open_end)
                store_planes<(G > 0)>(a.out, l.slot[first + c], i, activate(sum[0], sum[1]));
        }
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
    int each, rest;    // output rows of a block; the first `rest` blocks have one more
    float *y;          // [n][H] of the workspace, or null where the slots' results fit in shared memory
};

// A block's output rows [row0, row1) in groups of up to 16*RB, times all entries.
template <int G, int RB>
struct DownItems {
    using F = typename FormatOf<G, (G > 0)>::F;
    static constexpr int kStep = 16;
    const DownArgs &a;
    const Lists &l;
    int row0, row1;
    float *y;              // [n], `stride` floats apart: the block's rows of each slot
    int stride;
    float *side, *open;    // this warp's kept pieces: of an item begun by another, and of one it began

    __device__ __forceinline__ RowRange rows(int item) const
    {
        const int b = quick_div(item, l.entries), q = item - b * l.entries;
        const int r = row0 + b * (16 * RB), n = min(row1 - r, 16 * RB);
        const int64_t row = (int64_t)l.id[l.owner[q]] * a.H + r;
        return RowRange{row, row + 8, n, n - 8};
    }

    __device__ __forceinline__ int cols(int item) const
    {
        const int q = item - quick_div(item, l.entries) * l.entries;
        return l.begin[q + 1] - l.begin[q];
    }

    template <int NT>
    __device__ __forceinline__ void columns(int item, Columns<NT, kPlanes> &x) const
    {
        x.plane_bytes = a.h.plane_bytes;
        set_columns<NT, kPlanes>(l, item - quick_div(item, l.entries) * l.entries, a.h.h, (int64_t)a.I * 2, 1, x);
    }

    template <int NT>
    __device__ __forceinline__ void done(int item, bool first, bool last, const float (&acc)[RB][NT][4]) const
    {
        if (!first || !last) {
            keep<RB, NT>(first ? open : side, acc);
            return;
        }
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
        const int b = item / l.entries, q = item - b * l.entries, rows = row1 - row0;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int s = l.begin[q] + nt * 8 + 2 * t + c;
                if (s < l.begin[q + 1]) {
                    float *p = y + (int64_t)l.slot[s] * stride;
#pragma unroll
                    for (int r = 0; r < RB; ++r) {
                        const int i = (b * RB + r) * 16 + g;
                        if (i < rows)
                            p[i] = acc[r][nt][c];
                        if (i + 8 < rows)
                            p[i + 8] = acc[r][nt][2 + c];
                    }
                }
            }
    }
};

template <int G, int RB>
__global__ void __launch_bounds__(32 * FormatOf<G, (G > 0)>::F::kWarps, 1)
moe_down_kernel(DownArgs a)
{
    extern __shared__ __align__(128) uint8_t dynamic[];   // ring, one side block per warp, y if it fits
    __shared__ Lists l;
    using F = typename FormatOf<G, (G > 0)>::F;
    __shared__ int begins[F::kWarps + 1];
    // topk_idx was complete before the up kernel began; h is complete after the wait
    const float weight = threadIdx.x < a.r.n ? a.weights[threadIdx.x] : 0.0f;   // in flight while the lists are built
    build_lists<F::kWarps>(a.r, l, reinterpret_cast<int *>(dynamic), nullptr);
    l.weight[threadIdx.x] = weight;
    for (int s = threadIdx.x + 32 * F::kWarps; s < a.r.n; s += 32 * F::kWarps)
        l.weight[s] = a.weights[s];
    const int warp = threadIdx.x >> 5;
    uint8_t *sides = dynamic + Room<F, RB>::kRing;
    DownItems<G, RB> items{a, l};
    items.row0 = a.each * blockIdx.x + min((int)blockIdx.x, a.rest);
    items.row1 = items.row0 + a.each + ((int)blockIdx.x < a.rest ? 1 : 0);
    const int rows = items.row1 - items.row0;
    items.y = a.y != nullptr ? a.y + items.row0 : reinterpret_cast<float *>(dynamic + Room<F, RB>::kFixed);
    items.stride = a.y != nullptr ? a.H : rows | 1;
    items.side = reinterpret_cast<float *>(sides + warp * Room<F, RB>::kSide);
    items.open = reinterpret_cast<float *>(dynamic + warp * Room<F, RB>::kWarpRing);
    const int n = (rows + 16 * RB - 1) / (16 * RB) * l.entries;
    Stream<F, RB, kPlanes, DownItems<G, RB>> stream(items, a.w, a.I, n, smem_u32(dynamic));
    stream.start();
    grid_dependency_wait();
    allow_dependents();
    stream.run();
    stream.meet(begins);
    if (stream.open_item >= 0) {
        const int b = quick_div(stream.open_item, l.entries), q = stream.open_item - b * l.entries;
        const int first = l.begin[q], cols = l.begin[q + 1] - first, nb = cols <= 8 ? 1 : 2;
        for (int v = threadIdx.x & 31; v < 16 * RB * cols; v += 32) {
            const int r = v % (16 * RB), c = v / (16 * RB), i = b * (16 * RB) + r;
            if (i < rows) {
                const int at[1] = {side_index(r >> 4, r & 15, nb, c)};
                float sum[1];
                stream.template add_pieces<1>(dynamic, at, sum);
                items.y[(int64_t)l.slot[first + c] * items.stride + i] = sum[0];
            }
        }
    }
    __syncthreads();
    for (int v = threadIdx.x; v < a.T * rows; v += 32 * F::kWarps) {
        const int tok = quick_div(v, rows), i = v - tok * rows;
        float sum = 0.0f;
        for (int k = 0; k < a.r.K; ++k) {
            const int slot = tok * a.r.K + k;
            if (l.use[slot] >= 0)
                sum = __fmaf_rn(l.weight[slot], items.y[(int64_t)slot * items.stride + i], sum);
        }
        const int64_t o = (int64_t)tok * a.H + items.row0 + i;
        if (a.out_f32)
            static_cast<float *>(a.out)[o] = sum;
        else
            static_cast<__nv_bfloat16 *>(a.out)[o] = __float2bfloat16_rn(sum);
    }
}

// ------------------------------------------------------------ launch policy --
// Dynamic shared memory of a block that owns an SM: all but the static part, both rounded up to the dynamic one's
// alignment of 128 bytes.
constexpr size_t kMaxSmem = 227 * 1024 - sizeof(Lists) - (kMostWarps + 1) * sizeof(int) - 256;

template <int G, int RB>
int launch_up(const UpArgs &a, int64_t elements, cudaStream_t stream)
{
    using F = typename FormatOf<G, false>::F;
    constexpr int kSmem = Room<F, RB>::kFixed;
    static_assert(EP_MAX_EXPERTS * sizeof(int) <= Room<F, RB>::kRing,
                  "the experts' counters use the ring before it starts");
    static_assert(kSmem <= kMaxSmem, "a block fits");
    static PerDevice set;
    const int rc = raise_smem(moe_up_kernel<G, RB>, kSmem, set);
    if (rc != EP_OK)
        return rc;
    const unsigned grid = (unsigned)std::min<int64_t>(elements, device_sm_count());
    return launch_dependent(moe_up_kernel<G, RB>, grid, 32 * F::kWarps, kSmem, stream, a);
}

template <int G, int RB>
int launch_down(DownArgs a, unsigned grid, cudaStream_t stream)
{
    using F = typename FormatOf<G, (G > 0)>::F;
    a.each = a.H / (int)grid;
    a.rest = a.H % (int)grid;
    static PerDevice set;
    // the slots' results stay in shared memory where there is room for them (128 tokens of 8 experts: 814 us, in the
    // workspace 827; 64 tokens of 4: 448 and 457; one token: alike)
    const size_t y = (size_t)a.r.n * ((size_t)ceil_div(a.H, grid) | 1) * sizeof(float);
    size_t smem = Room<F, RB>::kFixed;
    if (smem + y <= kMaxSmem) {
        smem += y;
        a.y = nullptr;
    }
    const int rc = raise_smem(moe_down_kernel<G, RB>, kMaxSmem, set);
    if (rc != EP_OK)
        return rc;
    return launch_dependent(moe_down_kernel<G, RB>, grid, 32 * F::kWarps, smem, stream, a);
}

template <int G, int RB = FormatOf<G, false>::F::kMaxBlocks>
int launch_up_blocks(const UpArgs &a, int64_t elements, int blocks, cudaStream_t stream)
{
    if constexpr (RB > 1) {
        if (blocks < RB)
            return launch_up_blocks<G, RB - 1>(a, elements, blocks, stream);
    }
    return launch_up<G, RB>(a, elements, stream);
}

constexpr int kMostDown = 3;   // row blocks of down at a time: 48 rows are a block's share up to H = 7296

template <int G, int RB>
int launch_down_blocks(const DownArgs &a, unsigned grid, int blocks, cudaStream_t stream)
{
    if constexpr (RB > 1) {
        if (blocks < RB)
            return launch_down_blocks<G, RB - 1>(a, grid, blocks, stream);
    }
    return launch_down<G, RB>(a, grid, stream);
}

template <int G>
int launch(const UpArgs &up, const DownArgs &down, cudaStream_t stream)
{
    constexpr int kMost = FormatOf<G, false>::F::kMaxBlocks, kDown = kMost < kMostDown ? kMost : kMostDown;
    const int sms = device_sm_count();
    // at most: the experts in use are not known here
    const int64_t elements = (int64_t)std::min(up.r.n, up.r.E_local) * up.I;
    const int up_blocks = blocks_at_once(ceil_div(ceil_div(elements, sms), 8), kMost, G > 0);
    const int rc = launch_up_blocks<G>(up, elements, up_blocks, stream);
    if (rc != EP_OK)
        return rc;
    const unsigned grid = (unsigned)std::min(sms, down.H);
    const int blocks = blocks_at_once(ceil_div(ceil_div(down.H, grid), 16), kDown, G > 0);
    return launch_down_blocks<G, kDown>(down, grid, blocks, stream);
}

}  // namespace ep
