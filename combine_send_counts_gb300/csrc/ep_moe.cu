// The experts of a mixture-of-experts layer for a few tokens, in two kernels.
//
//   up:    h[s] = silu(Wg x) * (Wu x) for every slot s = (t, k) that names a
//          local expert;
//   down:  out[t] = sum over k of w[t,k] * (W2 h[t,k]).
//
// Each expert that some token names has its matrices read once for all its
// slots (up to 32 at a time), by products of 16 weight rows with the slots as
// columns (ep_skinny.cuh).  No row of x is copied to an expert and no list is
// made on the host: every block derives the experts in use and their slots
// from topk_idx, which a graph replay may have changed.
//
// up's 16 rows are 8 gate rows and the 8 up rows of the same elements, which
// the matrix step's accumulators hold in the same lane; a block is one of a
// resident wave and takes (expert, 8 elements) units, whose columns S of its
// warps share, S chosen so that the units fill the wave evenly.
//
// down gives 16 rows of the output to a thread-block cluster, whose warps
// share the experts (and their columns when there are fewer experts than
// warps).  Each slot's 16 partial results stay in the shared memory of the
// block that made them and are weighted and added from there in ascending k,
// so nothing but out is written and nothing depends on the order of arrival.
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

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxBlocks8 = 4;          // blocks of 8 slots in one pass over the weights
constexpr int kMaxSlots = EP_MOE_MAX_SLOTS;
constexpr int kRow = 20;                // floats between slots in shared memory: 16 rows, no bank conflicts

struct Weights {
    const uint8_t *data;
    const uint16_t *scale;
    const uint8_t *zero;
};

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

// The experts in use and the slots of each, in shared memory.
struct Lists {
    int active;                       // experts in use
    int warp_sum[kWarps], warp_used[kWarps];
    uint16_t expert[kMaxSlots];       // [active]
    uint16_t begin[kMaxSlots + 1];    // slots of the j-th: slot[begin[j] .. begin[j+1])
    uint16_t slot[kMaxSlots];
    int16_t use[kMaxSlots];           // slot -> j, or -1
    uint16_t place[kMaxSlots];
};

// All threads of the block; count: E_local ints of shared memory.
__device__ __forceinline__ void build_lists(const Routing &r, Lists &l, int *count, int32_t *err)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int e = tid; e < r.E_local; e += kThreads)
        count[e] = 0;
    __syncthreads();
    for (int s = tid; s < r.n; s += kThreads) {
        const int e = r.local(s, err);
        l.use[s] = (int16_t)e;
        if (e >= 0)
            l.place[s] = (uint16_t)atomicAdd(&count[e], 1);   // the order within an expert moves no result
    }
    __syncthreads();
    // each thread owns a run of experts; scan of (experts in use, slots)
    const int per = (r.E_local + kThreads - 1) / kThreads;
    const int e0 = min(tid * per, r.E_local), e1 = min(e0 + per, r.E_local);
    int used = 0, slots = 0;
    for (int e = e0; e < e1; ++e) {
        used += count[e] > 0;
        slots += count[e];
    }
    int su = used, ss = slots;
    for (int o = 1; o < 32; o <<= 1) {
        const int a = __shfl_up_sync(kFull, su, o), b = __shfl_up_sync(kFull, ss, o);
        if (lane >= o) {
            su += a;
            ss += b;
        }
    }
    if (lane == 31) {
        l.warp_used[warp] = su;
        l.warp_sum[warp] = ss;
    }
    __syncthreads();
    int j = su - used, at = ss - slots;
    for (int w = 0; w < warp; ++w) {
        j += l.warp_used[w];
        at += l.warp_sum[w];
    }
    for (int e = e0; e < e1; ++e) {
        const int c = count[e];
        if (c > 0) {
            l.expert[j] = (uint16_t)e;
            l.begin[j] = (uint16_t)at;
            count[e] = j++;
            at += c;
        }
    }
    if (tid == kThreads - 1) {
        l.active = j;
        l.begin[j] = (uint16_t)at;
    }
    __syncthreads();
    for (int s = tid; s < r.n; s += kThreads) {
        const int e = l.use[s];
        if (e >= 0) {
            const int jj = count[e];
            l.slot[l.begin[jj] + l.place[s]] = (uint16_t)s;
            l.use[s] = (int16_t)jj;
        }
    }
    __syncthreads();
}

// The weight format of a kernel: G = 0 for bf16, else the group of 4-bit codes.
template <int G, bool PERMUTED>
struct Format {
    using Rows = RowsW4<G, PERMUTED>;
    static __device__ __forceinline__ Rows rows(const Weights &w, int64_t a, int64_t b, int K)
    {
        const int64_t bytes = K / 2, groups = K / G;
        return Rows{w.data + a * bytes, w.data + b * bytes, w.scale + a * groups, w.scale + b * groups,
                    w.zero != nullptr ? w.zero + a * groups : nullptr, w.zero != nullptr ? w.zero + b * groups : nullptr};
    }
};
template <bool PERMUTED>
struct Format<0, PERMUTED> {
    using Rows = RowsBf16;
    static __device__ __forceinline__ Rows rows(const Weights &w, int64_t a, int64_t b, int K)
    {
        const int64_t bytes = (int64_t)K * 2;
        return Rows{w.data + a * bytes, w.data + b * bytes};
    }
};

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

// (the truncated form above would turn a NaN whose payload sits in the low half into an infinity)
__device__ __forceinline__ float quiet(float v) { return isnan(v) ? __int_as_float(0x7fffffff) : v; }

__device__ __forceinline__ void group_sync(int id, int threads)
{
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// slots [base, base + 8*NT) of the list [first, end) times 16 rows, one warp's columns [u0, u1)
template <class F, int PLANES, int NT>
__device__ __forceinline__ void pass(const F &f, const Lists &l, int first, int end, const uint8_t *cols,
                                     int64_t row_bytes, int slots_per_row, int64_t plane_bytes, int u0, int u1, int K,
                                     float (&acc)[NT][4])
{
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    Columns<NT, PLANES> x;
    x.plane_bytes = plane_bytes;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int q = first + nt * 8 + g;
        x.p[nt] = q < end ? cols + (int64_t)(l.slot[q] / slots_per_row) * row_bytes : nullptr;
#pragma unroll
        for (int c = 0; c < 4; ++c)
            acc[nt][c] = 0.0f;
    }
    skinny<F, NT, PLANES>(f, u0, u1, K, t, x, acc);
}

struct UpArgs {
    const uint8_t *x;
    Routing r;
    int H, I;
    Weights w;
    Planes out;
    int32_t *err;
};

template <int G, int PLANES, int NT>
__device__ __forceinline__ void up_unit(const UpArgs &a, const Lists &l, int j, int tile, int base, int S, int part,
                                        int sub, float *red)
{
    using F = typename Format<G, false>::Rows;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int first = l.begin[j] + base, end = l.begin[j + 1];
    const int64_t row = (int64_t)l.expert[j] * 2 * a.I + tile * 8 + g;
    const F f = Format<G, false>::rows(a.w, row, row + a.I, a.H);
    const int units = (a.H + F::kUnit - 1) / F::kUnit;
    float acc[NT][4];
    pass<F, 1, NT>(f, l, first, end, a.x, (int64_t)a.H * 2, a.r.K, 0, units * part / S, units * (part + 1) / S, a.H,
                   acc);
    auto emit = [&](int q, float gate, float up) {
        const float h = quiet(__fmul_rn(__fdiv_rn(gate, __fadd_rn(1.0f, expf(-gate))), up));
        return h;
    };
    if (S == 1) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int q = first + nt * 8 + 2 * t + c;
                if (q < end)
                    store_planes<PLANES, (G > 0)>(a.out, l.slot[q], tile * 8 + g, emit(q, acc[nt][c], acc[nt][2 + c]));
            }
        return;
    }
    // the S warps' partial sums, added in ascending order of their columns
    float *mine = red + (size_t)part * NT * 128;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
        *reinterpret_cast<float4 *>(mine + (nt * 32 + lane) * 4) =
            make_float4(acc[nt][0], acc[nt][1], acc[nt][2], acc[nt][3]);
    group_sync(1 + sub, 32 * S);
    for (int v = part * 32 + lane; v < NT * 64; v += 32 * S) {
        // v: (block, lane that held it, which of its two columns)
        const int c = v & 1, src = (v >> 1) & 31, nt = v >> 6;
        const int q = first + nt * 8 + 2 * (src & 3) + c;
        if (q < end) {
            float gate = 0.0f, up = 0.0f;
            for (int s = 0; s < S; ++s) {
                const float *p = red + ((size_t)s * NT * 32 + nt * 32 + src) * 4;
                gate = __fadd_rn(gate, p[c]);
                up = __fadd_rn(up, p[2 + c]);
            }
            store_planes<PLANES, (G > 0)>(a.out, l.slot[q], tile * 8 + (src >> 2), emit(q, gate, up));
        }
    }
    group_sync(1 + sub, 32 * S);   // the sums are read before the next unit's overwrite them
}

template <int G, int PLANES>
__global__ void __launch_bounds__(kThreads, 2)
moe_up_kernel(UpArgs a)
{
    extern __shared__ __align__(16) uint8_t dynamic[];
    __shared__ Lists l;
    int *count = reinterpret_cast<int *>(dynamic);
    float *red = reinterpret_cast<float *>(dynamic);   // after the lists are built
    grid_dependency_wait();
    allow_dependents();
    build_lists(a.r, l, count, blockIdx.x == 0 ? a.err : nullptr);
    const int warp = threadIdx.x >> 5;
    const int tiles = a.I / 8;
    const int64_t units = (int64_t)l.active * tiles;
    // S warps to a unit: the S in 1, 2, 4, 8 that leaves the fullest last wave, the smaller on a tie
    const int64_t W = (int64_t)gridDim.x * kWarps;
    int S = 1;
    int64_t best = (units + W - 1) / W * kWarps;   // rounds, in eighths of a unit's time
    for (int s = 2; s <= kWarps; s *= 2) {
        const int64_t cost = (units * s + W - 1) / W * (kWarps / s);
        if (cost < best) {
            best = cost;
            S = s;
        }
    }
    const int sub = warp / S, part = warp % S, subs = kWarps / S;
    float *mine = red + (size_t)sub * S * kMaxBlocks8 * 128;
    for (int64_t u = (int64_t)blockIdx.x * subs + sub; u < units; u += (int64_t)gridDim.x * subs) {
        const int j = (int)(u / tiles), tile = (int)(u % tiles);
        const int m = l.begin[j + 1] - l.begin[j];
        int base = 0;
        for (; m - base > 16; base += 32)
            up_unit<G, PLANES, 4>(a, l, j, tile, base, S, part, sub, mine);
        if (m - base > 8)
            up_unit<G, PLANES, 2>(a, l, j, tile, base, S, part, sub, mine);
        else if (m - base > 0)
            up_unit<G, PLANES, 1>(a, l, j, tile, base, S, part, sub, mine);
    }
}

struct DownArgs {
    Routing r;
    const float *weights;
    int T, H, I;
    Weights w;
    Planes h;
    void *out;
    int out_f32;
    int max_slices;    // column slices per expert that the shared memory has room for
};

template <int G, int PLANES, int NT>
__device__ __forceinline__ void down_unit(const DownArgs &a, const Lists &l, int j, int64_t r0, int64_t r1, int base,
                                          int u0, int u1, float *y)
{
    using F = typename Format<G, (G > 0)>::Rows;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int first = l.begin[j] + base, end = l.begin[j + 1];
    const F f = Format<G, (G > 0)>::rows(a.w, r0, r1, a.I);
    float acc[NT][4];
    pass<F, PLANES, NT>(f, l, first, end, a.h.h, (int64_t)a.I * 2, 1, a.h.plane_bytes, u0, u1, a.I, acc);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int q = first + nt * 8 + 2 * t + c;
            if (q < end) {
                float *p = y + (int)l.slot[q] * kRow + g;
                p[0] = acc[nt][c];
                p[8] = acc[nt][2 + c];
            }
        }
}

__device__ __forceinline__ float ld_dsmem_f32(const float *p, uint32_t rank)
{
    return __int_as_float(ld_dsmem_s32(reinterpret_cast<const int32_t *>(p), rank));
}

template <int G, int PLANES>
__global__ void __launch_bounds__(kThreads, 2)
moe_down_kernel(DownArgs a)
{
    extern __shared__ __align__(16) uint8_t dynamic[];
    __shared__ Lists l;
    float *y = reinterpret_cast<float *>(dynamic);   // [slices][n][kRow], after the lists are built
    // topk_idx was complete before the up kernel began; h is complete after the wait
    build_lists(a.r, l, reinterpret_cast<int *>(dynamic), nullptr);
    grid_dependency_wait();
    allow_dependents();
    using F = typename Format<G, (G > 0)>::Rows;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2;
    const int C = (int)cluster_nctarank(), c = (int)cluster_ctarank();
    const int row0 = (int)(blockIdx.x / C) * 16;
    // column slices of an expert: enough units for every warp of the cluster
    const int W = C * kWarps, cols = (a.I + F::kUnit - 1) / F::kUnit;
    int S = 1;
    while (l.active * S < W && 2 * S <= a.max_slices && 2 * S <= cols)
        S *= 2;
    const int units = l.active * S;
    // unit u belongs to warp u % W of the cluster, block (u % W) % C
    for (int u = warp * C + c; u < units; u += W) {
        const int j = u / S, s = u % S;
        const int64_t base_row = (int64_t)l.expert[j] * a.H;
        // rows past H are read as the last one and not stored
        const int64_t r0 = base_row + min(row0 + g, a.H - 1), r1 = base_row + min(row0 + g + 8, a.H - 1);
        const int u0 = cols * s / S, u1 = cols * (s + 1) / S;
        float *ys = y + (size_t)s * a.r.n * kRow;
        const int m = l.begin[j + 1] - l.begin[j];
        int base = 0;
        for (; m - base > 16; base += 32)
            down_unit<G, PLANES, 4>(a, l, j, r0, r1, base, u0, u1, ys);
        if (m - base > 8)
            down_unit<G, PLANES, 2>(a, l, j, r0, r1, base, u0, u1, ys);
        else if (m - base > 0)
            down_unit<G, PLANES, 1>(a, l, j, r0, r1, base, u0, u1, ys);
    }
    if (C > 1)
        cluster_sync();
    else
        __syncthreads();
    // weighted sums over k; the blocks of the cluster share the tokens
    const int rows = min(16, a.H - row0), K = a.r.K;
    for (int v = threadIdx.x + c * kThreads; v < a.T * 16; v += kThreads * C) {
        const int tok = v >> 4, i = v & 15;
        if (i >= rows)
            continue;
        float sum = 0.0f;
        for (int k = 0; k < K; ++k) {
            const int slot = tok * K + k;
            const int j = l.use[slot];
            if (j < 0)
                continue;
            float p = 0.0f;
            for (int s = 0; s < S; ++s) {
                const float *at = y + ((size_t)s * a.r.n + slot) * kRow + i;
                const int owner = (j * S + s) % W % C;
                p = __fadd_rn(p, owner == c ? *at : ld_dsmem_f32(at, owner));
            }
            sum = __fmaf_rn(a.weights[slot], p, sum);
        }
        const int64_t o = (int64_t)tok * a.H + row0 + i;
        if (a.out_f32)
            static_cast<float *>(a.out)[o] = sum;
        else
            static_cast<__nv_bfloat16 *>(a.out)[o] = __float2bfloat16_rn(sum);
    }
    if (C > 1)
        cluster_sync();   // no block leaves while another reads its shared memory
}

// ------------------------------------------------------------ launch policy --
constexpr size_t kStaticSmem = sizeof(Lists) + 1024;
constexpr size_t kSmemPerBlock = 227 * 1024 / 2 - kStaticSmem;   // two blocks to an SM

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
int launch_dependent(Kernel kernel, unsigned grid, size_t smem, unsigned cluster, cudaStream_t stream, const Args &a)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
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
    const int used = std::min(up.r.n, up.r.E_local);   // experts in use, at most
    const size_t counts = align_up((size_t)up.r.E_local * sizeof(int), 16);
    {
        static PerDevice set;
        const size_t smem = std::max(counts, (size_t)kWarps * kMaxBlocks8 * 128 * sizeof(float));
        int rc = raise_smem(moe_up_kernel<G, PLANES>, smem, set);
        if (rc != EP_OK)
            return rc;
        // one resident wave, or fewer blocks when every unit already has a block's eight warps
        const int64_t units = (int64_t)used * (up.I / 8);
        rc = launch_dependent(moe_up_kernel<G, PLANES>, (unsigned)std::min<int64_t>(units, 2 * sms), smem, 1, stream, up);
        if (rc != EP_OK)
            return rc;
    }
    static PerDevice set;
    const size_t slice = (size_t)up.r.n * kRow * sizeof(float);
    // blocks of a cluster: the count that leaves the fullest last wave of two blocks to an SM
    const int tiles = (int)ceil_div(up.H, 16), wave = 2 * sms;
    int C = 1;
    int64_t best = INT64_MAX;
    for (int c = 1; c <= 8; c *= 2) {
        const int64_t cost = ceil_div((int64_t)tiles * c, wave) * (8 / c);
        if (cost < best) {
            best = cost;
            C = c;
        }
    }
    int slices = 1;
    while (slices < kWarps * C && (size_t)(2 * slices) * slice <= kSmemPerBlock)
        slices *= 2;
    down.max_slices = slices;
    const size_t smem = std::max(counts, slices * slice);
    const int rc = raise_smem(moe_down_kernel<G, PLANES>, smem, set);
    if (rc != EP_OK)
        return rc;
    return launch_dependent(moe_down_kernel<G, PLANES>, (unsigned)(tiles * C), smem, (unsigned)C, stream, down);
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
    if (T > kMaxSlots || T * K > kMaxSlots || H >= (1 << 20) || I >= (1 << 20))
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
