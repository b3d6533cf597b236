// Products of a streamed weight matrix with a few columns (internal).
//
// With a few tokens every weight is used a handful of times, so these products
// are bound by reading the weights from HBM, and what counts is that enough of
// them is in flight all the time.  A block owns an SM and a share of the weight
// rows; its 16 warps share that work in equal runs of K, each streaming its own
// 16 rows at a time through a ring of its own in shared memory:
//
//   - cp.async copies 16 bytes of a row to the slot of the very lane that will
//     use them, so a lane waits for its own copies only: no barrier stands
//     between the copy and its use, and the ring runs across items;
//   - lane (g, t) holds rows g and g+8 of an m16n8k16 matrix step and takes
//     whole 16-byte pieces of them, offering the same columns of x for the
//     instruction's k positions: a sum over k does not care about its order;
//   - the columns (tokens) are the instruction's N = 8 side, so one token costs
//     what eight do, which is nothing beside the weight stream.
//
// Accumulators: the matrix step's fp32 sums run over at most 128 columns of K
// (one group of 4-bit weights); these partial sums are then scaled and added
// with IEEE fp32 operations.
#pragma once

#include <cstdint>

#include "ep_device.cuh"

namespace ep {

constexpr int kSkinnyWarps = 16;
constexpr int kSkinnyThreads = 32 * kSkinnyWarps;
constexpr int kGroupUnits = 2;       // units (1 KB: 16 rows) of one ring stage
constexpr int kStages = 3;           // stages in flight per warp: 96 KB per SM, twice what 45 KB/us x 1 us needs
constexpr int kStageBytes = kGroupUnits * 1024;
constexpr int kRingBytes = kSkinnyWarps * kStages * kStageBytes;
constexpr int kMaxCols = 32;         // columns of one pass over the weights: 4 blocks of 8
constexpr int kSideBytes = 16 * kMaxCols * 4;   // one 16 x 32 block of partial sums

// D += A (16x16, row) * B (16x8, col), bf16 in, fp32 sums.
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                 "{%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// 16 bytes to shared memory, zeros where !ok (src is then not read).
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool ok)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}

__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

template <int N>
__device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint4 ld_shared16(uint32_t a)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}

// The columns of the product, bf16, for this lane: column g of each of NT
// blocks of 8.  PLANES copies of the columns (a value split into a sum of bf16
// terms) lie plane_bytes apart.  A null pointer is a column of zeros.
template <int NT, int PLANES>
struct Columns {
    const uint8_t *p[NT];
    int64_t plane_bytes;

    __device__ __forceinline__ uint4 load(int nt, int plane, int k, int K) const
    {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (p[nt] != nullptr && k < K)
            v = __ldg(reinterpret_cast<const uint4 *>(p[nt] + plane * plane_bytes + (int64_t)k * 2));
        return v;
    }
};

// Where a lane's two rows lie.  A row past the end of its block has a null data
// pointer: it is not read, and its sums are not used.
struct RowPtrs {
    const uint8_t *r0, *r1;     // data of rows g and g+8
    const uint16_t *s0, *s1;    // 4-bit: scales (bf16 bits)
    const uint8_t *z0, *z1;     // 4-bit: zero points, or null
};

struct Weights {
    const uint8_t *data;
    const uint16_t *scale;
    const uint8_t *zero;
};

// bf16 weights.  A unit is 32 columns: lane (g, t) holds columns 8t .. 8t+7 of
// rows g and g+8, two k16 steps.
struct FormatBf16 {
    static constexpr int kUnit = 32;
    static constexpr bool kPermuted = false;
    // what an item costs beside one n-block's columns: 1 KB of weights to 0.5 KB of x
    static constexpr int kItemCost = 4;
    struct Extra {};

    static __device__ __forceinline__ RowPtrs rows(const Weights &w, int64_t a, int64_t b, bool has_a, bool has_b, int K)
    {
        const int64_t bytes = (int64_t)K * 2;
        RowPtrs r = {};
        r.r0 = has_a ? w.data + a * bytes : nullptr;
        r.r1 = has_b ? w.data + b * bytes : nullptr;
        return r;
    }

    static __device__ __forceinline__ int column(int u, int t) { return u * kUnit + 8 * t; }
    static __device__ __forceinline__ int64_t offset(int k) { return (int64_t)k * 2; }
    static __device__ __forceinline__ Extra extra(const RowPtrs &, int, int, int) { return Extra{}; }

    template <int NT, int PLANES>
    static __device__ __forceinline__ void unit(const uint4 &a, const uint4 &b, const Extra &, int u, int K, int t,
                                                const Columns<NT, PLANES> &x, float (&acc)[NT][4])
    {
        const int k = column(u, t);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float part[4] = {};
#pragma unroll
            for (int p = 0; p < PLANES; ++p) {
                const uint4 v = x.load(nt, p, k, K);
                mma_bf16(part, a.x, b.x, a.y, b.y, v.x, v.y);
                mma_bf16(part, a.z, b.z, a.w, b.w, v.z, v.w);
            }
#pragma unroll
            for (int c = 0; c < 4; ++c)
                acc[nt][c] = __fadd_rn(acc[nt][c], part[c]);
        }
    }
};

// 4-bit weights with a scale (and zero point) per G columns.  A unit is 128
// columns: lane (g, t) loads the 32 codes of columns 32t .. 32t+31 of rows g
// and g+8.  Codes become bf16 integers exactly: 0x4300 | q is 128 + q, less
// 128 + zero.  Word bits 4j hold code j, so masking 0x000f000f takes codes
// (j, j+4) as a pair; x's columns are paired the same way (by the stored order
// where PERMUTED, else by byte permutes).  With G < 128 a lane's words belong
// to other groups than its neighbours', so the four lanes of a row trade words
// until each matrix step stays in one group.
template <int G, bool PERMUTED>
struct FormatW4 {
    static constexpr int kUnit = 128;
    static constexpr bool kPermuted = PERMUTED;
    static constexpr int kItemCost = 2;
    struct Extra {
        uint32_t q0, q1;    // scale in the high half, bf16(128 + zero) in the low half
    };

    static __device__ __forceinline__ RowPtrs rows(const Weights &w, int64_t a, int64_t b, bool has_a, bool has_b, int K)
    {
        const int64_t bytes = K / 2, groups = K / G;
        RowPtrs r = {};
        if (has_a) {
            r.r0 = w.data + a * bytes;
            r.s0 = w.scale + a * groups;
            r.z0 = w.zero != nullptr ? w.zero + a * groups : nullptr;
        }
        if (has_b) {
            r.r1 = w.data + b * bytes;
            r.s1 = w.scale + b * groups;
            r.z1 = w.zero != nullptr ? w.zero + b * groups : nullptr;
        }
        return r;
    }

    static __device__ __forceinline__ int column(int u, int t) { return u * kUnit + 32 * t; }
    static __device__ __forceinline__ int64_t offset(int k) { return k >> 1; }

    static __device__ __forceinline__ uint32_t group(const uint16_t *s, const uint8_t *z, int gi)
    {
        const uint32_t zero = z != nullptr ? (uint32_t)__ldg(z + gi) : 8u;
        return ((uint32_t)__ldg(s + gi) << 16) | 0x4300u | zero;
    }

    static __device__ __forceinline__ Extra extra(const RowPtrs &r, int u, int K, int t)
    {
        const int k = column(u, t);
        Extra e{0x4308u, 0x4308u};
        if (k < K) {
            if (r.s0 != nullptr)
                e.q0 = group(r.s0, r.z0, k / G);
            if (r.s1 != nullptr)
                e.q1 = group(r.s1, r.z1, k / G);
        }
        return e;
    }

    // (a, b) -> the low lane keeps a and gets its partner's a, the high lane keeps b and gets b
    static __device__ __forceinline__ void trade(uint32_t &a, uint32_t &b, int mask, bool high)
    {
        const uint32_t out = high ? a : b;
        const uint32_t in = __shfl_xor_sync(kFull, out, mask);
        a = high ? in : a;
        b = high ? b : in;
    }

    // after it, word i of lane t lies in columns word_column(i, t) of the unit
    static __device__ __forceinline__ void arrange(uint4 &w, int t)
    {
        if (G == 64) {
            trade(w.x, w.z, 2, t & 2);
            trade(w.y, w.w, 2, t & 2);
        } else if (G == 32) {
            trade(w.x, w.y, 1, t & 1);
            trade(w.z, w.w, 1, t & 1);
            trade(w.x, w.z, 2, t & 2);
            trade(w.y, w.w, 2, t & 2);
        }
    }

    static __device__ __forceinline__ int word_column(int i, int t)
    {
        if (G == 128)
            return 32 * t + 8 * i;
        if (G == 64)
            return 64 * (i >> 1) + 32 * (t & 1) + 16 * (t >> 1) + 8 * (i & 1);
        return 32 * i + 8 * t;
    }

    static __device__ __forceinline__ uint32_t codes(uint32_t w, uint32_t zz)
    {
        return sub_bf16x2((w & 0x000f000fu) | 0x43004300u, zz);
    }

    template <int NT, int PLANES>
    static __device__ __forceinline__ void unit(uint4 wa, uint4 wb, const Extra &e, int u, int K, int t,
                                                const Columns<NT, PLANES> &x, float (&acc)[NT][4])
    {
        constexpr int kWords = G / 32;   // words of a lane in one group
        arrange(wa, t);
        arrange(wb, t);
        const uint32_t va[4] = {wa.x, wa.y, wa.z, wa.w}, vb[4] = {wb.x, wb.y, wb.z, wb.w};
#pragma unroll
        for (int gi = 0; gi < 4 / kWords; ++gi) {
            uint32_t q0 = e.q0, q1 = e.q1;
            if (G < 128) {   // the lane of this row that loaded this group's scale
                const int from = (threadIdx.x & 28) | (gi * kWords);
                q0 = __shfl_sync(kFull, q0, from);
                q1 = __shfl_sync(kFull, q1, from);
            }
            const uint32_t zz0 = __byte_perm(q0, q0, 0x1010), zz1 = __byte_perm(q1, q1, 0x1010);
            float part[NT][4] = {};
#pragma unroll
            for (int j = 0; j < kWords; ++j) {
                const int w = gi * kWords + j;
                const int k = u * kUnit + word_column(w, t);
                const uint32_t a = va[w], b = vb[w];
                const uint32_t a0 = codes(a, zz0), a1 = codes(a >> 4, zz0), a2 = codes(a >> 8, zz0),
                               a3 = codes(a >> 12, zz0);
                const uint32_t c0 = codes(b, zz1), c1 = codes(b >> 4, zz1), c2 = codes(b >> 8, zz1),
                               c3 = codes(b >> 12, zz1);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int p = 0; p < PLANES; ++p) {
                        uint4 v = x.load(nt, p, k, K);
                        if (!PERMUTED)   // columns (0,4) (1,5) (2,6) (3,7)
                            v = make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632),
                                           __byte_perm(v.y, v.w, 0x5410), __byte_perm(v.y, v.w, 0x7632));
                        mma_bf16(part[nt], a0, c0, a1, c1, v.x, v.y);
                        mma_bf16(part[nt], a2, c2, a3, c3, v.z, v.w);
                    }
            }
            const float f0 = __uint_as_float(q0 & 0xffff0000u), f1 = __uint_as_float(q1 & 0xffff0000u);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                acc[nt][0] = __fmaf_rn(part[nt][0], f0, acc[nt][0]);
                acc[nt][1] = __fmaf_rn(part[nt][1], f0, acc[nt][1]);
                acc[nt][2] = __fmaf_rn(part[nt][2], f1, acc[nt][2]);
                acc[nt][3] = __fmaf_rn(part[nt][3], f1, acc[nt][3]);
            }
        }
    }
};

// The weight format of a kernel: G = 0 for bf16, else the group of 4-bit codes.
template <int G, bool PERMUTED>
struct FormatOf {
    using F = FormatW4<G, PERMUTED>;
};
template <bool PERMUTED>
struct FormatOf<0, PERMUTED> {
    using F = FormatBf16;
};

// Where column j of a block of 8 stands in memory, for a producer of columns.
template <bool PERMUTED>
__device__ __forceinline__ int column_place(int j)
{
    return PERMUTED ? ((j & 3) << 1) | (j >> 2) : j;
}

// A warp's sums of one item as they are kept: [block of 8 columns][lane] float4.
__device__ __forceinline__ int side_index(int row, int col)   // in floats
{
    const int lane = ((row & 7) << 2) | ((col & 7) >> 1);
    return (((col >> 3) * 32 + lane) << 2) | ((row >> 3) << 1) | (col & 1);
}

// One warp's run of a block's items.  Items are numbered 0 .. items-1; each is
// 16 rows times all of K (`per` units).  The run is units [begin, end) of the
// items laid end to end: it may start or stop inside an item.
//
// Items is the kernel's view of its work: rows(item) gives this lane's RowPtrs,
// blocks(item) the number of 8-column blocks (1 .. 4), columns<NT>(item, x)
// sets the column pointers, and done<NT>(item, first, last, acc) takes the sums
// of a piece; first / last say whether the piece holds the item's first and
// last unit.
template <class F, int PLANES, class Items>
class Stream {
public:
    __device__ __forceinline__ Stream(Items &items, int K, int n_items, uint32_t ring)
        : items_(items), K_(K), per_((K + F::kUnit - 1) / F::kUnit)
    {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        t_ = lane & 3;
        const int64_t total = (int64_t)n_items * per_;
        begin_ = (int)(total * warp / kSkinnyWarps);
        end_ = (int)(total * (warp + 1) / kSkinnyWarps);
        slot_ = ring + warp * (kStages * kStageBytes) + lane * 16;
        ahead_ = begin_;
        item_ahead_ = begin_ / per_;
        u_ahead_ = begin_ - item_ahead_ * per_;
        stage_ahead_ = stage_ = 0;
        fresh_ = true;
    }

    // the first copies of the run; they read weights only
    __device__ __forceinline__ void start()
    {
#pragma unroll
        for (int s = 0; s < kStages; ++s)
            issue();
    }

    __device__ __forceinline__ void run()
    {
        int at = begin_;
        while (at < end_) {
            const int item = at / per_, u0 = at - item * per_;
            const int u1 = min(per_, u0 + end_ - at);
            const int nb = items_.blocks(item);
            if (nb <= 1)
                piece<1>(item, u0, u1);
            else if (nb == 2)
                piece<2>(item, u0, u1);
            else
                piece<4>(item, u0, u1);
            at += u1 - u0;
        }
    }

private:
    __device__ __forceinline__ void issue()
    {
        if (ahead_ < end_) {
            if (fresh_) {
                src_ = items_.rows(item_ahead_);
                fresh_ = false;
            }
            const int left = min(per_ - u_ahead_, end_ - ahead_);
            const uint32_t dst = slot_ + stage_ahead_ * kStageBytes;
#pragma unroll
            for (int i = 0; i < kGroupUnits; ++i)
                if (i < left) {
                    const int k = F::column(u_ahead_ + i, t_);
                    const bool ok = k < K_;
                    const int64_t off = ok ? F::offset(k) : 0;
                    if (src_.r0 != nullptr)
                        cp_async16(dst + i * 1024, src_.r0 + off, ok);
                    if (src_.r1 != nullptr)
                        cp_async16(dst + i * 1024 + 512, src_.r1 + off, ok);
                }
            const int n = min(left, kGroupUnits);
            ahead_ += n;
            u_ahead_ += n;
            if (u_ahead_ == per_) {
                u_ahead_ = 0;
                ++item_ahead_;
                fresh_ = true;
            }
        }
        cp_async_commit();
        stage_ahead_ = stage_ahead_ == kStages - 1 ? 0 : stage_ahead_ + 1;
    }

    template <int NT>
    __device__ __forceinline__ void piece(int item, int u0, int u1)
    {
        Columns<NT, PLANES> x;
        items_.template columns<NT>(item, x);
        const RowPtrs rows = items_.rows(item);
        float acc[NT][4] = {};
        typename F::Extra e[kGroupUnits];
#pragma unroll
        for (int i = 0; i < kGroupUnits; ++i)
            e[i] = F::extra(rows, u0 + i, K_, t_);
        for (int u = u0; u < u1; u += kGroupUnits) {
            cp_async_wait<kStages - 1>();
            const uint32_t src = slot_ + stage_ * kStageBytes;
            uint4 a[kGroupUnits], b[kGroupUnits];
            typename F::Extra f[kGroupUnits];
#pragma unroll
            for (int i = 0; i < kGroupUnits; ++i) {
                a[i] = ld_shared16(src + i * 1024);
                b[i] = ld_shared16(src + i * 1024 + 512);
                f[i] = e[i];
                e[i] = F::extra(rows, u + kGroupUnits + i, K_, t_);
            }
            issue();
#pragma unroll
            for (int i = 0; i < kGroupUnits; ++i)
                if (u + i < u1)
                    F::template unit<NT, PLANES>(a[i], b[i], f[i], u + i, K_, t_, x, acc);
            stage_ = stage_ == kStages - 1 ? 0 : stage_ + 1;
        }
        items_.template done<NT>(item, u0 == 0, u1 == per_, acc);
    }

    Items &items_;
    RowPtrs src_;
    int K_, per_, t_;
    int begin_, end_, ahead_, item_ahead_, u_ahead_;
    int stage_ahead_, stage_;
    uint32_t slot_;
    bool fresh_;
};

// The first unit of warp w's run (see Stream), for whoever adds up the pieces.
__device__ __forceinline__ int run_begin(int n_items, int per, int w)
{
    return (int)((int64_t)n_items * per * w / kSkinnyWarps);
}

}  // namespace ep
