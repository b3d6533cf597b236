// Products of a streamed weight matrix with a few columns (internal): one warp
// sums 16 weight rows times up to 8*NT columns over a range of K.
//
// With a few tokens every weight is used a handful of times, so these products
// are bound by reading the weights from HBM.  Each lane loads its weights
// straight from the row-major matrix into the registers of an m16n8k16 matrix
// instruction, 16 bytes per row and load; nothing is staged in shared memory,
// so no barrier stands between a load and its use.  The sum over k does not
// care about the order of k: lane (g, t) takes whole 16-byte pieces of rows g
// and g+8 and offers the same columns of x, whatever k the instruction's
// layout gives those positions.  The columns (tokens) are the instruction's
// N = 8 side, so one token costs what eight do, which is still nothing beside
// the weight stream.
//
// Accumulators: the matrix instruction's fp32 sums run over at most 128 columns
// (one group of 4-bit weights); these partial sums are then scaled and added
// with IEEE fp32 operations.
#pragma once

#include <cstdint>

#include "ep_device.cuh"

namespace ep {

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

__device__ __forceinline__ uint4 ld_cached(const void *p)
{
    return __ldg(reinterpret_cast<const uint4 *>(p));
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
            v = ld_cached(p[nt] + plane * plane_bytes + (int64_t)k * 2);
        return v;
    }
};

// bf16 weights.  A unit of work is 32 columns: lane (g, t) holds columns 8t ..
// 8t+7 of rows g and g+8, which are two k16 steps.
struct RowsBf16 {
    static constexpr int kUnit = 32;
    static constexpr int kBatch = 4;    // units loaded together: 128 columns, 4 KB per warp
    static constexpr bool kPermuted = false;
    const uint8_t *r0, *r1;             // rows g and g+8 of this lane

    struct Regs {
        uint4 a0[kBatch], a1[kBatch];
    };

    __device__ __forceinline__ void load(Regs &r, int u0, int u1, int K, int t) const
    {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int k = (u0 + i) * kUnit + 8 * t;
            if (u0 + i < u1 && k < K) {
                r.a0[i] = ld_stream(reinterpret_cast<const uint4 *>(r0 + (int64_t)k * 2));
                r.a1[i] = ld_stream(reinterpret_cast<const uint4 *>(r1 + (int64_t)k * 2));
            } else {
                r.a0[i] = r.a1[i] = make_uint4(0, 0, 0, 0);
            }
        }
    }

    template <int NT, int PLANES>
    __device__ __forceinline__ void compute(const Regs &r, int u0, int u1, int K, int t,
                                            const Columns<NT, PLANES> &x, float (&acc)[NT][4]) const
    {
        float part[NT][4] = {};
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if (u0 + i >= u1)
                break;
            const int k = (u0 + i) * kUnit + 8 * t;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int p = 0; p < PLANES; ++p) {
                    const uint4 b = x.load(nt, p, k, K);
                    mma_bf16(part[nt], r.a0[i].x, r.a1[i].x, r.a0[i].y, r.a1[i].y, b.x, b.y);
                    mma_bf16(part[nt], r.a0[i].z, r.a1[i].z, r.a0[i].w, r.a1[i].w, b.z, b.w);
                }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c)
                acc[nt][c] = __fadd_rn(acc[nt][c], part[nt][c]);
    }
};

// 4-bit weights with a scale (and zero point) per G columns.  A unit is 128
// columns: lane (g, t) loads the 32 codes of columns 32t .. 32t+31 of rows g
// and g+8.  Codes become bf16 integers exactly: 0x4300 | q is 128 + q, less
// 128 + zero.  Word bits 4j hold code j, so masking 0x000f000f takes codes
// (j, j+4) as a pair; x's columns are paired the same way (by the stored order
// where PERMUTED, else by byte permutes).  With G < 128 a lane's words belong
// to different groups than its neighbours', so the four lanes of a row trade
// words until each matrix step stays in one group.
template <int G, bool PERMUTED>
struct RowsW4 {
    static constexpr int kUnit = 128;
    static constexpr int kBatch = 2;    // 256 columns, 2 KB per warp
    static constexpr bool kPermuted = PERMUTED;
    const uint8_t *r0, *r1;
    const uint16_t *s0, *s1;            // scales (bf16 bits) of rows g and g+8
    const uint8_t *z0, *z1;             // zero points, or null

    struct Regs {
        uint4 a0[kBatch], a1[kBatch];
        uint32_t q0[kBatch], q1[kBatch];   // scale in the high half, bf16(128 + zero) in the low half
    };

    __device__ __forceinline__ uint32_t group(const uint16_t *s, const uint8_t *z, int gi) const
    {
        const uint32_t zero = z != nullptr ? (uint32_t)__ldg(z + gi) : 8u;
        return ((uint32_t)__ldg(s + gi) << 16) | 0x4300u | zero;
    }

    __device__ __forceinline__ void load(Regs &r, int u0, int u1, int K, int t) const
    {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int k = (u0 + i) * kUnit + 32 * t;
            r.a0[i] = r.a1[i] = make_uint4(0, 0, 0, 0);
            r.q0[i] = r.q1[i] = 0x4308u;
            if (u0 + i < u1 && k < K) {
                r.a0[i] = ld_stream(reinterpret_cast<const uint4 *>(r0 + (k >> 1)));
                r.a1[i] = ld_stream(reinterpret_cast<const uint4 *>(r1 + (k >> 1)));
                r.q0[i] = group(s0, z0, k / G);
                r.q1[i] = group(s1, z1, k / G);
            }
        }
    }

    // the words a lane sends to lane ^ mask are replaced by those it gets:
    // (a, b) -> low lane keeps a and gets the partner's a; high lane keeps b
    static __device__ __forceinline__ void trade(uint32_t &a, uint32_t &b, int mask, bool high)
    {
        const uint32_t out = high ? a : b;
        const uint32_t in = __shfl_xor_sync(kFull, out, mask);
        a = high ? in : a;
        b = high ? b : in;
    }

    // after it, word i of lane t lies in columns column(i, t) of the unit
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

    static __device__ __forceinline__ int column(int i, int t)
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
    __device__ __forceinline__ void compute(const Regs &r, int u0, int u1, int K, int t,
                                            const Columns<NT, PLANES> &x, float (&acc)[NT][4]) const
    {
        constexpr int kWords = G / 32;   // words of a lane in one group
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if (u0 + i >= u1)
                break;
            const int k0 = (u0 + i) * kUnit;
            uint4 wa = r.a0[i], wb = r.a1[i];
            arrange(wa, t);
            arrange(wb, t);
            const uint32_t va[4] = {wa.x, wa.y, wa.z, wa.w}, vb[4] = {wb.x, wb.y, wb.z, wb.w};
#pragma unroll
            for (int gi = 0; gi < 4 / kWords; ++gi) {
                uint32_t q0 = r.q0[i], q1 = r.q1[i];
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
                    const int k = k0 + column(w, t);
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
    }
};

// Where column j of a block of 8 stands in memory, for a producer of columns.
template <bool PERMUTED>
__device__ __forceinline__ int column_place(int j)
{
    return PERMUTED ? ((j & 3) << 1) | (j >> 2) : j;
}

// acc += the 16 rows of f times the columns x, over units [u0, u1) of K.
// acc[nt]: rows g, g, g+8, g+8; columns 8*nt + 2t, +1, +0, +1.
template <class F, int NT, int PLANES>
__device__ __forceinline__ void skinny(const F &f, int u0, int u1, int K, int t, const Columns<NT, PLANES> &x,
                                       float (&acc)[NT][4])
{
    typename F::Regs a, b;
    f.load(a, u0, u1, K, t);
    // the next batch is in flight while one is used
    for (int u = u0; u < u1; u += 2 * F::kBatch) {
        f.load(b, u + F::kBatch, u1, K, t);
        f.compute(a, u, u1, K, t, x, acc);
        f.load(a, u + 2 * F::kBatch, u1, K, t);
        f.compute(b, u + F::kBatch, u1, K, t, x, acc);
    }
}

}  // namespace ep
