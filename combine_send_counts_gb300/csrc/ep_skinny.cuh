// Products of a streamed weight matrix with a few columns (internal).
//
// With a few tokens every weight is used a handful of times, so these products
// are bound by reading the weights from HBM, and what counts is that enough of
// them is in flight all the time.  A block owns an SM and a share of the weight
// rows; its warps share that work in equal runs of K, each streaming up to 64
// rows at a time through a ring of its own in shared memory:
//
//   - cp.async brings 16 rows times 256 bytes (4-bit: 128) to a stage of the
//     ring, whole row pieces by neighbouring lanes.  No block barrier stands
//     between a copy and its use, and the ring runs on across items.  (Copied
//     in pieces of 64, 128, 256 and 512 bytes, a plain stream of rows ran at
//     6.1, 6.4, 6.9 and 7.1 TB/s.)
//   - lane (g, t) holds rows g and g+8 of an m16n8k16 matrix step and takes
//     whole 16-byte pieces of them, offering the same columns of x for the
//     instruction's k positions: a sum over k does not care about its order;
//   - the columns (tokens) are the instruction's N = 8 side, so one token costs
//     what eight do, which is nothing beside the weight stream;
//   - x comes through L1 and L2 into registers, one unit of K ahead, and serves
//     all of the warp's row blocks.  (With 16 rows a warp and x loaded where it
//     is used, eight tokens ran at 3.5 TB/s, waiting for x.)
//
// Accumulators: the matrix step's fp32 sums run over at most 128 columns of K
// (one group of 4-bit weights); these partial sums are then scaled and added
// with IEEE fp32 operations.
//
// What bounds them, by the counters of a profile: bf16 weights, HBM (128 tokens
// of 128 experts 4096x1536 read 4.8 GB in 814 us, 5.9 TB/s, 0.87 of what a copy
// reaches); 4-bit weights, the instructions that make bf16 of the codes (50021
// rows of 7168: 4.4 TB/s, with the ALU pipe at 59% and the warps' waits short).
// Kernels that end before 20 us are latency: the first weights, the first x,
// the join and the launch take 3 us or so whatever the size.
#pragma once

#include <cstdint>

#include "ep_device.cuh"

namespace ep {

constexpr int kMaxCols = 16;         // columns of one pass over the weights: 2 blocks of 8

// The shared memory of a block whose warps take RB blocks of 16 rows at a time:
// 64 KB of weights are in flight per SM (a unit of each warp at least), and 45
// KB/us times about 1 us are needed; what more there is serves x better as L1
// (with 128 KB one token of 4-bit experts takes 61.2 us instead of 59.3, 128
// tokens of bf16 experts 830 instead of 814).
template <class F, int RB>
struct Room {
    static constexpr int kStage = 16 * F::kRowPiece;                         // one row block, one unit of K
    static constexpr int kFit = 64 * 1024 / F::kWarps / (RB * kStage);
    static constexpr int kUnits = kFit > 0 ? kFit : 1;                       // units in a warp's ring
    static constexpr int kWarpRing = kUnits * RB * kStage;
    static constexpr int kRing = F::kWarps * kWarpRing;
    static constexpr int kSide = RB * 16 * kMaxCols * 4;                     // one warp's kept sums
    static constexpr int kFixed = kRing + F::kWarps * kSide;
    static_assert(kUnits >= 1 && kSide <= kWarpRing, "the ring holds a unit, and kept sums after the run");
};

// n / d for 0 <= n < 2^30, 0 < d and a quotient below 2^22: by the approximate
// reciprocal, put right by the remainder (the estimate is off by two at most).
// The general division and the exact reciprocal cost the kernels' prologues a
// microsecond.
__device__ __forceinline__ int quick_div(int n, int d)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(__int2float_rn(d)));
    int q = __float2int_rz(__fmul_rn(__int2float_rn(n), r));
    int left = n - q * d;
    q += left >= d ? 1 : left < 0 ? -1 : 0;
    left = n - q * d;
    return q + (left >= d ? 1 : left < 0 ? -1 : 0);
}

// D += A (16x16, row) * B (16x8, col), bf16 in, fp32 sums.
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
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
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(a)
                 : "memory");
    return v;
}

__device__ __forceinline__ uint2 ld_shared8(uint32_t a)
{
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
    return v;
}

__device__ __forceinline__ uint32_t ld_shared4(uint32_t a)
{
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}

// The columns of the product, bf16, for this lane: column g of each of NT
// blocks of 8.  PLANES copies of the columns (a value split into a sum of bf16
// terms) lie plane_bytes apart.
template <int NT, int PLANES>
struct Columns {
    const uint8_t *p[NT];
    int64_t plane_bytes;
    int end[NT];          // K, or 0 for a column of zeros

    __device__ __forceinline__ void set(int nt, const uint8_t *column, int K)
    {
        p[nt] = column;
        end[nt] = column != nullptr ? K : 0;
    }

    // columns k + offset .. +7; the offset is a constant
    __device__ __forceinline__ uint4 load(int nt, int plane, int k, int offset) const
    {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (k + offset < end[nt])
            v = ld_global(reinterpret_cast<const uint4 *>(p[nt] + plane * plane_bytes + (uint32_t)k * 2 + offset * 2));
        return v;
    }
};

// An item's rows: block r takes rows a + r*step .. +7 (the first n of a's rows
// exist) and b + r*step .. +7 (the first m of b's), as rows 0-7 and 8-15 of the
// matrix step.  Rows that do not exist are not read, and their sums not used.
struct RowRange {
    int64_t a, b;
    int n, m;
};

struct Weights {
    const uint8_t *data;
    const uint16_t *scale;
    const uint8_t *zero;
    // 0x43004300, the bf16 pair 128, 128.  As an argument it stays in a register and a code pair takes one
    // and-or; as a constant it took a second instruction.  (With the scales shared by a row's lanes: 522 -> 383
    // instructions of a warp per stage, one token of 4-bit experts 95 -> 68 us.)
    uint32_t magic;
};
constexpr uint32_t kMagic = 0x43004300u;

// bf16 weights.  A unit is 128 columns; word j of lane (g, t) are columns
// 32j + 8t .. +7 of its rows, two k16 steps.
struct FormatBf16 {
    static constexpr int kWarps = 8;
    static constexpr int kMaxBlocks = 4;     // row blocks that a warp takes at a time
    static constexpr int kUnit = 128;
    static constexpr int kRowPiece = 256;    // bytes of a row in a unit
    static constexpr int kWordsX = 4;        // 8-column words of a unit that a lane holds
    static constexpr bool kPermuted = false;
    static constexpr int kPieces = 4;        // 16-byte pieces of a lane's row in a stage

    static __device__ __forceinline__ int64_t row_bytes(int K) { return (int64_t)K * 2; }

    // 16-byte piece p of a row stands at p ^ fold(row) in its stage, so that the lanes of a load meet all banks
    static __device__ __forceinline__ int fold(int row) { return (row & 1) << 2; }
    static __device__ __forceinline__ constexpr uint32_t refold(int) { return 0; }
    // a lane's 16 of 64 bytes come by kReads loads, the i-th at place(g, t) ^ i * kReadStep
    static constexpr int kReads = 1, kReadStep = 0;
    static __device__ __forceinline__ int place(int, int t) { return 16 * t; }
    static __device__ __forceinline__ uint4 read(const uint32_t (&at)[kReads], int offset)
    {
        return ld_shared16(at[0] + offset);
    }

    // word w of lane t are columns lane_column(t) + word_column(w) .. +7 of the unit
    static __device__ __forceinline__ int lane_column(int t) { return 8 * t; }
    static __device__ __forceinline__ constexpr int word_column(int w) { return 32 * w; }
    static __device__ __forceinline__ uint4 pair(uint4 v) { return v; }

    template <int RB, int STEP>
    struct Scales {
        __device__ __forceinline__ void begin(const Weights &, const RowRange &, int, int, int) {}
        __device__ __forceinline__ void load(int) {}
    };

    // acc += block r of the unit; next(w) is called once word w of x is used up
    template <int RB, int STEP, int NT, int PLANES, class Next>
    static __device__ __forceinline__ void block(const uint4 (&a)[kPieces], const uint4 (&b)[kPieces], int,
                                                 const Scales<RB, STEP> &, uint4 (&x)[kWordsX][NT][PLANES], int,
                                                 float (&acc)[NT][4], Next next)
    {
        // Two chains, so that a matrix step need not wait for the one before: of one plane, half of the columns each; of
        // several, the first plane and the others.  A step may drop bits below its accumulator's last, and so drops
        // few of the small planes' (fp32 results of 16 tokens of experts 4096x1536: 3.0e-7 from 64 bits, with half of
        // the columns each 4.7e-7, in the same time).
        float part[2][NT][4] = {};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int p = 0; p < PLANES; ++p) {
                    const uint4 v = x[j][nt][p];
                    mma_bf16(part[p > 0][nt], a[j].x, b[j].x, a[j].y, b[j].y, v.x, v.y);
                    mma_bf16(part[PLANES == 1 || p > 0][nt], a[j].z, b[j].z, a[j].w, b[j].w, v.z, v.w);
                }
            next(j);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                acc[nt][i] = __fadd_rn(acc[nt][i], __fadd_rn(part[0][nt][i], part[1][nt][i]));
    }
};

// 4-bit weights with a scale (and zero point) per G columns.  A unit is 256
// columns, two halves; lane (g, t) reads 32 codes of each for each of its rows.
// Codes become bf16 integers exactly: 0x4300 | q is 128 + q, less 128 + zero.
// Word bits 4j hold code j, so masking 0x000f000f takes codes (j, j+4) as a
// pair; x's columns are paired the same way (by the stored order where
// PERMUTED, else by byte permutes).
template <int G, bool PERMUTED>
struct FormatW4 {
    static constexpr int kWarps = 8;
    static constexpr int kMaxBlocks = 4;
    static constexpr int kUnit = 256;
    static constexpr int kRowPiece = 128;
    static constexpr int kWordsX = 8;
    static constexpr bool kPermuted = PERMUTED;
    static constexpr int kPieces = 2;
    static constexpr int kWords = G / 32;   // words of a lane in one group

    static __device__ __forceinline__ int64_t row_bytes(int K) { return K / 2; }

    // A half's 64 bytes of a row are four 16-byte pieces of 32 codes.  A matrix step takes codes of one group: with
    // G = 128 a lane takes a whole piece, with 64 half of each of two pieces, with 32 a word of each of the four.
    // Piece p of a row stands at p ^ fold(row) in its stage, so that the lanes of each of these loads meet all banks.
    static __device__ __forceinline__ int fold(int row) { return (row & 1) << 2 | (G == 128 ? 0 : row >> 1 & 3); }
    // what fold(4i + row) changes in an address against fold(row), for rows below 4
    static __device__ __forceinline__ constexpr uint32_t refold(int i) { return G == 128 ? 0 : 32 * i; }
    static constexpr int kReads = 128 / G, kReadStep = G == 64 ? 32 : 16;
    static __device__ __forceinline__ int place(int g, int t)
    {
        const int low = (fold(g) & 3) << 4;
        return G == 128 ? 16 * t : G == 64 ? (16 * (t & 1) ^ low) + 8 * (t >> 1) : low + 4 * t;
    }
    static __device__ __forceinline__ uint4 read(const uint32_t (&at)[kReads], int offset)
    {
        if constexpr (G == 128) {
            return ld_shared16(at[0] + offset);
        } else if constexpr (G == 64) {
            const uint2 a = ld_shared8(at[0] + offset), b = ld_shared8(at[1] + offset);
            return make_uint4(a.x, a.y, b.x, b.y);
        } else {
            return make_uint4(ld_shared4(at[0] + offset), ld_shared4(at[1] + offset), ld_shared4(at[2] + offset),
                              ld_shared4(at[3] + offset));
        }
    }

    // word w of lane t are columns lane_column(t) + word_column(w) .. +7 of the unit
    static __device__ __forceinline__ int lane_column(int t)
    {
        return G == 128 ? 32 * t : G == 64 ? 32 * (t & 1) + 16 * (t >> 1) : 8 * t;
    }
    static __device__ __forceinline__ constexpr int word_column(int w)
    {
        return 128 * (w >> 2) + (G == 128 ? 8 * (w & 3) : G == 64 ? 64 * ((w & 3) >> 1) + 8 * (w & 1) : 32 * (w & 3));
    }

    static __device__ __forceinline__ uint4 pair(uint4 v)
    {
        if (PERMUTED)
            return v;
        // columns (0,4) (1,5) (2,6) (3,7)
        return make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632),
                          __byte_perm(v.y, v.w, 0x5410), __byte_perm(v.y, v.w, 0x7632));
    }

    static __device__ __forceinline__ uint32_t codes(uint32_t w, uint32_t magic, uint32_t zz)
    {
        return sub_bf16x2((w & 0x000f000fu) | magic, zz);
    }

    // The scales and zero points of a unit: lane (g, t) keeps those of rows g and g+8 of row block t, the scale in
    // the high half and bf16(128 + zero) in the low half of a word per group, and hands them out when that
    // block's turn comes.
    template <int RB, int STEP>
    struct Scales {
        static_assert(RB <= 4, "a lane of a row for each block");
        static constexpr int kGroups = kUnit / G;
        uint32_t q[2][kGroups];
        uint32_t magic;
        const uint16_t *s0, *s1;    // the lane's rows
        const uint8_t *z0, *z1;
        int n0, n1, y0, y1;         // their groups and zero points to load: all of K's, or none
        bool wide;

        __device__ __forceinline__ void begin(const Weights &w, const RowRange &rows, int K, int g, int t)
        {
            const int groups = K / G, i = t * STEP + g;
            const int64_t a = (rows.a + i) * groups, b = (rows.b + i) * groups;
            magic = w.magic;
            s0 = w.scale + a;
            s1 = w.scale + b;
            z0 = w.zero + a;
            z1 = w.zero + b;
            n0 = t < RB && i < rows.n ? groups : 0;
            n1 = t < RB && i < rows.m ? groups : 0;
            y0 = w.zero != nullptr ? n0 : 0;
            y1 = w.zero != nullptr ? n1 : 0;
            wide = groups % kGroups == 0 && reinterpret_cast<uintptr_t>(w.scale) % (2 * kGroups) == 0 &&
                   reinterpret_cast<uintptr_t>(w.zero) % kGroups == 0;
        }

        // unit u's: in one load per row where every row's start allows it (eight loads of a row took 37.7 us for
        // 24x7168x4096 with groups of 32, one 27.7; for the two of a group of 128 it is not worth its selects: 43.4
        // instead of 42.1 us for 50021x7168, and loads a unit ahead were no better)
        __device__ __forceinline__ void load(int u)
        {
            const int first = u * kGroups;
            if (G < 128 && wide) {
                uint32_t v[2][kGroups / 2], y[2][(kGroups + 3) / 4];
                fetch(v[0], s0 + first, first < n0);
                fetch(v[1], s1 + first, first < n1);
                fetch_zero(y[0], z0 + first, first < y0);
                fetch_zero(y[1], z1 + first, first < y1);
#pragma unroll
                for (int i = 0; i < kGroups; ++i)
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        q[k][i] = (i & 1 ? v[k][i / 2] & 0xffff0000u : v[k][i / 2] << 16) | 0x4300u |
                                  (y[k][i / 4] >> (8 * (i % 4)) & 0xff);
                return;
            }
#pragma unroll
            for (int i = 0; i < kGroups; ++i) {
                const int at = first + i;
                const uint32_t v0 = at < n0 ? ld_global(s0 + at) : 0, v1 = at < n1 ? ld_global(s1 + at) : 0;
                const uint32_t w0 = at < y0 ? ld_global(z0 + at) : 8, w1 = at < y1 ? ld_global(z1 + at) : 8;
                q[0][i] = v0 << 16 | 0x4300u | w0;
                q[1][i] = v1 << 16 | 0x4300u | w1;
            }
        }

        static __device__ __forceinline__ void fetch(uint32_t (&v)[kGroups / 2], const uint16_t *p, bool in)
        {
#pragma unroll
            for (int i = 0; i < kGroups / 2; ++i)
                v[i] = 0;
            if (!in)
                return;
            if constexpr (kGroups == 2) {
                v[0] = ld_global(reinterpret_cast<const uint32_t *>(p));
            } else if constexpr (kGroups == 4) {
                const uint2 t = ld_global(reinterpret_cast<const uint2 *>(p));
                v[0] = t.x, v[1] = t.y;
            } else {
                const uint4 t = ld_global(reinterpret_cast<const uint4 *>(p));
                v[0] = t.x, v[1] = t.y, v[2] = t.z, v[3] = t.w;
            }
        }

        static __device__ __forceinline__ void fetch_zero(uint32_t (&y)[(kGroups + 3) / 4], const uint8_t *p, bool in)
        {
#pragma unroll
            for (int i = 0; i < (kGroups + 3) / 4; ++i)
                y[i] = 0x08080808u;
            if (!in)
                return;
            if constexpr (kGroups == 2) {
                y[0] = ld_global(reinterpret_cast<const uint16_t *>(p));
            } else if constexpr (kGroups == 4) {
                y[0] = ld_global(reinterpret_cast<const uint32_t *>(p));
            } else {
                const uint2 t = ld_global(reinterpret_cast<const uint2 *>(p));
                y[0] = t.x, y[1] = t.y;
            }
        }

        // of group i of row block r, for the lane's row g + 8*half
        __device__ __forceinline__ uint32_t get(int r, int half, int i) const
        {
            return __shfl_sync(kFull, q[half][i], (threadIdx.x & 28) | r);
        }
    };

    // Chains of matrix steps whose sums are added at a group's end, so that a step need not wait for the one before.
    // A group of 32 is two steps, too short for that: with one chain 24x7168x4096 took 24.2 us, with two 27.8; groups
    // of 64 lost 1% with one.
    static constexpr int kChains = G == 32 ? 1 : 2;
    template <int NT>
    static __device__ __forceinline__ float sum_of(const float (&part)[kChains][NT][4], int nt, int i)
    {
        return kChains == 1 ? part[0][nt][i] : __fadd_rn(part[0][nt][i], part[kChains - 1][nt][i]);
    }

    template <int RB, int STEP, int NT, int PLANES, class Next>
    static __device__ __forceinline__ void block(const uint4 (&va)[kPieces], const uint4 (&vb)[kPieces], int r,
                                                 const Scales<RB, STEP> &s, uint4 (&x)[kWordsX][NT][PLANES], int t,
                                                 float (&acc)[NT][4], Next next)
    {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t a[4] = {va[h].x, va[h].y, va[h].z, va[h].w}, b[4] = {vb[h].x, vb[h].y, vb[h].z, vb[h].w};
#pragma unroll
            for (int gi = 0; gi < 4 / kWords; ++gi) {
                const uint32_t q0 = s.get(r, 0, h * (128 / G) + gi), q1 = s.get(r, 1, h * (128 / G) + gi);
                const uint32_t zz0 = __byte_perm(q0, q0, 0x1010), zz1 = __byte_perm(q1, q1, 0x1010);
                float part[kChains][NT][4] = {};
#pragma unroll
                for (int j = 0; j < kWords; ++j) {
                    const int i = gi * kWords + j, w = 4 * h + i;
                    const uint32_t a0 = codes(a[i], s.magic, zz0), a1 = codes(a[i] >> 4, s.magic, zz0),
                                   a2 = codes(a[i] >> 8, s.magic, zz0), a3 = codes(a[i] >> 12, s.magic, zz0);
                    const uint32_t b0 = codes(b[i], s.magic, zz1), b1 = codes(b[i] >> 4, s.magic, zz1),
                                   b2 = codes(b[i] >> 8, s.magic, zz1), b3 = codes(b[i] >> 12, s.magic, zz1);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int p = 0; p < PLANES; ++p) {
                            const uint4 v = x[w][nt][p];
                            mma_bf16(part[0][nt], a0, b0, a1, b1, v.x, v.y);
                            mma_bf16(part[kChains - 1][nt], a2, b2, a3, b3, v.z, v.w);
                        }
                    next(w);
                }
                const float f0 = __uint_as_float(q0 & 0xffff0000u), f1 = __uint_as_float(q1 & 0xffff0000u);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    acc[nt][0] = __fmaf_rn(sum_of(part, nt, 0), f0, acc[nt][0]);
                    acc[nt][1] = __fmaf_rn(sum_of(part, nt, 1), f0, acc[nt][1]);
                    acc[nt][2] = __fmaf_rn(sum_of(part, nt, 2), f1, acc[nt][2]);
                    acc[nt][3] = __fmaf_rn(sum_of(part, nt, 3), f1, acc[nt][3]);
                }
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

// A warp's sums of one item as they are kept: [row block][column block][lane] float4.
__device__ __forceinline__ int side_index(int block, int row, int nt_blocks, int col)   // in floats
{
    const int lane = ((row & 7) << 2) | ((col & 7) >> 1);
    return (((block * nt_blocks + (col >> 3)) * 32 + lane) << 2) | ((row >> 3) << 1) | (col & 1);
}

template <int RB, int NT>
__device__ __forceinline__ void keep(float *side, const float (&acc)[RB][NT][4])
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int r = 0; r < RB; ++r)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
            *reinterpret_cast<float4 *>(side + ((r * NT + nt) * 32 + lane) * 4) =
                make_float4(acc[r][nt][0], acc[r][nt][1], acc[r][nt][2], acc[r][nt][3]);
}

// One warp's run of a block's items.  Items are numbered 0 .. items-1; each is
// up to 16*RB rows times all of K (`per` units).  The run is units [begin, end)
// of the items laid end to end: it may start or stop inside an item.
//
// Items is the kernel's view of its work: rows(item) gives its rows, kStep the
// rows from one block to the next, cols(item) the number of columns,
// columns<NT>(item, x) sets this lane's column pointers, and done<NT>(item,
// first, last, acc) takes the sums of a piece; first / last say whether the
// piece holds the item's first and last unit.
//
// The ring holds whole units, one stage for each of the RB row blocks; the
// stages of blocks that an item does not have stay unread.
template <class F, int RB, int PLANES, class Items>
class Stream {
public:
    static constexpr int kStageBytes = Room<F, RB>::kStage;
    static constexpr int kUnits = Room<F, RB>::kUnits;
    static constexpr int kLanes = F::kRowPiece / 16;   // lanes that copy one row
    static constexpr int kAtOnce = 32 / kLanes;        // rows of one copy instruction

    __device__ __forceinline__ Stream(const Items &items, const Weights &w, int K, int n_items, uint32_t ring)
        : items_(items), w_(w), K_(K), per_((K + F::kUnit - 1) / F::kUnit)
    {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        g_ = lane >> 2;
        t_ = lane & 3;
        const int64_t total = (int64_t)n_items * per_;
        begin_ = (int)(total * warp / F::kWarps);
        end_ = (int)(total * (warp + 1) / F::kWarps);
        const int row = lane / kLanes, piece = lane % kLanes;
        put_ = ring + warp * Room<F, RB>::kWarpRing + row * F::kRowPiece + (piece ^ F::fold(row)) * 16;
        get_ = ring + warp * Room<F, RB>::kWarpRing + g_ * F::kRowPiece + (g_ & 1) * 64 + F::place(g_, t_);
        left_ = end_ - begin_;
        item_ahead_ = first_item_ = quick_div(begin_, per_);
        u_ahead_ = begin_ - item_ahead_ * per_;
        slot_ahead_ = slot_ = 0;
        fresh_ = true;
    }

    // the first copies of the run; they read weights only
    __device__ __forceinline__ void start()
    {
        for (int s = 0; s < kUnits; ++s) {
            open();
#pragma unroll
            for (int r = 0; r < RB; ++r)
                issue(r);
        }
    }

    __device__ __forceinline__ void run()
    {
        int item = first_item_, u0 = begin_ - item * per_, left = end_ - begin_;
        open_item = -1;
        while (left > 0) {
            const int u1 = min(per_, u0 + left);
            if (u0 == 0 && u1 < per_)
                open_item = item;
            if (items_.cols(item) <= 8)
                piece<1>(item, u0, u1);
            else
                piece<2>(item, u0, u1);
            left -= u1 - u0;
            ++item;
            u0 = 0;
        }
    }

    // All threads, after their run: holds a barrier, after which the kept pieces may be read.  begins: F::kWarps + 1
    // ints of shared memory.
    __device__ __forceinline__ void meet(int *begins)
    {
        if ((threadIdx.x & 31) == 0) {
            const int warp = threadIdx.x >> 5;
            begins[warp] = begin_;
            if (warp == F::kWarps - 1)
                begins[F::kWarps] = end_;
        }
        __syncthreads();
        // the warps (a bit each) that went on with the item that this one began
        unsigned more = 0;
        if (open_item >= 0) {
            const int stop = (open_item + 1) * per_;
#pragma unroll
            for (int o = 1; o < F::kWarps; ++o)
                more |= (unsigned)(o > (threadIdx.x >> 5) && begins[o] < stop && begins[o] < begins[o + 1]) << o;
        }
        more_ = more;
    }

    // The sums at places `at` of the item that this warp began and others went on with: the pieces in the order of K.
    // `dynamic`: the ring, whose warps' parts hold the pieces that begin an item, then the side blocks.
    template <int N>
    __device__ __forceinline__ void add_pieces(const uint8_t *dynamic, const int (&at)[N], float (&v)[N]) const
    {
        const int warp = threadIdx.x >> 5;
#pragma unroll
        for (int i = 0; i < N; ++i)
            v[i] = reinterpret_cast<const float *>(dynamic + warp * Room<F, RB>::kWarpRing)[at[i]];
        for (unsigned m = more_; m != 0; m &= m - 1) {
            const uint8_t *kept = dynamic + Room<F, RB>::kRing + (__ffs(m) - 1) * Room<F, RB>::kSide;
            const float *p = reinterpret_cast<const float *>(kept);
#pragma unroll
            for (int i = 0; i < N; ++i)
                v[i] = __fadd_rn(v[i], p[at[i]]);
        }
    }

    // The same for all of the item's sums, as the lanes hold them: four of a lane by one load.  For an item of many
    // columns: each sum by itself took 8 of the 24 us of 24x7168x4096.  The experts' entries have few columns, and
    // there the sums by themselves are faster (64 experts' pieces for 13 tokens: 70 us, so 76).
    template <int NT>
    __device__ __forceinline__ void join(const uint8_t *dynamic, float (&acc)[RB][NT][4]) const
    {
        const int lane = threadIdx.x & 31;
        const auto add = [&](const uint8_t *kept, bool more) {
            const float4 *p = reinterpret_cast<const float4 *>(kept) + lane;
#pragma unroll
            for (int r = 0; r < RB; ++r)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const float4 v = p[(r * NT + nt) * 32];
                    acc[r][nt][0] = more ? __fadd_rn(acc[r][nt][0], v.x) : v.x;
                    acc[r][nt][1] = more ? __fadd_rn(acc[r][nt][1], v.y) : v.y;
                    acc[r][nt][2] = more ? __fadd_rn(acc[r][nt][2], v.z) : v.z;
                    acc[r][nt][3] = more ? __fadd_rn(acc[r][nt][3], v.w) : v.w;
                }
        };
        add(dynamic + (threadIdx.x >> 5) * Room<F, RB>::kWarpRing, false);
        for (unsigned m = more_; m != 0; m &= m - 1)
            add(dynamic + Room<F, RB>::kRing + (__ffs(m) - 1) * Room<F, RB>::kSide, true);
    }

    int open_item;   // the item that this warp's run began and did not finish, or -1

private:
    // moves on to the next unit to copy
    __device__ __forceinline__ void open()
    {
        live_ = left_ > 0;
        if (!live_)
            return;
        --left_;
        const int row_bytes = (int)F::row_bytes(K_), lane = threadIdx.x & 31;
        if (fresh_) {
            const RowRange r = items_.rows(item_ahead_);
            const int row = lane / kLanes;
            const int64_t mine = (int64_t)row * row_bytes;
            pa_ = w_.data + r.a * row_bytes + mine;
            pb_ = w_.data + r.b * row_bytes + mine;
            n_ = r.n - row;
            m_ = r.m - row;
            fresh_ = false;
        }
        off_ = u_ahead_ * F::kRowPiece + (lane % kLanes) * 16;
        if (off_ >= row_bytes)    // past the row: zeros
            n_ = m_ = 0;
        if (++u_ahead_ == per_) {
            u_ahead_ = 0;
            ++item_ahead_;
            fresh_ = true;
        }
    }

    // its copies of row block r (zeros for rows that it does not have)
    __device__ __forceinline__ void issue(int r)
    {
        if (live_) {
            const int row_bytes = (int)F::row_bytes(K_);
#pragma unroll
            for (int i = 0; i < 8 / kAtOnce; ++i) {
                const int row = r * Items::kStep + i * kAtOnce, off = off_ + row * row_bytes;
                const uint32_t dst = (put_ ^ F::refold(i)) + slot_ahead_ + r * kStageBytes + i * kAtOnce * F::kRowPiece;
                cp_async16(dst, pa_ + off, row < n_);
                cp_async16(dst + 8 * F::kRowPiece, pb_ + off, row < m_);
            }
        }
        if (r == RB - 1) {
            cp_async_commit();
            slot_ahead_ = slot_ahead_ == (kUnits - 1) * RB * kStageBytes ? 0 : slot_ahead_ + RB * kStageBytes;
        }
    }

    template <int NT>
    __device__ __forceinline__ void piece(int item, int u0, int u1)
    {
        Columns<NT, PLANES> c;
        items_.template columns<NT>(item, c);
        float acc[RB][NT][4] = {};
        typename F::template Scales<RB, Items::kStep> scales;
        uint4 x[F::kWordsX][NT][PLANES];
        auto load_x = [&](int w, int u) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int p = 0; p < PLANES; ++p)
                    x[w][nt][p] = F::pair(c.load(nt, p, u * F::kUnit + F::lane_column(t_), F::word_column(w)));
        };
        scales.begin(w_, items_.rows(item), K_, g_, t_);
        scales.load(u0);
#pragma unroll
        for (int w = 0; w < F::kWordsX; ++w)
            load_x(w, u0);
        for (int u = u0; u < u1; ++u) {
            open();
            cp_async_wait<kUnits - 1>();
            __syncwarp();   // every lane's copies of the unit have arrived
            uint32_t even[F::kReads], odd[F::kReads];
#pragma unroll
            for (int i = 0; i < F::kReads; ++i) {
                even[i] = (get_ ^ i * F::kReadStep) + slot_;
                odd[i] = even[i] + 64 - 128 * (g_ & 1);
            }
#pragma unroll
            for (int r = 0; r < RB; ++r) {
                uint4 a[F::kPieces], b[F::kPieces];
#pragma unroll
                for (int j = 0; j < F::kPieces; ++j) {   // 64 bytes of a row: those of odd rows change places
                    const int offset = r * kStageBytes + (j & ~1) * 64;
                    a[j] = F::read(j & 1 ? odd : even, offset);
                    b[j] = F::read(j & 1 ? odd : even, offset + 8 * F::kRowPiece);
                }
                __syncwarp();   // every lane has read the stage
                issue(r);
                F::template block<RB, Items::kStep, NT, PLANES>(a, b, r, scales, x, t_, acc[r], [&](int w) {
                    if (r == RB - 1)
                        load_x(w, u + 1);
                });
            }
            scales.load(u + 1);
            slot_ = slot_ == (kUnits - 1) * RB * kStageBytes ? 0 : slot_ + RB * kStageBytes;
        }
        items_.template done<NT>(item, u0 == 0, u1 == per_, acc);
    }

    const Items &items_;
    const Weights &w_;
    int K_, per_, g_, t_;
    unsigned more_;
    int begin_, end_, left_, first_item_, item_ahead_, u_ahead_;
    int slot_ahead_, slot_, off_;
    uint32_t put_, get_;
    const uint8_t *pa_, *pb_;
    int n_, m_;
    bool fresh_, live_;
};

}  // namespace ep
