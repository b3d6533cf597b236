// Low-rank adapters (internal): what the kernels for few rows (ep_lora.cu) and for
// many (ep_lora_many.cu) share.
#pragma once

#include <cuda_runtime.h>

#include "ep_device.cuh"
#include "ep_internal.h"

namespace ep {

constexpr int kLoraFewRows = 1024;      // most of the kernels for few rows
constexpr int kLoraMaxRank = 128;
constexpr int kLoraMaxSplits = 16;      // parts of K
constexpr int kLoraBlocks = 2 * 152;    // that fill the GPU
constexpr int kPlanes = 3;              // bf16 terms of v

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

// Four of them, r % 4 == 0.
__device__ __forceinline__ float4 four_ranks_of(const Lora &p, int64_t m, int r, float scaling)
{
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (m < 0 || r >= p.R)
        return v;
    const float4 *part = reinterpret_cast<const float4 *>(p.parts + m * p.R + r);
    const int64_t next = p.M * p.R / 4;
    for (int z = 0; z < p.splits; z += 4) {
        float4 u[4];   // loaded together
#pragma unroll
        for (int i = 0; i < 4; ++i)
            u[i] = z + i < p.splits ? part[(z + i) * next] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v.x = __fadd_rn(v.x, u[i].x);
            v.y = __fadd_rn(v.y, u[i].y);
            v.z = __fadd_rn(v.z, u[i].z);
            v.w = __fadd_rn(v.w, u[i].w);
        }
    }
    return make_float4(__fmul_rn(v.x, scaling), __fmul_rn(v.y, scaling), __fmul_rn(v.z, scaling), __fmul_rn(v.w, scaling));
}

// Two values as sums of kPlanes bf16 terms each: the first eight bits, the next and the last, by cutting, which is
// exact.  What is left of an infinity or NaN is nothing.
__device__ __forceinline__ void split(float2 v, uint32_t (&w)[kPlanes])
{
    uint32_t a = __float_as_uint(v.x), b = __float_as_uint(v.y);
    if ((a & 0x7f800000u) == 0x7f800000u || (b & 0x7f800000u) == 0x7f800000u) {
        // a NaN keeps a bit that the first term holds
        a |= isnan(v.x) ? 0x400000u : 0u;
        b |= isnan(v.y) ? 0x400000u : 0u;
        w[0] = a >> 16 | (b & 0xffff0000u);
        v.x = isfinite(v.x) ? __fsub_rn(v.x, __uint_as_float(a & 0xffff0000u)) : 0.0f;
        v.y = isfinite(v.y) ? __fsub_rn(v.y, __uint_as_float(b & 0xffff0000u)) : 0.0f;
    } else {
        w[0] = a >> 16 | (b & 0xffff0000u);
        v.x = __fsub_rn(v.x, __uint_as_float(a & 0xffff0000u));
        v.y = __fsub_rn(v.y, __uint_as_float(b & 0xffff0000u));
    }
#pragma unroll
    for (int i = 1; i < kPlanes; ++i) {
        a = __float_as_uint(v.x);
        b = __float_as_uint(v.y);
        w[i] = a >> 16 | (b & 0xffff0000u);
        v.x = __fsub_rn(v.x, __uint_as_float(a & 0xffff0000u));
        v.y = __fsub_rn(v.y, __uint_as_float(b & 0xffff0000u));
    }
}

__device__ __forceinline__ float scaling_of(const Lora &p, int adapter)
{
    return adapter < 0 || p.scaling == nullptr
               ? 1.0f : __uint_as_float(ld_global(reinterpret_cast<const uint32_t *>(p.scaling) + adapter));
}

// The two kernels for more than kLoraFewRows rows.
int launch_lora_many(const Lora &p, cudaStream_t stream);

}  // namespace ep
