// rows.cuh -- one token's row in its owner's page: where it lies and, for the
// 4-bit and fp8 caches, how 8 consecutive values become codes.  Shared by the
// append, read-back and norm-and-rotate kernels.
//
// Ownership follows "Efficient Decode Context Parallelism with vLLM for Long
// Context Workloads", section 4, with the granularity of the "Decode Context
// Parallel Guide"'s cp_kv_cache_interleave_size.
#pragma once

#include <cuda_fp4.h>

#include "common.cuh"
#include "kernels.h"

namespace dcp {

// Bytes of a 4-bit block: one KV head's rows of one page, codes then scales.
__host__ __device__ __forceinline__ int fp4_block_bytes(int P, int D) { return P * (D / 2 + D / 16); }

// Resolve (req, pos) -> physical page and in-page offset; -1 page when invalid,
// -2 when another rank owns the position (rank-local cache).
__device__ __forceinline__ int append_target(const AppendArgs& a, int64_t i, int* off) {
    const int p = a.pos[i];
    int b = a.req ? a.req[i] : (int)i;
    if (p < 0 || b < 0 || b >= a.batch) return -1;
    // positions are below 2^31, so unsigned 32-bit division serves: p / (I N) = (p / I) / N
    const uint32_t q = (uint32_t)p / (uint32_t)a.interleave;
    const uint32_t round = q / (uint32_t)a.n_shards;
    int r = (int)(q - round * (uint32_t)a.n_shards);
    if (a.only_shard >= 0) {
        if (r != a.only_shard) return -2;
        r = 0;  // the rank's tables are row 0
    }
    const uint32_t l = round * (uint32_t)a.interleave + ((uint32_t)p - q * (uint32_t)a.interleave);
    const int j = (int)(l >> (a.page_size == 16 ? 4 : 6));  // pages are 16 or 64 tokens
    if (j >= a.max_local_pages) return -1;
    int pg = a.block_tables[((int64_t)r * a.batch + b) * a.max_local_pages + j];
    if (pg < 0 || pg >= a.num_pages) return -1;
    *off = (int)(l & (uint32_t)(a.page_size - 1));
    return pg;
}

__device__ __forceinline__ uint32_t max2_nan(uint32_t a, uint32_t b) {  // bf16x2, a NaN wins
    const __nv_bfloat162 m = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                         *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&m);
}

__device__ __forceinline__ void unpack8(const uint4& w, float* x) {
    const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 4; e++) {
        x[2 * e] = bf16_lo(ws[e]);
        x[2 * e + 1] = bf16_hi(ws[e]);
    }
}

// Scale byte of a run whose largest magnitude is the larger half of am2 (bf16x2, a NaN
// wins): e4m3(amax / (6 factor)), and the scale's value times the factor.
//
// Divisions by the scale (and by 6) are products with the reciprocal, for factor 1:
// the dividend has 8 significant bits and a border between two codes, times the
// divisor, at most 7, so that the quotient either IS the border or is 2^-15 away from
// it, relatively.  The product is within 2^-22 of the quotient; rounding it to 18 bits
// (snap) puts it back on the border exactly when the quotient is there, and the
// conversion then takes the even code.
__device__ __forceinline__ float snap(float x) { return __uint_as_float((__float_as_uint(x) + 0x20u) & ~0x3fu); }

__device__ __forceinline__ uint8_t fp4_scale(uint32_t am2, float factor, float* scale) {
    const float amax = bf16_lo(max2_nan(am2, am2 >> 16));
    // an infinity or NaN passes through neither the reciprocal nor the rounding
    const float q = factor == 1.f && amax < 1e38f ? snap(amax * (1.f / 6.f)) : __fdiv_rn(amax, 6.f * factor);
    const uint8_t sb = __nv_cvt_float_to_fp8(q, __NV_SATFINITE, __NV_E4M3);
    const __half_raw hr = __nv_cvt_fp8_to_halfraw(sb, __NV_E4M3);
    *scale = __half2float(*reinterpret_cast<const __half*>(&hr)) * factor;
    return sb;
}

__device__ __forceinline__ uint32_t fp4_abs_max(const uint4& v) {
    constexpr uint32_t kAbs = 0x7fff7fffu;
    return max2_nan(max2_nan(v.x & kAbs, v.y & kAbs), max2_nan(v.z & kAbs, v.w & kAbs));
}

// Codes of 8 bf16 values against a scale (zero or NaN: zero codes).  The scale is the
// rounded one, so a value may lie past 6 and saturates there.
__device__ __forceinline__ uint32_t fp4_codes8(const uint4& v, float s, float factor) {
    if (s > 0.f) {
        float x[8];
        unpack8(v, x);
        if (factor == 1.f) {
            const float inv = __frcp_rn(s);
#pragma unroll
            for (int e = 0; e < 8; e++) x[e] = snap(x[e] * inv);
        } else {
#pragma unroll
            for (int e = 0; e < 8; e++) x[e] = __fdiv_rn(x[e], s);
        }
        uint32_t w;
        asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
            "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
            : "=r"(w)
            : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
        return w;
    }
    return 0;
}

// Quantise a run of 16 bf16 values held by two neighbouring lanes, 8 each: returns
// this lane's 8 codes and the run's scale byte.  `both` is the mask of the lanes that
// take part (whole pairs).
__device__ __forceinline__ uint32_t fp4_quantise8(const uint4& v, float factor, uint32_t both, uint8_t* scale_byte) {
    uint32_t am2 = fp4_abs_max(v);
    am2 = max2_nan(am2, __shfl_xor_sync(both, am2, 1));
    float s;
    *scale_byte = fp4_scale(am2, factor, &s);
    return fp4_codes8(v, s, factor);
}

// Codes of 8 values of an fp8 row whose largest magnitude is amax > 0.
__device__ __forceinline__ uint2 fp8_quantise8(const float* x, float scale) {
    uint32_t packed[2] = {0, 0};
#pragma unroll
    for (int e = 0; e < 4; e++) {
        const uint32_t b0 = __nv_cvt_float_to_fp8(__fdiv_rn(x[2 * e], scale), __NV_SATFINITE, __NV_E4M3);
        const uint32_t b1 = __nv_cvt_float_to_fp8(__fdiv_rn(x[2 * e + 1], scale), __NV_SATFINITE, __NV_E4M3);
        packed[e >> 1] |= (b0 | (b1 << 8)) << (16 * (e & 1));
    }
    return make_uint2(packed[0], packed[1]);
}

__device__ __forceinline__ uint4 pack8(const float* x) {
    uint4 w;
    uint32_t* ws = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
    for (int e = 0; e < 4; e++) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
        ws[e] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return w;
}

// Store 8 values (dimensions 8 li .. 8 li + 7, bf16 in `w`) of KV head g's row at
// (pg, off) of a 4-bit pool.  Every lane of `both` takes part: the row's D/8 lanes.
__device__ __forceinline__ void store_fp4x8(const AppendArgs& a, uint8_t* pool, int pg, int g, int off, int li,
                                            const uint4& w, float factor, uint32_t both) {
    const int D = a.dk, P = a.page_size;
    uint8_t sb;
    const uint32_t codes = fp4_quantise8(w, factor, both, &sb);
    uint8_t* blk = pool + ((int64_t)pg * a.hkv + g) * fp4_block_bytes(P, D);
    *reinterpret_cast<uint32_t*>(blk + off * (D / 2) + li * 4) = codes;
    if ((li & 1) == 0) blk[P * (D / 2) + (li >> 1) * P + off] = sb;
}

}  // namespace dcp
