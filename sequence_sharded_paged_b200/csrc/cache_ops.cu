// cache_ops.cu -- shard map, per-shard counts and KV append (integer / copy work).
//
// Ownership follows the interleaved split of "Efficient Decode Context
// Parallelism with vLLM for Long Context Workloads", section 4 (each GPU holds
// the KV of a subset of positions) with the granularity of the "Decode
// Context Parallel Guide"'s cp_kv_cache_interleave_size: p -> shard
// (p / I) mod N, local index (p / (I N)) * I + p mod I.
#include "common.cuh"
#include "kernels.h"
#include "rows.cuh"

namespace dcp {

__global__ void shard_counts_kernel(int B, const int32_t* __restrict__ seq_lens, int N, int I,
                                    int32_t* __restrict__ counts, int* status) {
    int i = blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= N * B) return;
    int n = i / B, b = i - n * B;
    int64_t L = seq_lens[b];
    if (L < 0) {
        record_status(status, DCP_ERR_INVALID_ARG);
        L = 0;
    }
    counts[i] = (int32_t)count_of(L, N, I, n);
}

__global__ void shard_map_kernel(int64_t n_pos, const int32_t* __restrict__ pos, const int32_t* __restrict__ req,
                                 int N, int I, int P, const int32_t* __restrict__ bt, int B, int maxp, int num_pages,
                                 int32_t* __restrict__ rank_out, int32_t* __restrict__ local_out,
                                 int64_t* __restrict__ slot_out, int* status) {
    int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= n_pos) return;
    int64_t p = pos[i];
    int b = req ? req[i] : (int)i;
    if (p < 0) {
        record_status(status, DCP_ERR_INVALID_ARG);
        rank_out[i] = -1;
        local_out[i] = -1;
        slot_out[i] = -1;
        return;
    }
    int r = owner_of(p, N, I);
    int64_t l = local_of(p, N, I);
    rank_out[i] = r;
    local_out[i] = (int32_t)l;
    int64_t j = l / P;
    int pg = -1;
    if (b >= 0 && b < B && j < maxp) pg = bt[((int64_t)r * B + b) * maxp + j];
    if (pg < 0 || pg >= num_pages) {
        record_status(status, DCP_ERR_UNALLOCATED_PAGE);
        slot_out[i] = -1;
    } else {
        slot_out[i] = (int64_t)pg * P + l % P;
    }
}

// GQA: one warp per (token, kv head): copy the K and V rows (16-byte vectors).
__global__ void append_gqa_kernel(AppendArgs a) {
    int64_t w = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    int lane = threadIdx.x & 31;
    if (w >= a.n_tok * a.hkv) return;
    int64_t i = w / a.hkv;
    int g = (int)(w - i * a.hkv);
    int off = 0;
    int pg = append_target(a, i, &off);
    if (pg < 0) {
        if (pg == -1 && lane == 0) record_status(a.status, DCP_ERR_UNALLOCATED_PAGE);
        return;
    }
    const int P = a.page_size;
    {
        const uint4* src = reinterpret_cast<const uint4*>(a.k_new + ((i * a.hkv + g) * a.dk) * 2);
        uint4* dst = reinterpret_cast<uint4*>(a.k_pages + ((((int64_t)pg * a.hkv + g) * P + off) * a.dk) * 2);
        for (int v = lane; v < a.dk / 8; v += 32) dst[v] = src[v];
    }
    {
        const uint4* src = reinterpret_cast<const uint4*>(a.v_new + ((i * a.hkv + g) * a.dv) * 2);
        uint4* dst = reinterpret_cast<uint4*>(a.v_pages + ((((int64_t)pg * a.hkv + g) * P + off) * a.dv) * 2);
        for (int v = lane; v < a.dv / 8; v += 32) dst[v] = src[v];
    }
}

// MLA bf16: one warp per token: copy the 576-wide latent row.
__global__ void append_mla_bf16_kernel(AppendArgs a) {
    int64_t i = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    int lane = threadIdx.x & 31;
    if (i >= a.n_tok) return;
    int off = 0;
    int pg = append_target(a, i, &off);
    if (pg < 0) {
        if (pg == -1 && lane == 0) record_status(a.status, DCP_ERR_UNALLOCATED_PAGE);
        return;
    }
    const uint4* src = reinterpret_cast<const uint4*>(a.k_new + i * a.dk * 2);
    uint4* dst = reinterpret_cast<uint4*>(a.k_pages + (((int64_t)pg * a.page_size + off) * a.dk) * 2);
    for (int v = lane; v < a.dk / 8; v += 32) dst[v] = src[v];
}

// MLA fp8: one warp per token: amax over the row, scale = amax / 448 (fp32,
// round to nearest), code = RNE(x / scale) saturated to +-448.
__global__ void append_mla_fp8_kernel(AppendArgs a) {
    int64_t i = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    int lane = threadIdx.x & 31;
    if (i >= a.n_tok) return;
    int off = 0;
    int pg = append_target(a, i, &off);
    if (pg < 0) {
        if (pg == -1 && lane == 0) record_status(a.status, DCP_ERR_UNALLOCATED_PAGE);
        return;
    }
    // 576 bf16 = 72 chunks of 8; lane owns chunks lane, lane+32, lane+64 (< 72)
    const uint4* src = reinterpret_cast<const uint4*>(a.k_new + i * a.dk * 2);
    const int nch = a.dk / 8;
    uint4 c[3];
    float amax = 0.f;
#pragma unroll
    for (int k = 0; k < 3; k++) {
        int ch = lane + 32 * k;
        if (ch < nch) {
            c[k] = src[ch];
            uint32_t w[4] = {c[k].x, c[k].y, c[k].z, c[k].w};
#pragma unroll
            for (int e = 0; e < 4; e++) amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(w[e])), fabsf(bf16_hi(w[e]))));
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    float scale = amax == 0.f ? 1.f : __fdiv_rn(amax, 448.f);
    uint8_t* dst = a.k_pages + ((int64_t)pg * a.page_size + off) * a.dk;
#pragma unroll
    for (int k = 0; k < 3; k++) {
        int ch = lane + 32 * k;
        if (ch < nch) {
            uint32_t w[4] = {c[k].x, c[k].y, c[k].z, c[k].w};
            uint32_t packed[2] = {0, 0};
#pragma unroll
            for (int e = 0; e < 4; e++) {
                float x0 = amax == 0.f ? 0.f : __fdiv_rn(bf16_lo(w[e]), scale);
                float x1 = amax == 0.f ? 0.f : __fdiv_rn(bf16_hi(w[e]), scale);
                uint32_t b0 = __nv_cvt_float_to_fp8(x0, __NV_SATFINITE, __NV_E4M3);
                uint32_t b1 = __nv_cvt_float_to_fp8(x1, __NV_SATFINITE, __NV_E4M3);
                packed[e >> 1] |= (b0 | (b1 << 8)) << (16 * (e & 1));
            }
            *reinterpret_cast<uint2*>(dst + ch * 8) = make_uint2(packed[0], packed[1]);
        }
    }
    if (lane == 0) a.kv_scales[(int64_t)pg * a.page_size + off] = scale;
}

// GQA, 4-bit: D/16 lanes per token, a run of 16 dimensions (one scale) each.  The
// token's page is looked up once for up to kHeadsPerLane heads, whose K and V rows are
// all loaded before any is quantised.  The floor is HBM's, 4 D bytes in and
// 2 (D/2 + D/16) out for each head; what bounds it is the arithmetic of the codes (issue
// slots and the ALU pipe are 74% busy, DRAM 48%).  50021 prompt tokens of 8 heads of 128,
// 263 MB: append 59 us, 4.5 TB/s (68 us with a byte stored for each scale, whose scattered
// stores were waited for); read-back 44 us, 5.9 TB/s.
constexpr int kHeadsPerLane = 2;

// A warp holds the same head's rows of four tokens that follow one another in the call:
// in a prompt they do in a page too, and their scales are one word.
struct RowLane {
    int64_t i;  // token
    int g0;     // first head
    int li;     // run of dimensions
    int pg, off;
};

__device__ __forceinline__ int row_shift(const AppendArgs& a) { return a.dk == 128 ? 3 : 2; }  // log2 of D/16

__device__ __forceinline__ RowLane row_lane(const AppendArgs& a) {
    const int shift = row_shift(a);
    const int hb = (a.hkv + kHeadsPerLane - 1) / kHeadsPerLane;
    const int64_t w = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> shift, four = w >> 2;
    const int64_t t = four >> 32 ? four / hb : (int64_t)((uint32_t)four / (uint32_t)hb);
    RowLane r{4 * t + (w & 3), (int)(four - t * hb) * kHeadsPerLane, (int)threadIdx.x & ((1 << shift) - 1), -2, 0};
    if (r.i < a.n_tok) r.pg = append_target(a, r.i, &r.off);
    if (r.pg == -1 && r.li == 0 && r.g0 == 0) record_status(a.status, DCP_ERR_UNALLOCATED_PAGE);
    return r;
}
static int64_t row_lanes(const AppendArgs& a) {
    return (a.n_tok + 3) / 4 * 4 * ((a.hkv + kHeadsPerLane - 1) / kHeadsPerLane) * (a.dk / 16);
}

// 32 bytes at once where the address allows it (`wide`): a warp's requests are then whole
// lines instead of two halves of each (read-back of 50021 tokens 54 -> 43 us; loads gain
// nothing from it, the second half comes from L1).
__device__ __forceinline__ void store32(uint8_t* p, bool wide, const uint4* v) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0].x), "r"(v[0].y),
                     "r"(v[0].z), "r"(v[0].w), "r"(v[1].x), "r"(v[1].y), "r"(v[1].z), "r"(v[1].w)
                     : "memory");
    } else {
        reinterpret_cast<uint4*>(p)[0] = v[0];
        reinterpret_cast<uint4*>(p)[1] = v[1];
    }
}
__device__ __forceinline__ bool aligned32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }

// Stores a lane's run: codes, and the scales of the warp's four tokens as a word where
// they lie in one (`word`).  Executed by whole warps; `live`: this lane has a row.
__device__ __forceinline__ void store_fp4x16(uint8_t* blk, int P, int D, int off, int li, const uint4* v, float factor,
                                             bool live, bool word, int shift) {
    float s;
    const uint32_t sb = fp4_scale(max2_nan(fp4_abs_max(v[0]), fp4_abs_max(v[1])), factor, &s);
    uint32_t all = sb | __shfl_down_sync(0xffffffffu, sb, 1 << shift) << 8;
    all |= __shfl_down_sync(0xffffffffu, all, 2 << shift) << 16;
    if (!live) return;
    *reinterpret_cast<uint2*>(blk + off * (D / 2) + li * 8) =
        make_uint2(fp4_codes8(v[0], s, factor), fp4_codes8(v[1], s, factor));
    uint8_t* scale = blk + P * (D / 2) + li * P + off;
    if (!word)
        *scale = (uint8_t)sb;
    else if ((off & 3) == 0)
        *reinterpret_cast<uint32_t*>(scale) = all;
}

__global__ void __launch_bounds__(256, 4) append_gqa_fp4_kernel(AppendArgs a) {
    const RowLane r = row_lane(a);
    const int P = a.page_size, D = a.dk, lane = threadIdx.x & 31, shift = row_shift(a);
    // do the four tokens lie in one page, from a multiple of 4 on?
    const int four = 3 << shift, first = lane & ~four;
    const int pg0 = __shfl_sync(0xffffffffu, r.pg, first), off0 = __shfl_sync(0xffffffffu, r.off, first);
    const bool fits = r.pg >= 0 && r.pg == pg0 && (off0 & 3) == 0 && r.off - off0 == (lane & four) >> shift;
    const uint32_t tokens = (1u | 1u << (1 << shift) | 1u << (2 << shift) | 1u << (3 << shift)) << first;
    const bool word = (__ballot_sync(0xffffffffu, fits) & tokens) == tokens;
    const float fk = a.kv_scales ? __ldg(a.kv_scales) : 1.f, fv = a.kv_scales ? __ldg(a.kv_scales + 1) : 1.f;
    uint4 k[kHeadsPerLane][2], v[kHeadsPerLane][2];
#pragma unroll
    for (int e = 0; e < kHeadsPerLane; e++) {
        const bool live = r.pg >= 0 && r.g0 + e < a.hkv;
        const int64_t at = ((r.i * a.hkv + r.g0 + e) * D + r.li * 16) * 2;
#pragma unroll
        for (int h = 0; h < 2; h++) {
            k[e][h] = v[e][h] = make_uint4(0, 0, 0, 0);
            if (live) k[e][h] = __ldg(reinterpret_cast<const uint4*>(a.k_new + at) + h);
            if (live) v[e][h] = __ldg(reinterpret_cast<const uint4*>(a.v_new + at) + h);
        }
    }
#pragma unroll
    for (int e = 0; e < kHeadsPerLane; e++) {
        const bool live = r.pg >= 0 && r.g0 + e < a.hkv;
        const int64_t blk = ((int64_t)r.pg * a.hkv + r.g0 + e) * fp4_block_bytes(P, D);
        store_fp4x16(a.k_pages + blk, P, D, r.off, r.li, k[e], fk, live, word, shift);
        store_fp4x16(a.v_pages + blk, P, D, r.off, r.li, v[e], fv, live, word, shift);
    }
}

// 16 values of a 4-bit row as bf16.
__device__ __forceinline__ void unpack_fp4x16(uint2 codes, uint8_t scale, float factor, uint4* out) {
    const __half_raw hr = __nv_cvt_fp8_to_halfraw(scale, __NV_E4M3);
    const float s = __half2float(*reinterpret_cast<const __half*>(&hr)) * factor;
#pragma unroll
    for (int h = 0; h < 2; h++) {
        const uint32_t c = h ? codes.y : codes.x;
        float x[8];
#pragma unroll
        for (int e = 0; e < 4; e++) {
            const __half2_raw h2 = __nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)(c >> (8 * e)), __NV_E2M1);
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
            x[2 * e] = f.x * s;
            x[2 * e + 1] = f.y * s;
        }
        out[h] = pack8(x);
    }
}

// Read-back, GQA: the append's lanes in reverse.
template <bool FP4>
__global__ void __launch_bounds__(256, FP4 ? 6 : 4) gather_gqa_kernel(AppendArgs a, uint8_t* k_out, uint8_t* v_out) {
    const RowLane r = row_lane(a);
    if (r.pg < 0) return;
    const int P = a.page_size, D = a.dk;
    const float fk = FP4 && a.kv_scales ? __ldg(a.kv_scales) : 1.f, fv = FP4 && a.kv_scales ? __ldg(a.kv_scales + 1) : 1.f;
    const uint8_t* pools[2] = {a.k_pages, a.v_pages};
    uint8_t* outs[2] = {k_out, v_out};
    const bool wide[2] = {aligned32(k_out), aligned32(v_out)};
    uint4 w[2 * kHeadsPerLane][2];  // bf16: the row's bytes; 4-bit: codes in x, y and the scale in z
#pragma unroll
    for (int e = 0; e < 2 * kHeadsPerLane; e++) {
        const int g = r.g0 + (e >> 1);
        if (g >= a.hkv || !outs[e & 1]) continue;
        const int64_t row = (int64_t)r.pg * a.hkv + g;
        if (FP4) {
            const uint8_t* blk = pools[e & 1] + row * fp4_block_bytes(P, D);
            const uint2 c = __ldg(reinterpret_cast<const uint2*>(blk + r.off * (D / 2) + r.li * 8));
            w[e][0] = make_uint4(c.x, c.y, __ldg(blk + P * (D / 2) + r.li * P + r.off), 0);
        } else {
            const uint4* src = reinterpret_cast<const uint4*>(pools[e & 1] + ((row * P + r.off) * D + r.li * 16) * 2);
            w[e][0] = __ldg(src);
            w[e][1] = __ldg(src + 1);
        }
    }
#pragma unroll
    for (int e = 0; e < 2 * kHeadsPerLane; e++) {
        const int g = r.g0 + (e >> 1);
        if (g >= a.hkv || !outs[e & 1]) continue;
        if (FP4) unpack_fp4x16(make_uint2(w[e][0].x, w[e][0].y), (uint8_t)w[e][0].z, e & 1 ? fv : fk, w[e]);
        store32(outs[e & 1] + ((r.i * a.hkv + g) * D + r.li * 16) * 2, wide[e & 1], w[e]);
    }
}

// Read-back, MLA: one warp per token, 8 elements a lane and step.
__global__ void __launch_bounds__(256) gather_mla_kernel(AppendArgs a, uint8_t* k_out) {
    const int64_t i = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    const int lane = threadIdx.x & 31;
    if (i >= a.n_tok) return;
    int off = 0;
    const int pg = append_target(a, i, &off);
    if (pg == -1 && lane == 0) record_status(a.status, DCP_ERR_UNALLOCATED_PAGE);
    if (pg < 0) return;
    const int64_t row = (int64_t)pg * a.page_size + off;
    uint4* dst = reinterpret_cast<uint4*>(k_out + i * a.dk * 2);
    const float s = a.dtype == DCP_FP8_E4M3 ? __ldg(a.kv_scales + row) : 1.f;
    for (int c = lane; c < a.dk / 8; c += 32) {
        if (a.dtype == DCP_BF16) {
            dst[c] = __ldg(reinterpret_cast<const uint4*>(a.k_pages + row * a.dk * 2) + c);
        } else {
            const uint2 w = __ldg(reinterpret_cast<const uint2*>(a.k_pages + row * a.dk) + c);
            const uint32_t ws[2] = {w.x, w.y};
            float x[8];
#pragma unroll
            for (int e = 0; e < 2; e++) {
                const float2 f0 = e4m3x2_to_float2((uint16_t)(ws[e] & 0xFFFF));
                const float2 f1 = e4m3x2_to_float2((uint16_t)(ws[e] >> 16));
                x[4 * e] = f0.x * s;
                x[4 * e + 1] = f0.y * s;
                x[4 * e + 2] = f1.x * s;
                x[4 * e + 3] = f1.y * s;
            }
            dst[c] = pack8(x);
        }
    }
}

static int blocks_for(int64_t threads, int per_block) {
    int64_t g = (threads + per_block - 1) / per_block;
    return (int)(g < 1 ? 1 : g);
}

cudaError_t launch_shard_counts(int B, const int32_t* seq_lens, int N, int I, int32_t* counts, int* status,
                                cudaStream_t s) {
    shard_counts_kernel<<<blocks_for((int64_t)N * B, 256), 256, 0, s>>>(B, seq_lens, N, I, counts, status);
    return cudaGetLastError();
}

cudaError_t launch_shard_map(int64_t n_pos, const int32_t* pos, const int32_t* req, int N, int I, int P,
                             const int32_t* bt, int B, int maxp, int num_pages, int32_t* rank_out,
                             int32_t* local_out, int64_t* slot_out, int* status, cudaStream_t s) {
    if (n_pos == 0) return cudaSuccess;
    shard_map_kernel<<<blocks_for(n_pos, 256), 256, 0, s>>>(n_pos, pos, req, N, I, P, bt, B, maxp, num_pages,
                                                            rank_out, local_out, slot_out, status);
    return cudaGetLastError();
}

cudaError_t launch_append(const AppendArgs& a, cudaStream_t s) {
    if (a.n_tok == 0) return cudaSuccess;
    if (a.dtype == DCP_FP4_E2M1) {
        append_gqa_fp4_kernel<<<blocks_for(row_lanes(a), 256), 256, 0, s>>>(a);
    } else if (a.kind == DCP_GQA) {
        append_gqa_kernel<<<blocks_for(a.n_tok * a.hkv * 32, 256), 256, 0, s>>>(a);
    } else if (a.dtype == DCP_BF16) {
        append_mla_bf16_kernel<<<blocks_for(a.n_tok * 32, 256), 256, 0, s>>>(a);
    } else {
        append_mla_fp8_kernel<<<blocks_for(a.n_tok * 32, 256), 256, 0, s>>>(a);
    }
    return cudaGetLastError();
}

cudaError_t launch_gather(const AppendArgs& a, void* k_out, void* v_out, cudaStream_t s) {
    if (a.n_tok == 0) return cudaSuccess;
    if (a.kind == DCP_GQA) {
        (a.dtype == DCP_FP4_E2M1 ? gather_gqa_kernel<true> : gather_gqa_kernel<false>)
            <<<blocks_for(row_lanes(a), 256), 256, 0, s>>>(a, static_cast<uint8_t*>(k_out),
                                                                   static_cast<uint8_t*>(v_out));
    } else {
        gather_mla_kernel<<<blocks_for(a.n_tok * 32, 256), 256, 0, s>>>(a, static_cast<uint8_t*>(k_out));
    }
    return cudaGetLastError();
}

}  // namespace dcp
