// norm_rope.cu -- norms of queries and keys for each head, the rotation of their
// positions and the append to the owners' pages, in one pass
// (dcp_norm_rope_append).
//
// For a row x of a head: y = x / sqrt(mean x^2 + eps) * w; then each rotated pair
// (a, z) at position p becomes (a cos - z sin, z cos + a sin) with the angle
// p * f_i.  Everything is 32-bit between the bf16 load and the one rounding at the
// store, except the angle: p * f_i reaches 10^6 radians at far positions, where
// 32 bits keep no fraction of a turn.  f_i comes as a multiple of 2^-64 turns, so
// the 64-bit product p * turns[i] IS the angle modulo a turn (integer overflow
// drops the whole turns).  Its upper 32 bits, a signed fraction of a turn, are less than
// 2^-32 turns below it, and their 24-bit float is within another 2^-26 turns (half a turn
// is the largest): 9.5e-8 radians in all, about as much as cosine and sine round.
//
// Bound by HBM: every row is read once and written once, 4 D bytes, so what has to be
// kept down are the instructions for each row.  A row is D/16 lanes that hold two
// chunks of 8 dimensions each, half of the rotated (or of the other) dimensions apart:
// neither layout then exchanges anything between lanes, and a warp's accesses are whole
// lines.  The mean is a shuffle sum.  Cosine and sine are computed once for each token and
// pair and shared by all heads through shared memory; a block takes up to 8 tokens, so
// that positions, tables and angles are looked up side by side.  Rows of a 4-bit cache
// need 16 consecutive dimensions in two neighbouring lanes instead (one scale): D/8
// lanes of 8 dimensions, which exchange the pairs by shuffles and store a byte for each
// scale.
//
// Measured: 16384 tokens of 64 + 4 + 4 heads of 128, half rotated, 604 MB: 110 us, 5.5
// TB/s, 84% of a copy's rate (8 dimensions a lane: 125 us; 16 and the loads of two rows
// ahead, with half the blocks: 120-124 us).  4001 tokens of the MLA latent and 64
// absorbed queries, 599 MB: 105 us, 5.7 TB/s.  128 tokens: 4.3 us, a launch's latency.
//
// Where rows are placed follows "Efficient Decode Context Parallelism with vLLM for
// Long Context Workloads", section 4 (a position's row lies on its owner).
#include "common.cuh"
#include "kernels.h"
#include "rows.cuh"

namespace dcp {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 8;   // tokens per CTA
constexpr int kMlaHeads = 16;   // MLA: query heads per CTA

// cosine and sine of position p's pair i
__device__ __forceinline__ float2 cos_sin(const dcp_rope& rope, int p, int i) {
    const uint64_t t = (uint64_t)(uint32_t)p * rope.turns[i];
    const float half_turns = (float)(int32_t)(uint32_t)(t >> 32) * 4.656612873077393e-10f;  // 2^-31
    float s, c;
    sincospif(half_turns, &s, &c);
    return make_float2(c * rope.attn_factor, s * rope.attn_factor);
}

// One pair: (a, z) turned by the angle of c, s.
__device__ __forceinline__ void turn(float& a, float& z, float c, float s) {
    const float t = fmaf(a, c, -(z * s));
    z = fmaf(z, c, a * s);
    a = t;
}

// Rotate this lane's 8 consecutive values.  Lanes [0, 2h) of the row hold the rot_dim = 16 h
// rotated dimensions (li counts from the first of them); `cs` are the token's
// pairs.  HALF: the partner of dimension d is d +- rot_dim/2, in lane li +- h.
__device__ __forceinline__ void rotate8(float* x, const float2* cs, int layout, int h, int li, int base_lane,
                                        uint32_t mask) {
    if (layout == DCP_ROPE_HALF) {
        const bool low = li < h, in = li < 2 * h;
        const int src = base_lane + (in ? (low ? li + h : li - h) : li);
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; e++) y[e] = __shfl_sync(mask, x[e], src);
        if (!in) return;
        const float4* c4 = reinterpret_cast<const float4*>(cs + (low ? li : li - h) * 8);
#pragma unroll
        for (int e = 0; e < 4; e++) {
            const float4 c = c4[e];  // two pairs: cos, sin, cos, sin
            // low: a cos - z sin with z = y;  high: z cos + a sin with a = y
            const float s0 = low ? -c.y : c.y, s1 = low ? -c.w : c.w;
            x[2 * e] = fmaf(x[2 * e], c.x, y[2 * e] * s0);
            x[2 * e + 1] = fmaf(x[2 * e + 1], c.z, y[2 * e + 1] * s1);
        }
    } else if (li < 2 * h) {
        const float4* c4 = reinterpret_cast<const float4*>(cs + li * 4);
#pragma unroll
        for (int e = 0; e < 2; e++) {
            const float4 c = c4[e];
            turn(x[4 * e], x[4 * e + 1], c.x, c.y);
            turn(x[4 * e + 2], x[4 * e + 3], c.z, c.w);
        }
    }
}

struct NormRopeArgs {
    AppendArgs a;  // k_new / v_new: the strided inputs (null when absent)
    const uint8_t* q;
    int64_t q_stride, k_stride, v_stride;  // elements
    const uint8_t* q_weight;
    const uint8_t* k_weight;
    float eps;
    uint8_t* q_out;
    int32_t hq, tokens, rotate;  // tokens per CTA; rotate: the rope is present
};

// Token of this CTA: page and offset of its row (page -1: unallocated, -2: another
// rank's, -3: padding)
struct Target {
    int pg, off;
};

__device__ __forceinline__ Target find_target(const AppendArgs& a, int64_t i) {
    Target t{-3, 0};
    if (a.pos[i] < 0) return t;
    t.pg = append_target(a, i, &t.off);
    return t;
}

// FP4: the cache is a 4-bit one.
template <int D, bool FP4>
__global__ void __launch_bounds__(kThreads, 4) norm_rope_gqa_kernel(const __grid_constant__ NormRopeArgs n,
                                                                    const __grid_constant__ dcp_rope rope) {
    constexpr int V = FP4 ? 1 : 2;          // chunks of 8 dimensions a lane
    constexpr int LPR = D / (8 * V);        // lanes per row
    constexpr int GROUPS = kThreads / LPR;  // rows in flight
    struct Chunks {
        uint4 v[V];
    };
    __shared__ __align__(16) float2 s_cs[kMaxTokens * DCP_ROPE_MAX_PAIRS];
    __shared__ Target s_target[kMaxTokens];
    const AppendArgs& a = n.a;
    const int64_t i0 = (int64_t)blockIdx.x * n.tokens;
    const int nt = (int)min((int64_t)n.tokens, a.n_tok - i0);
    const int lane = threadIdx.x & 31, li = lane % LPR, base_lane = lane - li;
    const int grp = threadIdx.x / LPR;
    const uint32_t mask = ((1u << LPR) - 1u) << base_lane;
    const int nq = n.q ? n.hq : 0, nk = a.k_new ? a.hkv : 0;
    const int rows = nq + 2 * nk;  // queries, keys, values of one token

    // this lane's dimensions: chunks at o0 and, apart by half of the rotated or of the
    // other dimensions, at o1
    const int rot_lanes = n.rotate ? rope.rot_dim / (8 * V) : 0;
    const bool turns = li < rot_lanes, half = rope.layout == DCP_ROPE_HALF;
    const int part = turns ? 8 * V * rot_lanes : D - 8 * V * rot_lanes;  // dimensions of the part
    const int o0 = FP4 || turns ? 8 * li : 8 * (V - 1) * rot_lanes + 8 * li, o1 = o0 + part / 2;

    // rows are numbered token by token; a group steps GROUPS rows at a time
    struct At {
        int t, h;
    };
    auto next = [&](At& p) {
        p.h += GROUPS;
        while (p.h >= rows) {
            p.h -= rows;
            p.t++;
        }
    };
    auto load = [&](const uint8_t* row) -> Chunks {  // not read-only loads: q_out may be q
        Chunks w;
        w.v[0] = *reinterpret_cast<const uint4*>(row + o0 * 2);
        if (V == 2) w.v[V - 1] = *reinterpret_cast<const uint4*>(row + o1 * 2);
        return w;
    };
    auto source = [&](const At& p) -> const uint8_t* {
        const int64_t i = i0 + p.t;
        const uint8_t* base = n.q;
        int64_t at = i * n.q_stride;
        int h = p.h;
        if (h >= nq) {
            h -= nq;
            base = a.k_new;
            at = i * n.k_stride;
            if (h >= nk) {
                h -= nk;
                base = a.v_new;
                at = i * n.v_stride;
            }
        }
        return base + (at + h * D) * 2;
    };
    auto store = [&](uint8_t* row, const Chunks& w) {
        *reinterpret_cast<uint4*>(row + o0 * 2) = w.v[0];
        if (V == 2) *reinterpret_cast<uint4*>(row + o1 * 2) = w.v[V - 1];
    };
    // a group's next row is loaded beside the work on this one; the first rows' loads overlap the positions', tables' and angles' work
    Chunks w0 = {};
    At p0{0, grp - GROUPS};
    next(p0);
    if (p0.t < nt) w0 = load(source(p0));
    Chunks qw = {}, kw = {};
    if (n.q_weight) qw = load(n.q_weight);
    if (n.k_weight) kw = load(n.k_weight);

    const int pairs = rope.rot_dim / 2;
    if (n.rotate)
        for (int k = threadIdx.x; k < nt * pairs; k += kThreads) {
            const int t = k / pairs, i = k - t * pairs;
            s_cs[t * DCP_ROPE_MAX_PAIRS + i] = cos_sin(rope, max(0, a.pos[i0 + t]), i);
        }
    if (threadIdx.x >= kThreads - 32 && lane < nt) {
        const Target t = find_target(a, i0 + lane);
        s_target[lane] = t;
        if (nk && t.pg == -1) record_status(a.status, DCP_ERR_UNALLOCATED_PAGE);
    }
    __syncthreads();
    const float fk = FP4 && a.kv_scales && nk ? __ldg(a.kv_scales) : 1.f;
    const float fv = FP4 && a.kv_scales && nk ? __ldg(a.kv_scales + 1) : 1.f;

    auto process = [&](const At& p, Chunks w) {
        const int t = p.t, h = p.h;
        const Target tg = s_target[t];
        const bool is_q = h < nq;
        if (h < nq + nk) {
            const bool weight = is_q ? n.q_weight != nullptr : n.k_weight != nullptr;
            if (weight || rot_lanes) {  // otherwise the row goes through bit for bit
                float x[V][8];
#pragma unroll
                for (int c = 0; c < V; c++) unpack8(w.v[c], x[c]);
                if (weight) {
                    float ss = 0.f;
#pragma unroll
                    for (int c = 0; c < V; c++)
#pragma unroll
                        for (int e = 0; e < 8; e++) ss = fmaf(x[c][e], x[c][e], ss);
#pragma unroll
                    for (int o = LPR / 2; o; o >>= 1) ss += __shfl_xor_sync(mask, ss, o);
                    const float inv = rsqrtf(fmaf(ss, 1.f / D, n.eps));
#pragma unroll
                    for (int c = 0; c < V; c++) {
                        float wt[8];
                        unpack8(is_q ? qw.v[c] : kw.v[c], wt);
#pragma unroll
                        for (int e = 0; e < 8; e++) x[c][e] = x[c][e] * inv * wt[e];
                    }
                }
                const float2* cs = s_cs + t * DCP_ROPE_MAX_PAIRS;
                if (FP4) {
                    rotate8(x[0], cs, rope.layout, rot_lanes / 2, li, base_lane, mask);
                } else if (turns && half) {
                    const float4* c4 = reinterpret_cast<const float4*>(cs + o0);  // pairs o0 .. o0 + 7
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        const float4 c = c4[e];  // cos, sin, cos, sin
                        turn(x[0][2 * e], x[V - 1][2 * e], c.x, c.y);
                        turn(x[0][2 * e + 1], x[V - 1][2 * e + 1], c.z, c.w);
                    }
                } else if (turns) {
#pragma unroll
                    for (int k = 0; k < V; k++) {
                        const float4* c4 = reinterpret_cast<const float4*>(cs + (k ? o1 : o0) / 2);
#pragma unroll
                        for (int e = 0; e < 2; e++) {
                            const float4 c = c4[e];
                            turn(x[k][4 * e], x[k][4 * e + 1], c.x, c.y);
                            turn(x[k][4 * e + 2], x[k][4 * e + 3], c.z, c.w);
                        }
                    }
                }
#pragma unroll
                for (int c = 0; c < V; c++) w.v[c] = pack8(x[c]);
            }
        }
        if (is_q) {
            if (tg.pg != -3) store(n.q_out + ((i0 + t) * n.hq + h) * (D * 2), w);
            return;
        }
        if (tg.pg < 0) return;
        const bool is_k = h < nq + nk;
        const int g = h - nq - (is_k ? 0 : nk);
        uint8_t* pool = is_k ? a.k_pages : a.v_pages;
        if (FP4)
            store_fp4x8(a, pool, tg.pg, g, tg.off, li, w.v[0], is_k ? fk : fv, mask);
        else
            store(pool + (((int64_t)tg.pg * a.hkv + g) * a.page_size + tg.off) * (D * 2), w);
    };
    while (p0.t < nt) {
        const Chunks c0 = w0;
        const At a0 = p0;
        next(p0);
        if (p0.t < nt) w0 = load(source(p0));
        process(a0, c0);
    }
}

// MLA: CTA (token, block of kMlaHeads query heads); the first block also writes the
// token's latent row.  Only the last 64 of a query's 576 are rotated; the 512
// before them are copied, or left alone when q_out is q.
__global__ void __launch_bounds__(kThreads) norm_rope_mla_kernel(const NormRopeArgs n,
                                                                 const __grid_constant__ dcp_rope rope) {
    constexpr int DK = 576, NOPE = 512, ROT = 64;
    __shared__ __align__(16) float2 s_cs[ROT / 2];
    const AppendArgs& a = n.a;
    const int64_t i = blockIdx.x;
    const int h0 = blockIdx.y * kMlaHeads;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int p = a.pos[i];
    if (p < 0) return;  // padding
    const int nh = n.q ? min(kMlaHeads, n.hq - h0) : 0;
    const uint8_t* q = n.q + (i * n.q_stride + (int64_t)h0 * DK) * 2;
    uint8_t* qo = n.q_out + (i * n.hq + h0) * (int64_t)DK * 2;
    if (n.rotate && threadIdx.x < ROT / 2) s_cs[threadIdx.x] = cos_sin(rope, p, threadIdx.x);
    if (nh > 0 && qo != q) {
        for (int k = threadIdx.x; k < nh * (NOPE / 8); k += kThreads) {
            const int h = k / (NOPE / 8), c = k % (NOPE / 8);
            reinterpret_cast<uint4*>(qo + (int64_t)h * DK * 2)[c] =
                __ldg(reinterpret_cast<const uint4*>(q + (int64_t)h * DK * 2) + c);
        }
    }
    __syncthreads();
    // rotated part of the queries: 8 lanes a head
    {
        const int h = threadIdx.x / 8, li = threadIdx.x % 8;
        const uint32_t mask = 0xffu << (lane & ~7);
        if (h < nh) {
            const uint4 w = *(reinterpret_cast<const uint4*>(q + ((int64_t)h * DK + NOPE) * 2) + li);
            uint4 y = w;
            if (n.rotate) {
                float x[8];
                unpack8(w, x);
                rotate8(x, s_cs, rope.layout, ROT / 16, li, lane & ~7, mask);
                y = pack8(x);
            }
            *(reinterpret_cast<uint4*>(qo + ((int64_t)h * DK + NOPE) * 2) + li) = y;
        }
    }
    // the latent row: the last warp of the first block, 8 elements a lane and step
    // (two steps of the normed part, one of the rotated part in lanes 0..7)
    if (blockIdx.y != 0 || warp != kThreads / 32 - 1 || !a.k_new) return;
    int off = 0;
    const int pg = append_target(a, i, &off);
    if (pg < 0) {
        if (pg == -1 && lane == 0) record_status(a.status, DCP_ERR_UNALLOCATED_PAGE);
        return;
    }
    const uint4* src = reinterpret_cast<const uint4*>(a.k_new + i * n.k_stride * 2);
    uint4 y[3];
    y[0] = __ldg(src + lane);
    y[1] = __ldg(src + 32 + lane);
    y[2] = lane < 8 ? __ldg(src + 64 + lane) : make_uint4(0, 0, 0, 0);
    if (n.k_weight) {
        float x[2][8], ss = 0.f;
#pragma unroll
        for (int c = 0; c < 2; c++) {
            unpack8(y[c], x[c]);
#pragma unroll
            for (int e = 0; e < 8; e++) ss = fmaf(x[c][e], x[c][e], ss);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float inv = rsqrtf(ss * (1.f / NOPE) + n.eps);
#pragma unroll
        for (int c = 0; c < 2; c++) {
            float wt[8];
            unpack8(__ldg(reinterpret_cast<const uint4*>(n.k_weight) + c * 32 + lane), wt);
#pragma unroll
            for (int e = 0; e < 8; e++) x[c][e] = x[c][e] * inv * wt[e];
            y[c] = pack8(x[c]);
        }
    }
    if (n.rotate) {
        float x[8];
        unpack8(y[2], x);
        rotate8(x, s_cs, rope.layout, ROT / 16, lane, 0, 0xffffffffu);
        if (lane < 8) y[2] = pack8(x);
    }
    const int64_t row = (int64_t)pg * a.page_size + off;
    if (a.dtype == DCP_BF16) {
        uint4* dst = reinterpret_cast<uint4*>(a.k_pages + row * DK * 2);
        dst[lane] = y[0];
        dst[32 + lane] = y[1];
        if (lane < 8) dst[64 + lane] = y[2];
        return;
    }
    // fp8: scale = amax / 448 over the rounded row, as the append
    float x[3][8], amax = 0.f;
#pragma unroll
    for (int c = 0; c < 3; c++) {
        unpack8(y[c], x[c]);
#pragma unroll
        for (int e = 0; e < 8; e++) amax = fmaxf(amax, fabsf(x[c][e]));
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const float scale = amax == 0.f ? 1.f : __fdiv_rn(amax, 448.f);
    const uint32_t any = amax == 0.f ? 0u : ~0u;  // zero codes in a row of zeros, also of the -0 that a rotation leaves
    uint2* dst = reinterpret_cast<uint2*>(a.k_pages + row * DK);
    auto codes = [&](const float* v) {
        const uint2 w = fp8_quantise8(v, scale);
        return make_uint2(w.x & any, w.y & any);
    };
    dst[lane] = codes(x[0]);
    dst[32 + lane] = codes(x[1]);
    if (lane < 8) dst[64 + lane] = codes(x[2]);
    if (lane == 0) a.kv_scales[row] = scale;
}

}  // namespace

cudaError_t launch_norm_rope_append(const AppendArgs& a, const dcp_rope* rope, const void* q, int64_t q_stride,
                                    int64_t k_stride, int64_t v_stride, const void* q_weight, const void* k_weight,
                                    float eps, void* q_out, int hq, int num_sms, cudaStream_t s) {
    if (a.n_tok == 0) return cudaSuccess;
    NormRopeArgs n;
    n.a = a;
    n.q = static_cast<const uint8_t*>(q);
    n.q_stride = q_stride;
    n.k_stride = k_stride;
    n.v_stride = v_stride;
    n.q_weight = static_cast<const uint8_t*>(q_weight);
    n.k_weight = static_cast<const uint8_t*>(k_weight);
    n.eps = eps;
    n.q_out = static_cast<uint8_t*>(q_out);
    n.hq = hq;
    n.rotate = rope ? 1 : 0;
    n.tokens = 1;
    dcp_rope r = {};
    if (rope) r = *rope;
    if (a.kind == DCP_MLA) {
        const dim3 grid((unsigned)a.n_tok, q ? (unsigned)((hq + kMlaHeads - 1) / kMlaHeads) : 1u);
        norm_rope_mla_kernel<<<grid, kThreads, 0, s>>>(n, r);
        return cudaGetLastError();
    }
    // tokens per CTA: what comes before a CTA's first row (positions, tables, angles)
    // is shared by all its tokens, as long as eight CTAs for each SM remain
    while (n.tokens < kMaxTokens && a.n_tok / (2 * n.tokens) >= 8 * num_sms) n.tokens *= 2;
    const int64_t blocks = (a.n_tok + n.tokens - 1) / n.tokens;
    // queries alone go through the bf16 kernel whatever the cache
    const bool fp4 = a.dtype == DCP_FP4_E2M1 && a.k_new;
    if (a.dk == 64)
        (fp4 ? norm_rope_gqa_kernel<64, true> : norm_rope_gqa_kernel<64, false>)<<<(unsigned)blocks, kThreads, 0, s>>>(n, r);
    else
        (fp4 ? norm_rope_gqa_kernel<128, true> : norm_rope_gqa_kernel<128, false>)<<<(unsigned)blocks, kThreads, 0, s>>>(n, r);
    return cudaGetLastError();
}

}  // namespace dcp
