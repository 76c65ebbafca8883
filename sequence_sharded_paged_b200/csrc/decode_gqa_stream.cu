// decode_gqa_stream.cu -- GQA decode attention in which every warp streams its own
// part of the cache: over 4-bit caches (all decode calls) and under a sliding
// window with sinks (bf16 and 4-bit caches), for any group size and query length.
//
// "Efficient Decode Context Parallelism with vLLM for Long Context Workloads",
// section 4.1 ("Compute" on the local KV slice, partial output + LSE, and their
// LSE-weighted sum) and section 5.4 (each KV head broadcast to its query heads).
//
// Mathematics: s = scale q.k, p = exp(s - m), l = sum p, O = sum p v / l over the
// visible positions, in one pass with a running reference m.  m moves only when a
// row's maximum grows by more than 2^8 (lazy rescale).
//
// Work: a segment is (request, KV head, tile of 16 query rows) -- of one shard when
// partials are asked for, of all shards otherwise.  Its visible local positions are
// read in groups of 16 tokens; a group never leaves its page.  A team of 1, 2 or 4
// warps takes whole segments (short windows: one launch, nothing to merge), or an
// equal share of the flat list of all groups, whatever the lengths; the two ends of
// a share may then be parts of a segment, whose (O, LSE) go to the workspace and are
// summed by combine_kernel.
//
// Tile: 16 query rows x 16 tokens on mma.sync m16n8k16 with fp32 accumulators.
//
// bf16 caches.  Bound by HBM.  A group of K and of V arrives by one TMA copy each
// (box: 16 tokens of a head, 128-byte swizzle) in a queue of 3 groups (6 for 64
// dimensions) of the warp's own, with an mbarrier for each place and no other wait;
// ldmatrix hands out K's operands, ldmatrix.trans V's.  (Copies by each thread of its
// own bytes stayed at 4.1 TB/s however deep the queue; a barrier for K and one for V,
// with K a group ahead: 220 us instead of 195 us.)  Q K^T is exact products, P has
// three bf16 terms (24 bits), and O is summed by additions that round.
//
// 4-bit caches.  Bound by the latency of the arithmetic: codes to fp16, times their scale,
// and 16 + 32 + 2 matrix instructions (16 + 16 + 1 up to 8 rows) a group.  A loop of such
// instructions alone takes a scheduler 10.75 cycles each, 192 us for the first case below;
// but with two warps a scheduler, all that the registers allow, neither the tensor pipe
// (42% busy) nor the issue slots (43%) are full, and waits of a fixed length come first among
// the stalls.  The dimensions of a k-step and the tokens of a group may be
// permuted freely (Q, and P from S, are permuted alike), so each thread takes 16 or 8
// CONSECUTIVE bytes of a row as its operands:
//   Q K^T  thread (n = lane / 4, c = lane % 4), token tile t: token
//          4 (n >> 1) + 2 t + (n & 1), dimensions D/4 c .. + D/4 - 1;
//   P V    thread (n, c): tokens 4 c .. 4 c + 3, dimensions n D/8 .. + D/8 - 1 (n-tile
//          j is dimension n D/8 + j); S leaves tokens 4 c .. 4 c + 3 in thread c.
// So no data is exchanged between threads: every thread copies (cp.async) exactly the
// bytes it will use into its own places of the queue, and waits for its own copies
// only.  Tokens that no row may see are filled with zeros by the copy itself, so that
// stale or non-finite bytes in masked places never meet a product.  Code times scale
// has 6 significant bits and lies within 2^-10 .. 2688, so it is exact in fp16; q is
// scaled by a power of two into fp16's range; P has two fp16 terms, with the reference
// 2^7 below the maximum so that small weights stay above fp16's smallest step.
//
// With at most 8 query rows two terms of P share one instruction (rows 0..7 and 8..15
// of the tile).  The scores of the next groups are computed beside P V of these, two
// independent streams of instructions; what hides latency is that and a second block
// on the SM, both out of registers (three blocks of 168 registers spill and are no
// faster with 8 rows, slower with 16).
//
// Measured, K and V bytes / time, of a copy's 6.56 TB/s:
//   bf16   128 requests, 64 / 4 heads of 128, window 4096: 1081 MB, 184 us, 5.9 TB/s, 90%
//          1 request, window 65536: 134 MB, 39 us (20 us of it streaming, 9 us until the
//          first bytes, the rest the sums of 300 parts and two launches)
//          1 request, window 128, 8 / 2 heads of 64: 8 us, latency
//   4-bit  24 requests of 32k-128k, 64 / 4 heads: 906 MB, 297 us, 3.0 TB/s
//          48 requests of 1-14k, 64 / 8 heads: 85 MB, 46 us (8 rows; half of the segments
//          are of 5 groups and cost as much as 48)
//          64 requests, 4 tokens each, window 1021: 68 MB, 48.5 us (512 segments, two warps each)
//          2 requests of 400, 8 / 2 heads of 64: 8 us, latency
#include "common.cuh"
#include "finish.cuh"
#include "kernels.h"
#include "stream.cuh"

namespace dcp {

namespace {

constexpr int kWarps = 4;
constexpr int kWarpsPerSm = 8;  // by registers and by the queues' sizes
constexpr int kAcc = 17 * 32;  // float4 of a warp's O in memory, and what belongs to it
constexpr int kDescs = 64;   // group descriptors per warp (two batches of 32)

// Launch constants of one cache type and head size.
//   bf16: K and V of 16 tokens, each [D/64 halves][16 tokens][128 B] with 128-byte swizzle
//   4-bit, a lane and group: K 2 tiles x D/8 B, V 4 tokens x D/16 B, scales (D/64 + 1) words
template <bool FP4, int D>
struct Lane {
    static constexpr int kK = FP4 ? 2 * D / 8 : 2 * (D / 32) * 16;  // bytes of K
    static constexpr int kV = FP4 ? 4 * D / 16 : 4 * (D / 64) * 16;
    static constexpr int kS = FP4 ? (D / 64 + 1) * 4 : 0;
    static constexpr int kStage = 32 * (kK + kV + kS);
    // Groups that one softmax step takes.  4-bit: two, since the work for each byte is
    // what bounds it and two groups share the step's votes and hide each other's
    // latencies; bf16: one, since the bytes in flight are what counts.
    static constexpr int kStep = FP4 ? 2 : 1;
    // (4-bit: 5 steps of 128 dimensions measured 303 us against 300 for 3, 24 requests of 32k-128k tokens)
    static constexpr int kSteps = FP4 ? (D == 128 ? 3 : 4) : (D == 128 ? 3 : 6);  // steps in the queue
    static constexpr int kStages = kStep * kSteps;
};

// copies of this thread's own bytes; a masked copy that is not live writes zeros
template <bool MASK>
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool live) {
    if (MASK)
        asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                     "r"(live ? 16 : 0)
                     : "memory");
    else
        asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
template <bool MASK>
__device__ __forceinline__ void cp8(uint32_t dst, const void* src, bool live) {
    if (MASK)
        asm volatile("cp.async.ca.shared.global.L2::128B [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(live ? 8 : 0)
                     : "memory");
    else
        asm volatile("cp.async.ca.shared.global.L2::128B [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
template <bool MASK>
__device__ __forceinline__ void cp4(uint32_t dst, const void* src, bool live) {
    if (MASK)
        asm volatile("cp.async.ca.shared.global.L2::128B [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(live ? 4 : 0)
                     : "memory");
    else
        asm volatile("cp.async.ca.shared.global.L2::128B [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// orders this thread's writes to shared memory before later copies by the copy engine
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// four 8 x 8 matrices of 16-bit values, each lane giving one row's address; trans: transposed
template <bool TRANS>
__device__ __forceinline__ void ldmatrix4(const void* row, uint32_t& r0, uint32_t& r1, uint32_t& r2, uint32_t& r3) {
    if (TRANS)
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
                     : "r"(smem_u32(row))
                     : "memory");
    else
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
                     : "r"(smem_u32(row))
                     : "memory");
}

// d = a b + c
template <bool FP4>
__device__ __forceinline__ void mma(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1, const float* c) {
    if (FP4)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%10, %11, %12, %13};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%10, %11, %12, %13};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}
template <bool FP4>
__device__ __forceinline__ void mma(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    mma<FP4>(d, a0, a1, a2, a3, b0, b1, d);
}

// x ~ hi + lo (4-bit: fp16) or hi + lo + last (bf16), two values: 22 and 24 bits
template <bool FP4>
__device__ __forceinline__ void split(float x0, float x1, uint32_t& hi, uint32_t& lo, uint32_t& last) {
    if (FP4) {
        const __half2 h = __floats2half2_rn(x0, x1);
        const float2 f = __half22float2(h);
        const __half2 l = __floats2half2_rn(x0 - f.x, x1 - f.y);
        hi = *reinterpret_cast<const uint32_t*>(&h);
        lo = *reinterpret_cast<const uint32_t*>(&l);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x0, x1);
        const float2 f = __bfloat1622float2(h);
        x0 -= f.x, x1 -= f.y;
        const __nv_bfloat162 l = __floats2bfloat162_rn(x0, x1);
        const float2 g = __bfloat1622float2(l);
        const __nv_bfloat162 m = __floats2bfloat162_rn(x0 - g.x, x1 - g.y);
        hi = *reinterpret_cast<const uint32_t*>(&h);
        lo = *reinterpret_cast<const uint32_t*>(&l);
        last = *reinterpret_cast<const uint32_t*>(&m);
    }
}

// Everything a warp keeps for the segment it works on.
template <bool FP4, int D, bool HALF>
struct Warp {
    static constexpr int KS = D / 16;  // k-steps of Q K^T
    static constexpr int NT = D / 8;   // n-tiles of P V
    static constexpr int H = HALF ? 1 : 2;  // rows of this thread: qr (and qr + 8)
    using C = Lane<FP4, D>;
    static constexpr float kBias = FP4 ? 7.f : 0.f;
    // terms of P, each the A operands of one group [row half + 2 * tile]; with HALF the
    // first instruction takes terms 0 and 1 (in rows 8..15)
    static constexpr int kTerms = FP4 ? 2 : 3;
    using Terms = uint32_t[kTerms][4];
    // independent parts of a score's sum: see scores()
    static constexpr int kChains = FP4 && HALF ? 1 : 2;
    // The instruction cuts its sums off where it should round.  bf16 caches: each product
    // is added to O by an addition that rounds.  4-bit caches have no issue slots and
    // registers to spare for that: `ol`, the sum of P by the same instruction, cancels
    // what is common to all dimensions, and with two products a group (more than 8 rows)
    // O also goes to memory, added there with rounding, after kFlush groups.  24 requests
    // of 32k-128k tokens, relative error of O: 6.3e-6 without that, 4.9e-6 with it (fp32
    // throughout: 4.1e-6).  An addition that rounds for each product: 379 us against 299.
    static constexpr bool kExact = !FP4;
    static constexpr int kFlush = kExact || HALF ? 0 : 256;
    static constexpr int E = kExact ? 2 * H : 4;  // accumulators of an n-tile; HALF: rows 8..15 are the low terms'
    static constexpr uint32_t kOnes = FP4 ? 0x3c003c00u : 0x3f803f80u;

    uint32_t q[KS][HALF ? 2 : 4];
    float o[NT][E];
    float ol[4];  // !kExact: sum of P
    float m[2], l[2], scale[2];
    int at[2];  // positions of rows qr and qr + 8

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int j = 0; j < NT; j++)
#pragma unroll
            for (int e = 0; e < E; e++) o[j][e] = 0.f;
        ol[0] = ol[1] = ol[2] = ol[3] = 0.f;
    }
    __device__ __forceinline__ void reset() {
        clear();
        m[0] = m[1] = -INFINITY;
        l[0] = l[1] = 0.f;
    }

    // the four tokens that thread column c holds of P and V: x[t][e] is token_of(c, 2 t + e)
    __device__ __forceinline__ static int token_of(int c, int i) { return FP4 ? 4 * c + i : 2 * c + (i & 1) + 8 * (i >> 1); }

    // Masked scores are -inf before they are scaled, and -inf times 0 is no weight but NaN.
    // A scale of 0 (the caller's, or a product that 32 bits take for 0) is 2^-149 instead: it
    // brings every finite score, below 2^128, under 2^-21, and leaves -inf what it is.
    __device__ __forceinline__ static float row_scale(float s) { return s == 0.f ? __uint_as_float(1u) : s; }

    // Q fragments of rows qr (and qr + 8) of tile `tile` of KV head g
    __device__ __forceinline__ void load_q(const StreamArgs& a, int b, int g, int tile, int L, float kf) {
        const int lane = threadIdx.x & 31, qr = lane >> 2, c = lane & 3;
#pragma unroll
        for (int h = 0; h < 2; h++) {
            const int r = tile * kRows + qr + 8 * h;
            const bool live = r < a.rows && !(HALF && h);
            const int j = live ? r / a.group : 0, hh = live ? r - j * a.group : 0;
            at[h] = live ? L - a.q_len + j : INT_MIN / 2;
            scale[h] = row_scale(fabsf(a.scale_log2));
            if (HALF && h) continue;
            const uint2* src = reinterpret_cast<const uint2*>(
                a.q + (((int64_t)b * a.q_len + j) * a.hq + g * a.group + hh) * D);  // 4 dimensions each
            uint2 w[KS];
#pragma unroll
            for (int s = 0; s < KS; s++) {
                w[s] = make_uint2(0, 0);
                if (live && FP4) w[s] = __ldg(src + (D / 4 * c) / 4 + s);
                if (live && !FP4) {
                    const uint32_t* two = reinterpret_cast<const uint32_t*>(src) + 8 * s + c;
                    w[s] = make_uint2(__ldg(two), __ldg(two + 4));
                }
                if (a.scale_log2 < 0.f) {  // the sign of the scale goes into q: scale[] >= 0
                    w[s].x ^= 0x80008000u;
                    w[s].y ^= 0x80008000u;
                }
            }
            if (FP4) {
                // a power of two brings the row's largest magnitude into [1, 2)
                float amax = 0.f;
#pragma unroll
                for (int s = 0; s < KS; s++)
                    amax = fmaxf(fmaxf(amax, fmaxf(fabsf(bf16_lo(w[s].x)), fabsf(bf16_hi(w[s].x)))),
                                 fmaxf(fabsf(bf16_lo(w[s].y)), fabsf(bf16_hi(w[s].y))));
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
                const float2 pw = row_power(amax);
                const float f = pw.x;
                scale[h] = row_scale(fabsf(a.scale_log2) * kf * pw.y);
#pragma unroll
                for (int s = 0; s < KS; s++) {
                    const __half2 x = __floats2half2_rn(bf16_lo(w[s].x) * f, bf16_hi(w[s].x) * f);
                    const __half2 y = __floats2half2_rn(bf16_lo(w[s].y) * f, bf16_hi(w[s].y) * f);
                    w[s].x = *reinterpret_cast<const uint32_t*>(&x);
                    w[s].y = *reinterpret_cast<const uint32_t*>(&y);
                }
            }
#pragma unroll
            for (int s = 0; s < KS; s++) {
                if (HALF) {
                    q[s][0] = w[s].x;
                    q[s][1] = w[s].y;
                } else {
                    q[s][h] = w[s].x;
                    q[s][h + 2] = w[s].y;
                }
            }
        }
    }

    // This thread's places in the pools (4-bit).
    struct Places {
        const uint8_t *k, *v, *ks, *vs;
        int page;  // offset of the scales in a block, in rows of codes minus one
        __device__ __forceinline__ explicit Places(const StreamArgs& a) {
            const int lane = threadIdx.x & 31, n = lane >> 2, c = lane & 3;
            const int P = a.page_size;
            k = a.k_pages + (4 * (n >> 1) + (n & 1)) * (D / 2) + c * (D / 8);
            v = a.v_pages + 4 * c * (D / 2) + n * (D / 16);
            ks = a.k_pages + P * (D / 2) + (c * (D / 64)) * P + 4 * (n >> 1);
            vs = a.v_pages + P * (D / 2) + (n * D / 128) * P + 4 * c;
            page = P;
        }
    };

    // 4-bit: start the copies of group d, which not every row sees all of: a token is
    // copied if any query token sees it, and is zeros otherwise.  Its scales come in
    // words of four tokens; those of tokens that are not copied are cleared by the
    // reader (`keep`).
    __device__ __forceinline__ static void copy_masked(const Places& from, const Desc& d, uint32_t slot) {
        bool live[6];  // K tiles' tokens, V's four tokens
        const int lane = threadIdx.x & 31, n = lane >> 2, c = lane & 3;
        const uint32_t k = d.live >> (4 * (n >> 1) + (n & 1)), v = d.live >> (4 * c);
        live[0] = k & 1, live[1] = k & 4;
        live[2] = v & 1, live[3] = v & 2, live[4] = v & 4, live[5] = v & 8;
        Desc at = d;
        if (d.off < 0) at.off = at.sub = 0;  // no page: zeros, and block 0's scales (not used)
        copy<true>(from, at, live, slot);
    }

    template <bool MASK>
    __device__ __forceinline__ static void copy(const Places& from, const Desc& d, const bool* live, uint32_t slot) {
        const int lane = threadIdx.x & 31;
        const int P = from.page;
        // d.off is the group's first row of codes; its scales lie this much less than a row a token further
        const int64_t so = d.off - d.sub * (D / 2 - 1);
        const uint8_t *k = from.k + d.off, *v = from.v + d.off, *ks = from.ks + so, *vs = from.vs + so;
        const uint32_t ds = slot + (C::kK + C::kV) * 32 + lane * 4;
        if (D == 128) {
            cp16<MASK>(slot + lane * 16, k, live[0]);
            cp16<MASK>(slot + 512 + lane * 16, k + 2 * (D / 2), live[1]);
#pragma unroll
            for (int e = 0; e < 4; e++)
                cp8<MASK>(slot + 1024 + (e >> 1) * 512 + lane * 16 + (e & 1) * 8, v + e * (D / 2), live[2 + e]);
            cp4<false>(ds, ks, true);
            cp4<false>(ds + 128, ks + P, true);
            cp4<false>(ds + 256, vs, true);
        } else {
            cp8<MASK>(slot + lane * 16, k, live[0]);
            cp8<MASK>(slot + lane * 16 + 8, k + 2 * (D / 2), live[1]);
#pragma unroll
            for (int e = 0; e < 4; e++) cp4<MASK>(slot + 512 + lane * 16 + e * 4, v + e * (D / 2), live[2 + e]);
            cp4<false>(ds, ks, true);
            cp4<false>(ds + 128, vs, true);
        }
    }

    // bf16: byte offset of chunk `chunk` (8 dimensions) of a token's K or V row in a stage, as the
    // copies' 128-byte swizzle places it
    __device__ __forceinline__ static int row_place(int token, int chunk) {
        return (chunk >> 3) * 2048 + token * 128 + (((chunk ^ token) & 7) << 4);
    }

    // V operands of n-tiles 8 w .. 8 w + 7: b[j][h] tokens token_of(c, 2h), token_of(c, 2h + 1).
    // keep: bytes of the four tokens' scales that count
    __device__ __forceinline__ static void load_v(const uint8_t* slot, int w, uint32_t keep, uint32_t (*b)[2]) {
        const int lane = threadIdx.x & 31;
        if (!FP4) {
            // matrices: tokens 0..7 and 8..15 of chunk j, the same of chunk j + 1
#pragma unroll
            for (int j = 0; j < 8; j += 2)
                ldmatrix4<true>(slot + C::kK * 32 + row_place(lane & 15, 8 * w + j + (lane >> 4)), b[j][0], b[j][1],
                                b[j + 1][0], b[j + 1][1]);
        } else {
            uint32_t v[4];
#pragma unroll
            for (int e = 0; e < 4; e++)
                v[e] = D == 128 ? *reinterpret_cast<const uint32_t*>(slot + 1024 + (e >> 1) * 512 + lane * 16 +
                                                                     (e & 1) * 8 + w * 4)
                                : *reinterpret_cast<const uint32_t*>(slot + 512 + lane * 16 + e * 4);
            const uint32_t sw =
                keep & *reinterpret_cast<const uint32_t*>(slot + (C::kK + C::kV) * 32 + (D / 64) * 128 + lane * 4);
#pragma unroll
            for (int h = 0; h < 2; h++) {
                // low half of a byte: token 4c + 2h, high half: the next token, same dimension
                const uint32_t x = v[2 * h], y = v[2 * h + 1];
                const uint32_t s = e4m3x2(h ? sw >> 16 : sw & 0xffffu);
                uint32_t even[4], odd[4];
                e2m1x8((x & 0x0f0f0f0fu) | ((y << 4) & 0xf0f0f0f0u), even);
                e2m1x8(((x >> 4) & 0x0f0f0f0fu) | (y & 0xf0f0f0f0u), odd);
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    b[2 * k][h] = mul2(even[k], s);
                    b[2 * k + 1][h] = mul2(odd[k], s);
                }
            }
        }
    }

    // Scores of one group: x[t][e], e = 0, 1: row qr, token_of(c, 2t + e); e = 2, 3: row qr + 8
    // The instruction cuts its sums off where it should round, so each tile's sum is taken
    // in kChains independent parts, added at the end with rounding.
    __device__ __forceinline__ void scores(const uint8_t* slot, float (*x)[4]) {
        const int lane = threadIdx.x & 31, n = lane >> 2;
        float y[2][kChains][4];
        if (!FP4) {
            // matrices: chunks 2 s and 2 s + 1 of tokens 0..7, the same of tokens 8..15
#pragma unroll
            for (int s = 0; s < KS; s++) {
                uint32_t k[2][2];
                ldmatrix4<false>(slot + row_place((lane & 7) + (lane >> 4) * 8, 2 * s + (lane >> 3 & 1)), k[0][0], k[0][1],
                                 k[1][0], k[1][1]);
#pragma unroll
                for (int t = 0; t < 2; t++) qk(y[t], s, k[t][0], k[t][1]);
            }
        } else {
#pragma unroll
            for (int t = 0; t < 2; t++) {
                uint32_t kw[D / 32];
                if (D == 128) {
                    const uint4 k = *reinterpret_cast<const uint4*>(slot + t * 512 + lane * 16);
                    kw[0] = k.x, kw[1] = k.y, kw[D / 32 - 2] = k.z, kw[D / 32 - 1] = k.w;
                } else {
                    const uint2 k = *reinterpret_cast<const uint2*>(slot + lane * 16 + t * 8);
                    kw[0] = k.x, kw[1] = k.y;
                }
                // this token's byte of the scale words, twice
                const uint32_t sel = (uint32_t)(2 * t + (n & 1)) * 0x11u;
#pragma unroll
                for (int w = 0; w < D / 32; w++) {
                    const uint32_t sw = *reinterpret_cast<const uint32_t*>(slot + (C::kK + C::kV) * 32 +
                                                                           (w >> 1) * 128 + lane * 4);
                    const uint32_t s = e4m3x2(__byte_perm(sw, 0, sel));
                    uint32_t h[4];
                    e2m1x8(kw[w], h);
                    qk(y[t], 2 * w, mul2(h[0], s), mul2(h[1], s));
                    qk(y[t], 2 * w + 1, mul2(h[2], s), mul2(h[3], s));
                }
            }
        }
#pragma unroll
        for (int t = 0; t < 2; t++)
#pragma unroll
            for (int e = 0; e < 2 * H; e++) {
                x[t][e] = y[t][0][e];
#pragma unroll
                for (int i = 1; i < kChains; i++) x[t][e] += y[t][i][e];
            }
    }

    static constexpr int G = C::kStep;

    // Scores of a step whose groups lie in consecutive slots.
    __device__ __forceinline__ void step_scores(const uint8_t* at, float (*x)[4]) {
#pragma unroll
        for (int g = 0; g < G; g++) scores(at + g * C::kStage, x + 2 * g);
    }

    // Masks of a step that not every row sees all of: scores of what a row does not
    // see become -inf; of tokens that no row sees, keep[g] clears the scales (4-bit) and
    // the values are set to zero in the stage (bf16: each thread's own chunks).
    __device__ __forceinline__ void mask(const StreamArgs& a, const Desc* d, uint8_t* stage, float (*x)[4],
                                         uint32_t* keep) {
        const int c = threadIdx.x & 3, n = (threadIdx.x & 31) >> 2;
#pragma unroll
        for (int g = 0; g < G; g++) {
            keep[g] = 0;
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const bool live = d[g].live >> token_of(c, e) & 1;
                if (live) {
                    keep[g] |= 0xffu << (8 * e);
                } else if (!FP4) {
#pragma unroll
                    for (int w = 0; w < NT / 8; w++)
                        *reinterpret_cast<uint4*>(stage + C::kK * 32 + row_place(token_of(c, e), 8 * w + n)) =
                            make_uint4(0u, 0u, 0u, 0u);
                }
                bool row[2] = {live, live};
                if (a.q_len > 1 && live) {  // the rows' query tokens see different ends
                    const int64_t p = position_in(a, d[g].p0, token_of(c, e));
                    row[0] = sees(a, p, at[0]);
                    row[1] = sees(a, p, at[1]);
                }
#pragma unroll
                for (int h = 0; h < H; h++)
                    if (!row[h]) x[2 * g + (e >> 1)][2 * h + (e & 1)] = -INFINITY;
            }
        }
        if (!FP4) {
            fence_async();  // before the stage's next copy
            __syncwarp();
        }
    }

    // One softmax step: x becomes the terms of P.
    __device__ __forceinline__ void softmax(const float (*x)[4], Terms* p) {
        float mx[H];
        bool grow = false;
#pragma unroll
        for (int h = 0; h < H; h++) {
            mx[h] = -INFINITY;
#pragma unroll
            for (int t = 0; t < 2 * G; t++) mx[h] = fmaxf(mx[h], fmaxf(x[t][2 * h], x[t][2 * h + 1]));
            mx[h] *= scale[h];
            grow |= mx[h] > m[h] + (kLazy + kBias);
        }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
            for (int h = 0; h < H; h++) {
                float t = mx[h];
                t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 1));
                t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 2));
                if (t > m[h] + (kLazy + kBias)) {
                    const float mn = t - kBias;
                    const float f = m[h] == -INFINITY ? 0.f : fast_exp2(m[h] - mn);
                    m[h] = mn;
                    l[h] *= f;
                    rescale(h, f);
                }
            }
        }
#pragma unroll
        for (int h = 0; h < H; h++) {
            const float ref = m[h] == -INFINITY ? 0.f : m[h];
            float sum = 0.f;
#pragma unroll
            for (int t = 0; t < 2 * G; t++) {
                const float p0 = fast_exp2(fmaf(x[t][2 * h], scale[h], -ref));
                const float p1 = fast_exp2(fmaf(x[t][2 * h + 1], scale[h], -ref));
                sum += p0 + p1;
                const int i = h + 2 * (t & 1);
                split<FP4>(p0, p1, p[t >> 1][0][i], p[t >> 1][1][i], p[t >> 1][kTerms - 1][i]);
            }
            l[h] += sum;
        }
        if (HALF) {
#pragma unroll
            for (int g = 0; g < G; g++) {
                p[g][0][1] = p[g][1][0];
                p[g][0][3] = p[g][1][2];
                if (!FP4) p[g][kTerms - 1][1] = p[g][kTerms - 1][3] = 0u;
            }
        }
    }

    __device__ __forceinline__ static void mul(float* d, const uint32_t* p, uint32_t b0, uint32_t b1) {
        mma<FP4>(d, p[0], p[1], p[2], p[3], b0, b1);
    }
    __device__ __forceinline__ static void first(float* d, const Terms& p, uint32_t b0, uint32_t b1) {
        const float zero[4] = {0.f, 0.f, 0.f, 0.f};
        mma<FP4>(d, p[0][0], p[0][1], p[0][2], p[0][3], b0, b1, zero);
    }
    // o += t; with HALF rows 8..15 of t belong to rows 0..7
    __device__ __forceinline__ static void add(float* o, const float* t) {
#pragma unroll
        for (int e = 0; e < 4; e++) o[e % E] += t[e];
    }

    // O += P V
    __device__ __forceinline__ void values(const uint8_t* at, const uint32_t* keep, const Terms* p) {
#pragma unroll
        for (int g = 0; g < G; g++) {
#pragma unroll
            for (int w = 0; w < NT / 8; w++) {
                uint32_t b[8][2];
                load_v(at + g * C::kStage, w, keep[g], b);
                if (!kExact) {
#pragma unroll
                    for (int i = 0; i < (HALF ? 1 : kTerms); i++)
#pragma unroll
                        for (int j = 0; j < 8; j++) mul(o[8 * w + j], p[g][i], b[j][0], b[j][1]);
                    continue;
                }
                constexpr int kAhead = 4;  // products in flight
#pragma unroll
                for (int j0 = 0; j0 < 8; j0 += kAhead) {
                    float t[kAhead][4];
#pragma unroll
                    for (int j = 0; j < kAhead; j++) first(t[j], p[g], b[j0 + j][0], b[j0 + j][1]);
#pragma unroll
                    for (int i = HALF ? 2 : 1; i < kTerms; i++)
#pragma unroll
                        for (int j = 0; j < kAhead; j++) mul(t[j], p[g][i], b[j0 + j][0], b[j0 + j][1]);
#pragma unroll
                    for (int j = 0; j < kAhead; j++) add(o[8 * w + j0 + j], t[j]);
                }
            }
            if (!kExact) {
#pragma unroll
                for (int i = 0; i < (HALF ? 1 : kTerms); i++) mul(ol, p[g][i], kOnes, kOnes);
            }
        }
    }

    __device__ __forceinline__ void rescale(int h, float f) {
#pragma unroll
        for (int j = 0; j < NT; j++) {
            o[j][2 * h] *= f;
            o[j][2 * h + 1] *= f;
            if (HALF && E == 4) {
                o[j][E - 2] *= f;
                o[j][E - 1] *= f;
            }
        }
        ol[2 * h] *= f;
        ol[2 * h + 1] *= f;
        if (HALF) {
            ol[2] *= f;
            ol[3] *= f;
        }
    }

    __device__ __forceinline__ void qk(float (*y)[4], int s, uint32_t b0, uint32_t b1) {
        const float zero[4] = {0.f, 0.f, 0.f, 0.f};
        float* d = y[s % kChains];
        const float* c = s < kChains ? zero : d;
        if (HALF)
            mma<FP4>(d, q[s][0], 0u, q[s][1], 0u, b0, b1, c);
        else
            mma<FP4>(d, q[s][0], q[s][1], q[s][HALF ? 0 : 2], q[s][HALF ? 0 : 3], b0, b1, c);
    }

    // Does the group hold an infinity or NaN among its values?
    __device__ __forceinline__ static bool poisoned(const uint8_t* slot, uint32_t keep) {
        bool bad = false;
#pragma unroll 1
        for (int w = 0; w < NT / 8; w++) {
            uint32_t b[8][2];
            load_v(slot, w, keep, b);
            constexpr uint32_t e = FP4 ? 0x7c00u : 0x7f80u;
#pragma unroll
            for (int j = 0; j < 8; j++)
#pragma unroll
                for (int h = 0; h < 2; h++)
                    bad |= (b[j][h] & e) == e || ((b[j][h] >> 16) & e) == e;
        }
        return __any_sync(0xffffffffu, bad);
    }

    // O += P V of one group where some rows must not see a non-finite value that
    // others see: row by row, with the values that the row does not see set to zero.
    __device__ __forceinline__ void careful(const StreamArgs& a, const Desc& d, const uint8_t* slot, uint32_t keep,
                                            const Terms& p) {
        const int lane = threadIdx.x & 31, qr = lane >> 2;
#pragma unroll 1
        for (int r = 0; r < (HALF ? 8 : 16); r++) {
            // the position of row r, from a lane that holds it
            const int at_r = __shfl_sync(0xffffffffu, r < 8 ? at[0] : at[1], (r & 7) * 4);
            uint32_t sees_v[2];
#pragma unroll
            for (int h = 0; h < 2; h++) {
                sees_v[h] = 0;
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    const int64_t x = position_in(a, d.p0, token_of(lane & 3, 2 * h + e));
                    if (d.off >= 0 && sees(a, x, at_r)) sees_v[h] |= 0xffffu << (16 * e);
                }
            }
#pragma unroll
            for (int w = 0; w < NT / 8; w++) {
                uint32_t b[8][2];
                load_v(slot, w, keep, b);
#pragma unroll
                for (int j = 0; j < 8; j++) {
                    float t[4];
                    const uint32_t b0 = b[j][0] & sees_v[0], b1 = b[j][1] & sees_v[1];
                    first(t, p, b0, b1);
#pragma unroll
                    for (int i = HALF ? 2 : 1; i < kTerms; i++) mul(t, p[i], b0, b1);
                    if (qr == (r & 7)) {
#pragma unroll
                        for (int e = 0; e < 4; e++)
                            if (HALF || (e >> 1) == (r >> 3)) o[8 * w + j][e % E] += t[e];
                    }
                }
            }
        }
        if (!kExact) {
#pragma unroll
            for (int i = 0; i < (HALF ? 1 : kTerms); i++) mul(ol, p[i], kOnes, kOnes);
        }
    }

    // acc (this lane's own column) = acc + O, at the reference m, and O = 0; the last
    // float4 holds the reference and the sums `ol`.  (!kExact)
    __device__ __forceinline__ void flush(float4* acc, bool first) {
        if (!first) unflush(acc);
#pragma unroll
        for (int j = 0; j < NT; j++) acc[j * 32] = make_float4(o[j][0], o[j][1], o[j][E - 2], o[j][E - 1]);
        acc[kAcc - 32] = make_float4(m[0], m[1], ol[0], ol[2]);
        clear();
    }
    // O = O + acc, at the reference m
    __device__ __forceinline__ void unflush(const float4* acc) {
        const float4 s = acc[kAcc - 32];
        const float f0 = s.x == -INFINITY ? 0.f : fast_exp2(s.x - m[0]);
        const float f1 = HALF ? f0 : s.y == -INFINITY ? 0.f : fast_exp2(s.y - m[1]);
#pragma unroll
        for (int j = 0; j < NT; j++) {
            const float4 x = acc[j * 32];
            o[j][0] = fmaf(f0, x.x, o[j][0]);
            o[j][1] = fmaf(f0, x.y, o[j][1]);
            o[j][E - 2] = fmaf(f1, x.z, o[j][E - 2]);
            o[j][E - 1] = fmaf(f1, x.w, o[j][E - 1]);
        }
        ol[0] = fmaf(f0, s.z, ol[0]);
        ol[2] = fmaf(f1, s.w, ol[2]);
    }

    // O of row qr + 8 h, four dimensions at a time: put(first dimension, values).  bf16: neighbours
    // in c exchange pairs.  Executed by whole warps.
    template <class F>
    __device__ __forceinline__ void each(int h, int c, F put) const {
        if (FP4) {
#pragma unroll
            for (int e = 0; e < 2; e++)
#pragma unroll
                for (int j = 0; j < NT; j += 4)
                    put((2 * c + e) * NT + j, make_float4(o[j][2 * h + e], o[j + 1][2 * h + e], o[j + 2][2 * h + e],
                                                          o[j + 3][2 * h + e]));
        } else {
#pragma unroll
            for (int j = 0; j < NT; j += 2) {
                // the even lane takes n-tile j, the odd one n-tile j + 1
                const bool odd = c & 1;
                const float a0 = odd ? o[j + 1][2 * h] : o[j][2 * h], a1 = odd ? o[j + 1][2 * h + 1] : o[j][2 * h + 1];
                float b0 = odd ? o[j][2 * h] : o[j + 1][2 * h], b1 = odd ? o[j][2 * h + 1] : o[j + 1][2 * h + 1];
                b0 = __shfl_xor_sync(0xffffffffu, b0, 1);
                b1 = __shfl_xor_sync(0xffffffffu, b1, 1);
                put(8 * (j + (c & 1)) + 4 * (c >> 1), odd ? make_float4(b0, b1, a0, a1) : make_float4(a0, a1, b0, b1));
            }
        }
    }

    // what O is to be divided by
    __device__ __forceinline__ float sum(int h) const { return kExact ? l[h] : ol[2 * h]; }

    // After the last group: whole-row sums, the same in the row's four lanes; the low
    // terms' rows are added in.
    __device__ __forceinline__ void close() {
#pragma unroll
        for (int h = 0; h < H; h++) {
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
        }
        if (HALF && E == 4) {
#pragma unroll
            for (int j = 0; j < NT; j++) {
                o[j][0] += o[j][E - 2];
                o[j][1] += o[j][E - 1];
            }
            ol[0] += ol[2];
        }
    }
};

// Eight warps for each SM: what hides latency here is independent work within a warp,
// which takes registers, more than further warps would.
// WARPS: 4, in teams of 1 or 4, or 2, a team that takes whole segments.
template <bool FP4, int D, bool HALF, int WARPS>
__global__ void __launch_bounds__(32 * WARPS, kWarpsPerSm / WARPS) gqa_stream_kernel(const __grid_constant__ StreamArgs a) {
    using W = Warp<FP4, D, HALF>;
    using C = Lane<FP4, D>;
    constexpr int S = C::kStages;
    constexpr int kRing = S * C::kStage;
    constexpr int kMine = HALF ? 8 : kRows;  // rows that can be in use
    constexpr int kPitch = D + 4;  // floats a row of O in the team merge
    static_assert(kRing >= kMine * kPitch * 4, "a warp's queue holds its O");
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    // the swizzle of the bf16 stages goes by the address: 1024-byte alignment
    uint8_t* smem = FP4 ? smem_raw
                        : reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ uint64_t s_full[WARPS][C::kSteps];  // bf16: a stage's copies have landed
    __shared__ volatile int s_abort;
    __shared__ Desc s_desc[WARPS][kDescs];
    __shared__ float s_m[WARPS][16], s_l[WARPS][16], s_ol[WARPS][16];
    __shared__ ShareScratch<WARPS> s_share;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto size = [&]() { return WARPS == 2 ? 2 : a.team; };  // warps of a team
    auto whole = [&]() { return WARPS == 2 || a.whole; };
    const int team = warp / size(), wt = warp - team * size();  // team of the CTA, warp of the team
    const int teams = WARPS / size();
    const int worker = blockIdx.x * teams + team;
    uint8_t* ring = smem + (size_t)warp * kRing;
    const uint32_t ring_u32 = smem_u32(ring);
    Desc* descs = s_desc[warp];
    const int nb = (a.per_shard ? a.shard_hi - a.shard_lo : 1) * a.batch;
    const int per_base = a.hkv * a.tiles;
    const float kf = FP4 && a.factors ? __ldg(a.factors) : 1.f, vf = FP4 && a.factors ? __ldg(a.factors + 1) : 1.f;

    if (!FP4) {
        if (lane == 0) {
            for (int k = 0; k < C::kSteps; k++) mbar_init(&s_full[warp][k], 1);
            fence_barrier_init();
        }
        if (threadIdx.x == 0) {
            s_abort = 0;
            tma_prefetch_desc(&a.map_k);
            tma_prefetch_desc(&a.map_v);
        }
        __syncthreads();
    }
    check_lengths(a);

    // this worker's share: segments [worker, ..) step `workers`, or flat groups [r0, r1); no
    // share below 8 groups a warp, a partial costs about as much as those
    Share sh{0, 0, 0, 0, 0, 0, 0};
    if (!whole()) sh = find_share<WARPS>(a, nb, per_base, teams, team, 8ll * size(), s_share);
    int base = sh.base, sub = sh.sub, x0 = sh.x0;
    const typename W::Places places(a);
    // this lane's column of its warp's O in memory
    auto acc = [&]() { return a.acc + ((int64_t)blockIdx.x * WARPS + (threadIdx.x >> 5)) * kAcc + (threadIdx.x & 31); };
    uint32_t issued = 0, landed = 0;  // bf16: steps issued, and waited for
    uint32_t started = 0;             // lane 0: issued steps whose copies were started (all, but after a timeout)
    int4 tail = make_int4(-1, 0, 0, 0);
    long long pos = sh.r0;
    long long seg = worker;
    W st;

    auto team_sync = [&]() {
        if (size() == 1)
            __syncwarp();
        else
            __syncthreads();
    };

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    while (whole() ? seg < (long long)nb * per_base : pos < sh.r1) {
        if (whole()) {
            base = (int)(seg / per_base);
            sub = (int)(seg - (long long)base * per_base);
        }
        const int blk = a.per_shard ? base / a.batch : 0, b = base - blk * a.batch;
        const int g = sub / a.tiles, tile = sub - g * a.tiles;
        const int lo = a.shard_lo + blk, hi = a.per_shard ? lo + 1 : a.shard_hi;
        const int L = length_of(a, b);
        const Visible v(L, a);
        const int real = v.count(lo, hi, a);  // 0: nothing visible, one empty group
        const int ng = max(real, 1);
        // groups [i0, i0 + take) of the segment fall to this worker
        const int x1 = whole() ? ng : (int)min((long long)(ng + a.lead), x0 + (sh.r1 - pos));
        const int i0 = whole() ? 0 : max(0, x0 - a.lead), take = whole() ? ng : max(0, x1 - a.lead) - i0;
        if (take > 0) {
        const int nk = wt < take ? (take - wt + size() - 1) / size() : 0;  // this warp's groups

        // bit k % 32: every row sees all of group k (of the even and the odd batches); clear past the last group
        uint32_t full0 = 0, full1 = 0;
        // descriptors of this warp's groups 32 kb .. 32 kb + 31, one for each lane
        auto batch = [&](int kb) {
            const int k = 32 * kb + lane, i = i0 + wt + size() * k;
            Desc d{-1, 0, 0, 0};
            bool whole_group = false;
            if (k < nk && i < real) {
                const Place at = place_of(a, v, lo, hi, i);
                d = describe(a, v, at, page_at(a, at, b), g, FP4 ? fp4_block_bytes(a.page_size, D) : 0, D / 2,
                             &whole_group);
            }
            const uint32_t mask = __ballot_sync(0xffffffffu, whole_group);
            if (kb & 1)
                full1 = mask;
            else
                full0 = mask;
            descs[(kb & 1) * 32 + lane] = d;
            __syncwarp();
        };
        // are the groups of the step at k all seen whole by every row?
        auto step_full = [&](int k) {
            constexpr uint32_t m = (1u << C::kStep) - 1u;
            return (((k & 32 ? full1 : full0) >> (k & 31)) & m) == m;
        };

        auto start = [&](int k, int slot) {  // copies of one step
            if ((k & 31) == 0) batch(k >> 5);
            const Desc* d = descs + (k & (kDescs - 1));
            if (!FP4) {  // slots and phases run on from segment to segment
                if (k >= nk) return;
                __syncwarp();  // every lane is done with the stage
                if (lane == 0 && !s_abort) {
                    const uint32_t at = issued % C::kSteps;
                    uint8_t* stage = ring + at * C::kStage;
                    uint64_t* bar = &s_full[warp][at];
                    if (d->off >= 0) {
                        const int row = (int)d->off, y = d->sub;
                        mbar_arrive_expect_tx(bar, C::kStage);
                        tma_load_4d(stage, &a.map_k, 0, y, 0, row, bar);
                        tma_load_4d(stage + C::kK * 32, &a.map_v, 0, y, 0, row, bar);
                    } else {
                        mbar_arrive(bar);
                    }
                    started = issued + 1;
                }
                issued++;
                return;
            }
            if (k >= nk) {
            } else if (step_full(k)) {
                const bool live[6] = {true, true, true, true, true, true};
#pragma unroll
                for (int e = 0; e < C::kStep; e++)
                    W::template copy<false>(places, d[e], live, ring_u32 + (slot + e) * C::kStage);
            } else {
#pragma unroll 1
                for (int e = 0; e < C::kStep; e++)
                    W::copy_masked(places, d[e], ring_u32 + (slot + e) * C::kStage);
            }
            cp_commit();
        };
        // wait for step k and return its stage
        auto arrived = [&](int k, int slot) -> uint8_t* {
            if (FP4) {
                cp_wait<C::kSteps - 2>();
                return ring + slot * C::kStage;
            }
            const uint32_t at = landed % C::kSteps;
            if (k < nk) {  // on a timeout the copies' bytes are used as they are: the call's outputs are unspecified
                mbar_wait(&s_full[warp][at], (landed / C::kSteps) & 1, &s_abort, a.status);
                landed++;
            }
            return ring + at * C::kStage;
        };
#pragma unroll 1
        for (int k = 0; k < C::kSteps - 1; k++) start(k * C::kStep, k * C::kStep);
        st.reset();
        st.load_q(a, b, g, tile, L, kf);
        // Software pipeline: the scores of step k + 1 are computed beside P V of step k,
        // two independent streams of matrix instructions.  (Past the last step the
        // scores are of leftover bytes and nobody reads them.)
        int slot_in = (C::kSteps - 1) * C::kStep, slot_out = 0;
        float x[2 * C::kStep][4];
        uint8_t* here = arrived(0, 0);
        st.step_scores(here, x);
        int k = 0;
#pragma unroll 1
        for (;;) {
        const int stop = W::kFlush && a.acc ? min(nk, k + W::kFlush) : nk;
#pragma unroll 1
        for (; k < stop; k += C::kStep) {
            start(k + (C::kSteps - 1) * C::kStep, slot_in);
            if ((slot_in += C::kStep) == S) slot_in = 0;
            uint8_t* at = here;
            if ((slot_out += C::kStep) == S) slot_out = 0;
            here = arrived(k + C::kStep, slot_out);
            const Desc* d = descs + (k & (kDescs - 1));
            uint32_t keep[C::kStep];
            typename W::Terms p[C::kStep];
#pragma unroll
            for (int e = 0; e < C::kStep; e++) keep[e] = 0xffffffffu;
            const bool full = step_full(k);
            if (!full) st.mask(a, d, at, x, keep);
            st.softmax(x, p);
            bool safe = true;
            if (!full && a.q_len > 1) {
#pragma unroll
                for (int e = 0; e < C::kStep; e++) safe &= !W::poisoned(at + e * C::kStage, keep[e]);
            }
            if (safe) {
                st.step_scores(here, x);
                st.values(at, keep, p);
            } else {
#pragma unroll 1
                for (int e = 0; e < C::kStep; e++) {
                    typename W::Terms t;  // chosen without an index, so that p stays in registers
#pragma unroll
                    for (int i = 0; i < W::kTerms * 4; i++) t[i / 4][i % 4] = e ? p[C::kStep - 1][i / 4][i % 4] : p[0][i / 4][i % 4];
                    st.careful(a, d[e], at + e * C::kStage, e ? keep[C::kStep - 1] : keep[0], t);
                }
                st.step_scores(here, x);
            }
        }
        if (k >= nk) break;
        if (W::kFlush) st.flush(acc(), k == W::kFlush);
        }
        cp_wait<0>();
        __syncwarp();  // the next segment's descriptors overwrite these
        if (W::kFlush && nk > W::kFlush && a.acc) st.unflush(acc());
        st.close();

        // where the rows go: the caller's tensors, or a slot of the workspace
        const bool starts = i0 == 0, ends = i0 + take == ng;
        const bool final_rows = starts && ends;
        const int part = 2 * worker + (starts ? 1 : 0);
        const int rows = min(kMine, a.rows - tile * kRows);
        const int qr = lane >> 2, c = lane & 3;
        auto put = [&](int r, int d, const float4& x) {  // 4 dimensions of row r
            float* dst = final_rows ? out_row(a, base, g, tile, r, D).o : a.part_o + ((int64_t)part * kRows + r) * D;
            *reinterpret_cast<float4*>(dst + d) = x;
        };
        auto put_lse = [&](int r, float lse2) {
            if (final_rows)
                *out_row(a, base, g, tile, r, D).lse = lse2 * kLn2;
            else
                a.part_lse[(int64_t)part * kRows + r] = lse2;
        };
        if (size() == 1) {
#pragma unroll
            for (int h = 0; h < (HALF ? 1 : 2); h++) {
                const int r = qr + 8 * h;
                const float inv = st.l[h] == 0.f ? 0.f : vf / st.sum(h);
                st.each(h, c, [&](int d, const float4& x) {
                    if (r < rows) put(r, d, make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv));
                });
                if (r < rows) {
                    if (c == 0) put_lse(r, st.l[h] == 0.f ? -INFINITY : (st.m[h] == -INFINITY ? 0.f : st.m[h]) + log2f(st.l[h]));
                }
            }
        } else {
            // the team's warps: each leaves its O in its own (drained) queue, then all
            // threads sum the four with the weights of their references
            float* so = reinterpret_cast<float*>(ring);
#pragma unroll
            for (int h = 0; h < (HALF ? 1 : 2); h++) {
                const int r = qr + 8 * h;
                st.each(h, c, [&](int d, const float4& x) { *reinterpret_cast<float4*>(so + r * kPitch + d) = x; });
                if (!FP4) fence_async();
                if (c == 0) {
                    s_m[warp][r] = st.m[h];
                    s_l[warp][r] = st.l[h];
                    s_ol[warp][r] = st.sum(h);
                }
            }
            __syncthreads();
            for (int k = threadIdx.x; k < rows * (D / 4); k += 32 * WARPS) {
                const int r = k / (D / 4), d = (k - r * (D / 4)) * 4;
                float M = -INFINITY, ls = 0.f, ols = 0.f;
#pragma unroll
                for (int w = 0; w < WARPS; w++) M = fmaxf(M, s_m[w][r]);
                const float ref = M == -INFINITY ? 0.f : M;
                float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < WARPS; w++) {
                    if (s_l[w][r] == 0.f) continue;
                    const float f = s_m[w][r] == -INFINITY ? 1.f : fast_exp2(s_m[w][r] - ref);
                    const float4 x = *reinterpret_cast<const float4*>(
                        reinterpret_cast<const float*>(smem + (size_t)w * kRing) + r * kPitch + d);
                    ls = fmaf(f, s_l[w][r], ls);
                    ols = fmaf(f, s_ol[w][r], ols);
                    acc.x = fmaf(f, x.x, acc.x);
                    acc.y = fmaf(f, x.y, acc.y);
                    acc.z = fmaf(f, x.z, acc.z);
                    acc.w = fmaf(f, x.w, acc.w);
                }
                const float inv = ls == 0.f ? 0.f : vf / ols;
                put(r, d, make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
                if (d == 0) put_lse(r, ls == 0.f ? -INFINITY : ref + log2f(ls));
            }
        }
        if (a.finish_ns && take > 0) {
            team_sync();
            if (wt == 0 && lane == 0) record_finish(a, b);
        }
        if (!whole() && starts && !ends) {
            // the worker whose share holds the segment's last group
            tail = make_int4(base, sub, last_worker(sh, pos - x0 + a.lead + ng), 0);
        }
        team_sync();  // queues and s_m are free again
        }
        if (whole()) {
            seg += a.workers;
        } else {
            pos += x1 - x0;
            x0 = 0;
            if (++sub == per_base) {
                sub = 0;
                base++;
            }
        }
    }
    if (!whole() && wt == 0 && lane == 0) a.tail[worker] = tail;
    // after a timeout copies may still be in flight: wait for them, bounded, before the block's memory is given up
    if (!FP4 && lane == 0 && s_abort)
        for (uint32_t k = started < C::kSteps ? 0 : started - C::kSteps; k < started; k++)
            mbar_wait(&s_full[warp][k % C::kSteps], (k / C::kSteps) & 1, nullptr, a.status);
}

// Sums of the segments that are in parts: the tail of worker w and the heads of the
// workers after it up to tail[w].z.  CTA (x, block of rows): workers x, x + gridDim.x, ..,
// 32 at most; `wpr` warps share a row's parts.  The kernel may be resident while the parts are
// still being written (it is launched ahead), so they are read by plain loads only: the
// read-only path is for data that does not change while a kernel lives.
__global__ void __launch_bounds__(256) combine_kernel(const __grid_constant__ StreamArgs a, int D, int wpr) {
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the parts are complete and visible
    __shared__ float s_w[8];
    __shared__ float4 s_o[8][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rpc = 8 / wpr;
    const int r = blockIdx.y * rpc + warp / wpr, part = warp % wpr;
    const int nv = D / 4;
    const int mine = blockIdx.x + lane * gridDim.x;
    uint32_t todo = __ballot_sync(0xffffffffu, mine < a.workers && a.tail[mine].x >= 0);  // the same in every warp
    for (; todo; todo &= todo - 1) {
        const int first = blockIdx.x + (__ffs(todo) - 1) * gridDim.x;
        const int4 t = a.tail[first];
        const int g = t.y / a.tiles, tile = t.y - g * a.tiles;
        const bool live = r < min(kRows, a.rows - tile * kRows);
        const int K = t.z - first + 1;  // parts
        // part k's slot: the tail of the first worker, the heads of the others
        auto slot = [&](int k) { return (int64_t)(2 * (first + k) + (k == 0 ? 1 : 0)) * kRows + r; };
        float M = -INFINITY, ws = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        if (live) {
            for (int k = lane; k < K; k += 32) M = fmaxf(M, a.part_lse[slot(k)]);
#pragma unroll
            for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
            const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll 4
            for (int k = part; k < K; k += wpr) {
                const float e = a.part_lse[slot(k)];
                float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
                if (lane < nv) x = reinterpret_cast<const float4*>(a.part_o + slot(k) * D)[lane];
                const float w = e == -INFINITY ? 0.f : exp2f(e - ref);
                ws += w;
                acc.x = fmaf(w, x.x, acc.x);
                acc.y = fmaf(w, x.y, acc.y);
                acc.z = fmaf(w, x.z, acc.z);
                acc.w = fmaf(w, x.w, acc.w);
            }
        }
        s_w[warp] = ws;
        s_o[warp][lane] = acc;
        __syncthreads();
        if (live && part == 0) {
            for (int w = 1; w < wpr; w++) {
                const float4 x = s_o[warp + w][lane];
                ws += s_w[warp + w];
                acc.x += x.x;
                acc.y += x.y;
                acc.z += x.z;
                acc.w += x.w;
            }
            const float inv = ws == 0.f ? 0.f : 1.f / ws;
            const Row row = out_row(a, t.x, g, tile, r, D);
            if (lane < nv)
                reinterpret_cast<float4*>(row.o)[lane] = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
            if (lane == 0) *row.lse = ws == 0.f ? -INFINITY : ((M == -INFINITY ? 0.f : M) + log2f(ws)) * kLn2;
        }
        __syncthreads();
    }
}

__global__ void finish_init_kernel(int64_t* finish_ns, int64_t* t_start, int B) {
    for (int b = threadIdx.x; b < B; b += blockDim.x) finish_ns[b] = 0;
    if (threadIdx.x == 0) *t_start = (int64_t)global_timer_ns();
}

template <bool FP4, int D, bool HALF, int WARPS>
cudaError_t run(const StreamArgs& a, int ctas, cudaStream_t s) {
    constexpr int smem = WARPS * Lane<FP4, D>::kStages * Lane<FP4, D>::kStage + (FP4 ? 0 : 1024);
    // once per process and device would do; the call is cheap and keeps no state
    cudaError_t e = cudaFuncSetAttribute(gqa_stream_kernel<FP4, D, HALF, WARPS>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    gqa_stream_kernel<FP4, D, HALF, WARPS><<<ctas, 32 * WARPS, smem, s>>>(a);
    return cudaGetLastError();
}
template <bool FP4, int D>
cudaError_t run(const StreamArgs& a, int ctas, cudaStream_t s) {
    const bool half = a.rows <= 8;
    if (a.team == 2) return half ? run<FP4, D, true, 2>(a, ctas, s) : run<FP4, D, false, 2>(a, ctas, s);
    return half ? run<FP4, D, true, 4>(a, ctas, s) : run<FP4, D, false, 4>(a, ctas, s);
}

}  // namespace

bool gqa_stream_supported(int hq, int hkv, int dk, int q_len) {
    return (dk == 64 || dk == 128) && hq % hkv == 0 && q_len >= 1;
}

// Whole segments or equal shares.  The rule compares estimates in units of one group's
// work by a warp (about 1 us): whole segments -- rounds times the longest segment that
// the tables and the mask allow, plus what a segment costs beside its groups, more in a
// team (its sum) and most where other teams share the SM -- and equal shares: the mean,
// plus the scan of the lengths, the partials and a second kernel.  Measured: a window of
// 128 (2 segments of about 11 groups) 8.0 us in a team of 4, 15.3 us a warp, 10.5 us in
// shares; a window of 1021 (512 of 68) 48.5 us in teams of 2, 57 us a warp, 65 us in teams
// of 4, 71 us in shares; a window of 4096 (512 of 258) 184 us in teams of 2, 186 us in
// shares, 196 us in teams of 4, 280 us a warp.
// Shares: a team of 4 needs a fourth of the parts, a lone warp wastes nothing on short
// segments: 48 requests of 1-14k tokens, 384 segments 47.3 us in teams, 49.6 us alone;
// one request of 65536 tokens, 4 segments, 41 and 59 us (39 us since the sums of parts are
// read by plain loads).  The longest segment is taken from the tables' width, which a server
// keeps wider than its requests are long: the choice is then that of long requests.  lead: the same 48 requests 153,
// 65, 49 and 47 us at 4, 16, 32 and 48 groups a segment (teams; above 48 not measured), 72,
// 53, 50 and 52 us at 4, 8, 16 and 32 (a warp).
StreamPlan gqa_stream_plan(const dcp_cache_desc* c, int q_len, int window, int sinks, int shards, bool per_shard,
                           int num_sms) {
    StreamPlan p;
    const int64_t rows = (int64_t)q_len * (c->hq / c->hkv);
    const int64_t segs = (int64_t)(per_shard ? shards : 1) * c->batch * c->hkv * ((rows + kRows - 1) / kRows);
    const int64_t span = per_shard ? 1 : shards;
    // a shard's part starts and ends inside a group
    int64_t tokens = (int64_t)c->max_local_pages * c->page_size * shards;
    if (window != INT_MAX) {
        const int64_t seen = (int64_t)sinks + window + q_len - 1;
        if (seen < tokens) tokens = seen;
    }
    const int64_t groups = (tokens / shards + kTok - 1) / kTok * span + 2 * span;
    const int64_t warps = (int64_t)num_sms * kWarpsPerSm, ctas = warps / kWarps;
    const int64_t one = (segs + warps - 1) / warps * groups * (2 * segs <= warps ? 3 : 4) / 4 + 6;
    const int64_t four =
        (segs + ctas - 1) / ctas * ((groups + kWarps - 1) / kWarps + (2 * kWarps * segs > warps ? 14 : 8));
    const int64_t two = (2 * segs + warps - 1) / warps * ((groups + 1) / 2 + (4 * segs > warps ? 16 : 10));
    const int64_t share = (segs * (groups + 16) + warps - 1) / warps + 30;
    p.team = 1;
    p.whole = 1;
    int64_t best = one;
    if (four < best) {
        best = four;
        p.team = kWarps;
    }
    if (two < best) {
        best = two;
        p.team = 2;
    }
    if (share < best) {
        p.whole = 0;
        p.team = 2 * segs >= warps ? 1 : kWarps;
    }
    p.lead = p.team == 1 ? 16 : 48;
    const int wpc = p.team == 2 ? 2 : kWarps;  // warps of a CTA
    const int64_t grid = p.whole ? (segs * p.team + wpc - 1) / wpc : ctas;
    p.ctas = (int)(grid < warps / wpc ? grid : warps / wpc);
    p.workers = p.ctas * (wpc / p.team);
    p.segs = segs;
    p.off_start = 0;
    p.off_tail = 256;
    p.off_lse = p.off_o = p.off_acc = 0;
    size_t o = p.off_tail;
    using W = Warp<true, 64, false>;
    // sums in memory only where one warp can have more groups of a segment than it adds up without
    if (c->dtype == DCP_FP4_E2M1 && rows > kRows / 2 && (groups + p.team - 1) / p.team > W::kFlush) {
        p.off_acc = o;
        o += sizeof(float4) * kAcc * (size_t)p.ctas * wpc;
        p.off_tail = o;
    }
    if (!p.whole) {
        o = align256(o + sizeof(int4) * (size_t)p.workers);
        p.off_lse = o;
        o = align256(o + sizeof(float) * (size_t)p.workers * 2 * kRows);
        p.off_o = o;
        o = align256(o + sizeof(float) * (size_t)p.workers * 2 * kRows * c->dk);
    }
    p.total = o;
    return p;
}

cudaError_t launch_gqa_stream(const dcp_cache_desc* c, const StreamPlan& p, int q_len, int window, int sinks,
                              int shard_lo, int shard_hi, bool per_shard, int bt_shard0, const void* q,
                              const int32_t* seq_lens, float* out, float* lse, int64_t* finish_ns, void* ws,
                              int* status, cudaStream_t s) {
    uint8_t* w = static_cast<uint8_t*>(ws);
    StreamArgs a;
    a.k_pages = static_cast<const uint8_t*>(c->k_pages);
    a.v_pages = static_cast<const uint8_t*>(c->v_pages);
    a.factors = c->dtype == DCP_FP4_E2M1 ? c->kv_scales : nullptr;
    a.block_tables = c->block_tables;
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.seq_lens = seq_lens;
    a.out = out;
    a.lse = lse;
    a.part_o = p.whole ? nullptr : reinterpret_cast<float*>(w + p.off_o);
    a.part_lse = p.whole ? nullptr : reinterpret_cast<float*>(w + p.off_lse);
    a.acc = p.off_acc ? reinterpret_cast<float4*>(w + p.off_acc) : nullptr;
    a.tail = p.whole ? nullptr : reinterpret_cast<int4*>(w + p.off_tail);
    a.status = status;
    a.finish_ns = finish_ns;
    a.t_start = reinterpret_cast<int64_t*>(w + p.off_start);
    const uint64_t in = (uint64_t)c->interleave * (uint64_t)c->n_shards;
    a.in = in > 0xffffffffu ? 0xffffffffu : (uint32_t)in;
    a.n_shards = c->n_shards;
    a.interleave = c->interleave;
    a.page_size = c->page_size;
    a.num_pages = c->num_pages;
    a.batch = c->batch;
    a.max_local_pages = c->max_local_pages;
    a.hq = c->hq;
    a.hkv = c->hkv;
    a.q_len = q_len;
    a.group = c->hq / c->hkv;
    a.rows = q_len * a.group;
    a.tiles = (a.rows + kRows - 1) / kRows;
    a.window = window;
    a.sinks = sinks;
    // shard n's first position past its table, local index T, is past0 + n * interleave
    const int64_t T = (int64_t)c->max_local_pages * c->page_size, I = c->interleave;
    const int64_t past0 = T / I * I * c->n_shards + T % I, past = past0 + (c->n_shards - 1) * I + 1;
    a.past0 = past0 < INT_MAX ? (int)past0 : INT_MAX;
    a.past = past < INT_MAX ? (int)past : INT_MAX;
    a.shard_lo = shard_lo;
    a.shard_hi = shard_hi;
    a.per_shard = per_shard;
    a.bt_shard0 = bt_shard0;
    a.team = p.team;
    a.workers = p.workers;
    a.whole = p.whole;
    a.lead = p.lead;
    a.scale_log2 = c->scale * kLog2e;
    if (finish_ns) {
        finish_init_kernel<<<1, 256, 0, s>>>(finish_ns, reinterpret_cast<int64_t*>(w + p.off_start), c->batch);
        cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    const bool fp4 = c->dtype == DCP_FP4_E2M1;
    cudaError_t e;
    if (!fp4) {
        // the pools as [page * hkv + head][64-column half][token][64 columns]; a box is 16 tokens of one head
        const uint64_t dims[4] = {64, (uint64_t)c->page_size, (uint64_t)(c->dk / 64), (uint64_t)c->num_pages * c->hkv};
        const uint64_t strides[3] = {(uint64_t)c->dk * 2, 128, (uint64_t)c->page_size * c->dk * 2};
        const uint32_t box[4] = {64, (uint32_t)kTok, (uint32_t)(c->dk / 64), 1};
        if (!make_tmap_4d(&a.map_k, c->k_pages, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, dims, strides, box,
                          CU_TENSOR_MAP_SWIZZLE_128B) ||
            !make_tmap_4d(&a.map_v, c->v_pages, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, dims, strides, box,
                          CU_TENSOR_MAP_SWIZZLE_128B))
            return cudaErrorInvalidValue;
    }
    if (c->dk == 64) {
        if (fp4)
            e = run<true, 64>(a, p.ctas, s);
        else
            e = run<false, 64>(a, p.ctas, s);
    } else {
        if (fp4)
            e = run<true, 128>(a, p.ctas, s);
        else
            e = run<false, 128>(a, p.ctas, s);
    }
    if (e != cudaSuccess || p.whole) return e;
    // few parts a segment: a row for each warp; many: a CTA for each row
    const int wpr = p.workers >= 8 * p.segs ? 8 : 1;
    const int rows = a.rows < kRows ? a.rows : kRows;
    // at most one sum a segment: few segments take few CTAs (65536 tokens of 4 segments: 0.7 us less than a CTA for
    // each of 296 workers); four for each segment, so that a CTA seldom has two sums; a CTA takes 32 workers at most
    const int64_t least = (p.workers + 31) / 32, some = 4 * p.segs < p.workers ? 4 * p.segs : p.workers;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(some > least ? some : least), (unsigned)((rows + 8 / wpr - 1) / (8 / wpr)));
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute attr;  // the launch overlaps the kernel before it; combine_kernel waits for its end
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, combine_kernel, a, (int)c->dk, wpr);
}

}  // namespace dcp
