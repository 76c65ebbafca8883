// decode_gqa_fp4.cu -- GQA decode attention over a 4-bit cache on 5th-generation
// tensor cores (tcgen05, accumulators in TMEM), head size 128, 16 or 32 query rows.
//
// "Efficient Decode Context Parallelism with vLLM for Long Context Workloads",
// section 4.1 ("Compute" on the local KV slice, partial output + LSE) and section 5.4
// (each KV head broadcast to its query heads).
//
// Mathematics, for a tile of 128 visible tokens and N query rows (query heads of the KV
// head times query tokens):
//   S   = K Q^T    [128 tokens][N], K in fp16 as A operand in TMEM, Q in shared memory;
//   P   = exp2(scale S - m), one thread for a token and half of the rows;
//   O^T = V^T P    [128 dimensions][hi | lo], V in fp16 in shared memory (dimensions
//                  contiguous), P as two fp16 terms, 2 N columns.
// Code times scale has 6 significant bits and is exact in fp16; q is scaled by a power of
// two into fp16's range; the two terms of P carry 22 bits, and the reference m lies 2^7
// below the maximum so that small weights stay above fp16's smallest step.  m moves
// only when a row's maximum grows by more than 2^8.  O^T is taken out of TMEM into
// 32-bit registers every 8 tiles, so that what the tensor core cuts off at each
// accumulation does not add up over long requests.
//
// What bounds it: 144 bytes of K and V for each token and KV head, against the
// conversion of 256 codes.  On warp-level matrix instructions the tensor pipe itself
// was the limit (50 instructions for 16 tokens and 16 rows, 11 cycles each: the
// same call over 24 requests of 32k-128k tokens took 322 us); here the matrices cost an
// eighth of that and the threads do nothing but convert.  Two blocks of 256 threads
// share an SM (256 TMEM columns and ~105 KB each): one converts while the other's matrices
// or copies are under way.
//
// One iteration, tile t:   copies of K(t+3) and V(t+2) start; K(t+1) -> fp16 -> TMEM;
// V(t) -> fp16 -> shared memory once O^T of tile t-1 is done; S(t) -> P(t); one barrier;
// one thread issues O^T(t) and S(t+1).
#include "kernels.h"
#include "stream.cuh"
#include "umma.cuh"

namespace dcp {

namespace {

constexpr int D = 128;
constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kTile = 128;                  // tokens per tile
constexpr int kGroups = kTile / kTok;       // groups per tile
constexpr int kDescs = 64;                  // group descriptors: eight tiles
constexpr int kRing = 3;                    // K and V stages each
constexpr int kCode = kTile * D / 2;        // codes of a stage
constexpr int kScale = kTile * D / 16;      // scales of a stage: [D/16][128 tokens]
constexpr int kStage = kCode + kScale;
constexpr int kVBytes = kTile * D * 2;      // V in fp16: two boxes [128 tokens][64 dimensions], 128-byte swizzle
constexpr int kPBytes = kTile * 128;        // P: [128 tokens][hi rows | lo rows], 128-byte rows, swizzled
constexpr int kDrain = 8;                   // tiles between two reads of O^T
constexpr float kBias = 7.f;
constexpr uint32_t kTmemCols = 256;

template <int N>
constexpr uint32_t smem_bytes() {
    return 1024 + kVBytes + kPBytes + (uint32_t)N * D * 2 + 2u * kRing * kStage;
}

__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// 16-byte chunk c of row r in a box of 128-byte rows with 128-byte swizzle
__device__ __forceinline__ uint32_t sw128(int r, int c) { return (uint32_t)(r * 128 + (((c ^ r) & 7) << 4)); }

template <int N>
__global__ void __launch_bounds__(kThreads, 2) gqa_fp4_umma_kernel(const __grid_constant__ StreamArgs a) {
    constexpr int NH = N / 2;  // rows of a thread
    constexpr uint32_t IDESC_S = umma::idesc_f16(0u, 0, 0, 128, N);       // f16, K in TMEM, Q K-major
    constexpr uint32_t IDESC_PV = umma::idesc_f16(0u, 1, 1, 128, 2 * N);  // f16, V^T and P MN-major
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sV = sm;
    uint8_t* sP = sV + kVBytes;
    uint8_t* sQ = sP + kPBytes;  // [2 halves][N rows][128 B]
    uint8_t* sK4 = sQ + N * D * 2;
    uint8_t* sV4 = sK4 + kRing * kStage;
    __shared__ Desc s_desc[kDescs];
    __shared__ uint32_t s_full[2];           // bit k % 32: every row sees all of group k (even and odd batches)
    __shared__ ShareScratch<kWarps> s_share;
    __shared__ float s_scale[N];             // softmax scale times the row's power of two
    __shared__ float s_max[4][N], s_sum[4][N];
    __shared__ uint32_t s_poison[N];         // bit j: the row sees a NaN among values 16 j .. 16 j + 15
    __shared__ uint64_t s_bar[2];            // S ready, O^T done
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_abort;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int tok = tid & 127, hf = tid >> 7;  // this thread's token (dimension of O^T) and half of dimensions / rows
    const uint32_t lane_off = (uint32_t)(32 * (warp & 3)) << 16;
    const int worker = blockIdx.x;
    const int nb = (a.per_shard ? a.shard_hi - a.shard_lo : 1) * a.batch;
    const int per_base = a.hkv * a.tiles;
    const float kf = a.factors ? __ldg(a.factors) : 1.f, vf = a.factors ? __ldg(a.factors + 1) : 1.f;
    const int P = a.page_size, block = fp4_block_bytes(P, D);

    if (tid == 0) {
        mbar_init(&s_bar[0], 1);
        mbar_init(&s_bar[1], 1);
        s_abort = 0;
        fence_barrier_init();
    }
    if (warp == 0) umma::tmem_alloc(&s_tmem, kTmemCols);
    check_lengths(a);
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
    const uint32_t t_k = *reinterpret_cast<volatile uint32_t*>(&s_tmem);  // two buffers of 64 columns
    const uint32_t t_s = t_k + 128, t_o = t_s + N;
    const uint64_t dq = umma::smem_desc(smem_u32(sQ), 16, 1024, umma::kSw128);
    const uint64_t dv = umma::smem_desc(smem_u32(sV), kVBytes / 2, 1024, umma::kSw128);
    const uint64_t dp = umma::smem_desc(smem_u32(sP), kPBytes, 1024, umma::kSw128);

    // a tile costs a block about 8 groups' worth of the flat list; no share below two tiles
    Share sh{0, 0, 0, 0, 0, 0, 0};
    if (!a.whole) sh = find_share<kWarps>(a, nb, per_base, 1, 0, 2 * kGroups, s_share);
    int base = sh.base, sub = sh.sub, x0 = sh.x0;
    int4 tail = make_int4(-1, 0, 0, 0);
    long long pos = sh.r0, seg = worker;
    uint32_t ph_s = 0, ph_o = 0;  // phases of the two barriers
    bool fail = false;

    // S of a tile whose K lies in buffer `buf`: 8 k-steps of 16 dimensions
    auto issue_s = [&](int buf) {
#pragma unroll
        for (int k = 0; k < D / 16; k++)
            umma::mma_f16_ts(t_s, t_k + 64 * buf + 8 * k, dq + (uint64_t)(((k >> 2) * (N * 128) + (k & 3) * 32) >> 4),
                             IDESC_S, k ? 1u : 0u);
        umma::commit(&s_bar[0]);
    };
    // O^T (+)= V^T P: 8 k-steps of 16 tokens
    auto issue_o = [&](bool add) {
#pragma unroll
        for (int k = 0; k < kTile / 16; k++)
            umma::mma_f16(t_o, dv + (uint64_t)((k * 2048) >> 4), dp + (uint64_t)((k * 2048) >> 4), IDESC_PV,
                          add || k ? 1u : 0u);
        umma::commit(&s_bar[1]);
    };

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    while (!fail && (a.whole ? seg < (long long)nb * per_base : pos < sh.r1)) {
        if (a.whole) {
            base = (int)(seg / per_base);
            sub = (int)(seg - (long long)base * per_base);
        }
        const int blk = a.per_shard ? base / a.batch : 0, b = base - blk * a.batch;
        const int g = sub / a.tiles, tile = sub - g * a.tiles;
        const int lo = a.shard_lo + blk, hi = a.per_shard ? lo + 1 : a.shard_hi;
        const Visible v(length_of(a, b), a);
        const int real = v.count(lo, hi, a);  // 0: nothing visible, one empty group
        const int ng = max(real, 1);
        // groups [i0, i0 + take) of the segment fall to this block
        const int x1 = a.whole ? ng : (int)min((long long)(ng + a.lead), x0 + (sh.r1 - pos));
        const int i0 = a.whole ? 0 : max(0, x0 - a.lead), take = a.whole ? ng : max(0, x1 - a.lead) - i0;
        if (take > 0) {
            const int nt = (take + kGroups - 1) / kGroups;  // tiles
            const int rows = min(N, a.rows - tile * N);

            // warp 0: descriptors of groups 32 kb .. 32 kb + 31 (four tiles)
            auto batch = [&](int kb) {
                const int k = 32 * kb + lane;
                Desc d{-1, 0, 0, 0, 0};
                bool full = false;
                if (k < take && i0 + k < real) d = describe(a, v, lo, hi, b, g, i0 + k, block, D / 2, &full);
                s_desc[(kb & 1) * 32 + lane] = d;
                const uint32_t m = __ballot_sync(0xffffffffu, full);
                if (lane == 0) s_full[kb & 1] = m;
            };
            // start the copies of tile t's codes (this thread's token and half) and, by threads of
            // half 0, its scales (16 bytes of a row of 16 tokens each)
            auto copy = [&](int t, const uint8_t* pool, uint8_t* ring) {
                if (t >= nt) return;
                const uint32_t dst = smem_u32(ring + (t % kRing) * kStage);
                const Desc* d = s_desc + ((t * kGroups) & (kDescs - 1));
                const int64_t off = d[tok >> 4].off;
                if (off >= 0) {
                    const uint8_t* src = pool + off + (tok & 15) * (D / 2) + hf * (D / 4);
                    cp16(dst + hf * (kCode / 2) + tok * 16, src);
                    cp16(dst + hf * (kCode / 2) + 2048 + tok * 16, src + 16);
                }
                if (hf == 0 && tok < 64) {
                    const Desc& e = d[tok >> 3];
                    if (e.off >= 0) {
                        const int sub16 = e.t0 & (P - 1), j = tok & 7;
                        cp16(dst + kCode + j * kTile + (tok >> 3) * 16,
                             pool + e.off + (int64_t)P * (D / 2) - sub16 * (D / 2 - 1) + j * P);
                    }
                }
            };
            // 64 dimensions of this thread's token as fp16 (zeros when !live); NaN blocks in *nan
            auto dequant = [&](const uint8_t* stage, bool live, uint32_t* h, uint32_t* nan) {
                const uint4 c0 = *reinterpret_cast<const uint4*>(stage + hf * (kCode / 2) + tok * 16);
                const uint4 c1 = *reinterpret_cast<const uint4*>(stage + hf * (kCode / 2) + 2048 + tok * 16);
                const uint32_t w[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    const uint32_t sb = live ? stage[kCode + (4 * hf + j) * kTile + tok] : 0u;
                    if (nan && (sb & 0x7f) == 0x7f) *nan |= 1u << (4 * hf + j);
                    const uint32_t s = e4m3x2(sb * 0x101u);
#pragma unroll
                    for (int k = 0; k < 2; k++) {
                        e2m1x8(w[2 * j + k], h + 8 * j + 4 * k);
#pragma unroll
                        for (int e = 0; e < 4; e++) h[8 * j + 4 * k + e] = mul2(h[8 * j + 4 * k + e], s);
                    }
                }
            };
            auto convert_k = [&](int t) {
                uint32_t h[32];
                dequant(sK4 + (t % kRing) * kStage, true, h, nullptr);
                umma::st32(t_k + 64 * (t & 1) + 32 * hf + lane_off, h);
                umma::wait_st();
            };

            // the first tiles' descriptors, and Q: rows of 16 (N = 16) or 8 (N = 32) threads
            if (warp == 0) batch(0);
            {
                constexpr int TPR = kThreads / N, VPT = D / 8 / TPR;  // threads of a row, 16-byte pieces of a thread
                const int r = tid / TPR, p = tid % TPR;
                const int rr = tile * N + r;
                const bool live = r < rows;
                const int j = live ? rr / a.group : 0, hh = live ? rr - j * a.group : 0;
                const uint4* src = reinterpret_cast<const uint4*>(
                    a.q + (((int64_t)b * a.q_len + j) * a.hq + g * a.group + hh) * D);
                float x[VPT][8], amax = 0.f;
#pragma unroll
                for (int c = 0; c < VPT; c++) {
                    const uint4 w = live ? __ldg(src + p * VPT + c) : make_uint4(0, 0, 0, 0);
                    unpack8(w, x[c]);
#pragma unroll
                    for (int e = 0; e < 8; e++) amax = fmaxf(amax, fabsf(x[c][e]));
                }
#pragma unroll
                for (int o = TPR / 2; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
                const float2 pw = row_power(amax);
                const float f = a.scale_log2 < 0.f ? -pw.x : pw.x;  // the sign of the scale goes into q
#pragma unroll
                for (int c = 0; c < VPT; c++) {
                    uint4 w;
                    uint32_t* ws = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        const __half2 h = __floats2half2_rn(x[c][2 * e] * f, x[c][2 * e + 1] * f);
                        ws[e] = *reinterpret_cast<const uint32_t*>(&h);
                    }
                    const int ch = p * VPT + c;
                    *reinterpret_cast<uint4*>(sQ + (ch >> 3) * (N * 128) + sw128(r, ch & 7)) = w;
                }
                if (p == 0) {
                    s_scale[r] = fabsf(a.scale_log2) * kf * pw.y;
                    s_poison[r] = 0;
                }
            }
            __syncthreads();  // descriptors, scales of the rows
            copy(0, a.k_pages, sK4);
            cp_commit();
            copy(1, a.k_pages, sK4);
            copy(0, a.v_pages, sV4);
            cp_commit();
            copy(2, a.k_pages, sK4);
            copy(1, a.v_pages, sV4);
            cp_commit();
            float m[NH], l[NH], o[NH];
#pragma unroll
            for (int r = 0; r < NH; r++) {
                m[r] = -INFINITY;
                l[r] = o[r] = 0.f;
            }
            cp_wait<1>();  // K(0), K(1), V(0)
            __syncthreads();
            convert_k(0);
            umma::fence_proxy_async_smem();  // Q
            umma::fence_before_sync();
            __syncthreads();
            if (tid == 0) {
                umma::fence_after_sync();
                issue_s(0);
            }
            bool add = false;  // O^T in TMEM holds tiles that o[] does not
            // O^T of the tiles so far into o[] (their products have completed)
            auto drain = [&]() {
                umma::fence_after_sync();
#pragma unroll
                for (int c = 0; c < NH; c += 8) {
                    uint32_t h[8], w[8];
                    umma::ld8(t_o + hf * NH + c + lane_off, h);
                    umma::ld8(t_o + N + hf * NH + c + lane_off, w);
                    umma::wait_ld();
#pragma unroll
                    for (int r = 0; r < 8; r++) o[c + r] += __uint_as_float(h[r]) + __uint_as_float(w[r]);
                }
                add = false;
            };

#pragma unroll 1
            for (int t = 0; t < nt; t++) {
                copy(t + 3, a.k_pages, sK4);
                copy(t + 2, a.v_pages, sV4);
                cp_commit();
                if ((t & 3) == 0 && warp == 0) batch((t >> 2) + 1);
                if (t + 1 < nt) convert_k(t + 1);
                // this tile's masks
                const Desc d = s_desc[(t * kGroups + (tok >> 4)) & (kDescs - 1)];
                const bool whole_tile = ((s_full[(t >> 2) & 1] >> ((t & 3) * kGroups)) & 0xff) == 0xff;
                const bool live = whole_tile || (d.live >> (tok & 15) & 1);
                // V, once the products that read the last one are done
                if (t > 0) {
                    fail |= !mbar_wait(&s_bar[1], ph_o & 1, &s_abort, a.status);
                    ph_o++;
                    if ((t & (kDrain - 1)) == 0) drain();
                }
                uint32_t nan = 0;
                {
                    uint32_t h[32];
                    const bool careful = !whole_tile && a.q_len > 1;
                    dequant(sV4 + (t % kRing) * kStage, live, h, careful ? &nan : nullptr);
                    if (nan) {  // a NaN that not every row sees is kept out of the product: rows note it instead
#pragma unroll
                        for (int j = 0; j < 4; j++)
                            if (nan >> (4 * hf + j) & 1) {
#pragma unroll
                                for (int e = 0; e < 8; e++) h[8 * j + e] = 0u;
                            }
                    }
#pragma unroll
                    for (int c = 0; c < 8; c++)
                        *reinterpret_cast<uint4*>(sV + hf * (kVBytes / 2) + sw128(tok, c)) =
                            make_uint4(h[4 * c], h[4 * c + 1], h[4 * c + 2], h[4 * c + 3]);
                }
                // scores
                fail |= !mbar_wait(&s_bar[0], ph_s & 1, &s_abort, a.status);
                ph_s++;
                umma::fence_after_sync();
                float x[NH];
#pragma unroll
                for (int c = 0; c < NH; c += 8) {
                    uint32_t w[8];
                    umma::ld8(t_s + hf * NH + c + lane_off, w);
                    umma::wait_ld();
#pragma unroll
                    for (int r = 0; r < 8; r++) x[c + r] = __uint_as_float(w[r]) * s_scale[hf * NH + c + r];
                }
                if (!whole_tile) {
                    const int64_t p = position_of(a, d.shard, d.t0 + (tok & 15));
#pragma unroll
                    for (int r = 0; r < NH; r++) {
                        bool see = live;
                        if (live && a.q_len > 1)
                            see = sees(a, p, v.first + min(a.q_len - 1, (tile * N + hf * NH + r) / a.group));
                        if (!see) x[r] = -INFINITY;
                    }
                    if (a.q_len > 1) {
                        // both halves' threads of a token hold half of its blocks: each notes its own for all rows
                        for (int r = 0; nan && r < rows; r++)
                            if (sees(a, p, v.first + (tile * N + r) / a.group)) atomicOr(&s_poison[r], nan);
                    }
                }
                bool grow = false;
#pragma unroll
                for (int r = 0; r < NH; r++) grow |= x[r] > m[r] + (kLazy + kBias);
                // weights, against the references as they are
                auto weights = [&]() {
#pragma unroll
                    for (int c = 0; c < NH; c += 8) {
                        uint32_t hi[4], lw[4];
#pragma unroll
                        for (int e = 0; e < 4; e++) {
                            const int r = c + 2 * e;
                            const float p0 = fast_exp2(x[r] - (m[r] == -INFINITY ? 0.f : m[r]));
                            const float p1 = fast_exp2(x[r + 1] - (m[r + 1] == -INFINITY ? 0.f : m[r + 1]));
                            l[r] += p0;
                            l[r + 1] += p1;
                            const __half2 h = __floats2half2_rn(p0, p1);
                            const float2 f = __half22float2(h);
                            const __half2 w = __floats2half2_rn(p0 - f.x, p1 - f.y);
                            hi[e] = *reinterpret_cast<const uint32_t*>(&h);
                            lw[e] = *reinterpret_cast<const uint32_t*>(&w);
                        }
                        const int ch = (hf * NH + c) / 8;
                        *reinterpret_cast<uint4*>(sP + sw128(tok, ch)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                        *reinterpret_cast<uint4*>(sP + sw128(tok, N / 8 + ch)) = make_uint4(lw[0], lw[1], lw[2], lw[3]);
                    }
                };
                // the weights are computed on the guess that no reference moves
                float l_old[NH];
#pragma unroll
                for (int r = 0; r < NH; r++) l_old[r] = l[r];
                weights();
                umma::fence_proxy_async_smem();
                umma::fence_before_sync();
                cp_wait<1>();  // K(t + 2), V(t + 1)
                if (fail) s_abort = 1;
                if (__syncthreads_or(grow || fail)) {
                    if (s_abort) {
                        fail = true;
                        break;
                    }
                    // references: each row's maximum over the tile's tokens
#pragma unroll
                    for (int r = 0; r < NH; r++) {
                        float y = x[r];
#pragma unroll
                        for (int e = 16; e; e >>= 1) y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, e));
                        if (lane == 0) s_max[warp & 3][hf * NH + r] = y;
                    }
                    if (add) drain();
                    __syncthreads();
#pragma unroll
                    for (int r = 0; r < NH; r++) {
                        const int i = hf * NH + r;
                        const float y = fmaxf(fmaxf(s_max[0][i], s_max[1][i]), fmaxf(s_max[2][i], s_max[3][i]));
                        l[r] = l_old[r];
                        if (y > m[r] + (kLazy + kBias)) {
                            const float mn = y - kBias;
                            const float f = m[r] == -INFINITY ? 0.f : fast_exp2(m[r] - mn);
                            m[r] = mn;
                            l[r] *= f;
                            o[r] *= f;
                        }
                    }
                    weights();
                    umma::fence_proxy_async_smem();
                    umma::fence_before_sync();
                    __syncthreads();
                }
                if (tid == 0) {
                    umma::fence_after_sync();
                    issue_o(add);
                    if (t + 1 < nt) issue_s((t + 1) & 1);
                }
                add = true;
            }
            cp_wait<0>();
            if (!fail) {
                fail |= !mbar_wait(&s_bar[1], ph_o & 1, &s_abort, a.status);
                ph_o++;
                drain();
                // sums over the tokens
#pragma unroll
                for (int r = 0; r < NH; r++) {
                    float y = l[r];
#pragma unroll
                    for (int e = 16; e; e >>= 1) y += __shfl_xor_sync(0xffffffffu, y, e);
                    if (lane == 0) s_sum[warp & 3][hf * NH + r] = y;
                }
                umma::fence_before_sync();
                if (fail) s_abort = 1;
                __syncthreads();
                fail |= s_abort != 0;
                const bool starts = i0 == 0, ends = i0 + take == ng;
                const bool final_rows = starts && ends;
                const int part = 2 * worker + (starts ? 1 : 0);
#pragma unroll
                for (int r = 0; r < NH; r++) {
                    const int i = hf * NH + r;
                    if (i >= rows) continue;
                    const float ls = s_sum[0][i] + s_sum[1][i] + s_sum[2][i] + s_sum[3][i];
                    float y = ls == 0.f ? 0.f : o[r] * (vf / ls);
                    if (s_poison[i] >> (tok >> 4) & 1) y = __int_as_float(0x7fc00000);
                    const float lse2 = ls == 0.f ? -INFINITY : (m[r] == -INFINITY ? 0.f : m[r]) + log2f(ls);
                    if (final_rows) {
                        const Row row = out_row(a, base, g, tile, i, D);
                        row.o[tok] = y;
                        if (tok == 0) *row.lse = lse2 * kLn2;
                    } else {
                        a.part_o[((int64_t)part * N + i) * D + tok] = y;
                        if (tok == 0) a.part_lse[(int64_t)part * N + i] = lse2;
                    }
                }
                if (!a.whole && starts && !ends)
                    tail = make_int4(base, sub, last_worker(sh, pos - x0 + a.lead + ng), 0);
                __syncthreads();  // s_sum, s_poison and the descriptors are free again
                if (a.finish_ns && tid == 0) record_finish(a, b);
            }
        }
        if (a.whole) {
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
    if (!a.whole && tid == 0) a.tail[worker] = tail;
    // after a timeout matrices may still be under way: wait for them, bounded, before TMEM is freed
    cp_wait<0>();
    if (fail && tid == 0) {
        umma::commit(&s_bar[0]);
        umma::commit(&s_bar[1]);
        mbar_wait(&s_bar[1], ph_o & 1, nullptr, a.status);
    }
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
    if (warp == 0) umma::tmem_dealloc(t_k, kTmemCols);
}

}  // namespace

cudaError_t launch_gqa_fp4_umma(const StreamArgs& a, int ctas, cudaStream_t s) {
    cudaError_t e;
    if (a.tile_rows == 16) {
        e = cudaFuncSetAttribute(gqa_fp4_umma_kernel<16>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes<16>());
        if (e == cudaSuccess) gqa_fp4_umma_kernel<16><<<ctas, kThreads, smem_bytes<16>(), s>>>(a);
    } else {
        e = cudaFuncSetAttribute(gqa_fp4_umma_kernel<32>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes<32>());
        if (e == cudaSuccess) gqa_fp4_umma_kernel<32><<<ctas, kThreads, smem_bytes<32>(), s>>>(a);
    }
    return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace dcp
