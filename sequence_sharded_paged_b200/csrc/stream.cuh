// stream.cuh -- what the streamed GQA decode kernels share: which positions a query
// token sees, in groups of 16 local tokens of one page; how the groups of all
// requests, KV heads and row tiles are dealt to the workers; where rows go.
//
// A segment is (request, KV head, tile of query rows) -- of one shard when partials
// are asked for, of all shards otherwise -- and its visible groups.  "Efficient Decode
// Context Parallelism with vLLM for Long Context Workloads", section 4 (a shard owns
// a subset of the positions).
#pragma once

#include <limits.h>

#include "common.cuh"
#include "kernels.h"
#include "rows.cuh"
#include "tma.h"

namespace dcp {

constexpr int kTok = 16;      // tokens per group
constexpr int kRows = 16;     // query rows of a segment
constexpr float kLazy = 8.f;  // lazy rescale threshold (log2)

struct StreamArgs {
    alignas(64) CUtensorMap map_k, map_v;  // bf16: 4-D maps of the pools, boxes of one group
    const uint8_t* k_pages;
    const uint8_t* v_pages;
    const float* factors;  // 4-bit: {K, V} factors, or null
    const int32_t* block_tables;
    const __nv_bfloat16* q;
    const int32_t* seq_lens;
    float* out;
    float* lse;
    float* part_o;    // [2 * workers][kRows][D]
    float* part_lse;  // [2 * workers][kRows], log2
    float4* acc;      // [warps][kAcc] each warp's O between two flushes, or null
    int4* tail;  // [workers]: segment that starts in the worker's share and ends in another's: base, segment of
                 // the base, last worker
    int* status;
    int64_t* finish_ns;
    const int64_t* t_start;
    uint32_t in;  // interleave * n_shards, saturated
    int32_t n_shards, interleave, page_size, num_pages, batch, max_local_pages;
    int32_t hq, hkv, q_len, group, rows, tiles;  // tiles of kRows query rows for each KV head
    int32_t window, sinks;
    int32_t past0, past;  // every shard has a position past its table in [past0, past), and none before past0
    int32_t shard_lo, shard_hi, per_shard, bt_shard0;
    int32_t team;     // warps per team: 1, 2 (whole segments only) or 4
    int32_t workers;  // teams in the grid
    int32_t whole;    // whole segments, else equal shares
    int32_t lead;     // what a segment costs beside its groups, in groups (shares count it)
    float scale_log2;
};

// positions p < x that a shard owns; `off` is the shard's first position in a round,
// n * interleave (saturated, like a.in)
struct Counter {
    uint32_t base, rest;
    __device__ __forceinline__ Counter(uint32_t x, const StreamArgs& a) {
        const uint32_t q = x / a.in;
        base = q * (uint32_t)a.interleave;
        rest = x - q * a.in;
    }
    __device__ __forceinline__ int of(uint32_t off, uint32_t interleave) const {
        return (int)(base + min(rest - min(rest, off), interleave));
    }
};

// What request b's query tokens can see: positions [0, sinks) and [lo, L) (sinks = 0
// when the two meet).  Groups are counted as if all this ended at a.past: what lies past the
// tables is still looked at, and reported, but a length that cannot be costs no more than
// the tables' own.  (Up to a.past a window may lie behind what is missing, and is counted as
// it is.)
struct Visible {
    int L, first;  // length, position of query token 0 (may be negative)
    bool ends;     // sinks and window apart
    Counter cs, cl, ch;
    __device__ __forceinline__ Visible(int len, const StreamArgs& a)
        : L(len), first(len - a.q_len), ends(false), cs(0, a), cl(0, a), ch((uint32_t)min(len, a.past), a) {
        const int lo = a.window > first ? 0 : first - a.window + 1;
        if (lo > a.sinks) {
            ends = true;
            cs = Counter((uint32_t)min(a.sinks, a.past), a);
            cl = Counter((uint32_t)(len > a.past ? min(lo, a.past0) : lo), a);
        }
    }
    // groups of the shard at `off`: [0, sg) and [w0, w1)
    __device__ __forceinline__ void groups(uint32_t off, const StreamArgs& a, int* sg, int* w0, int* w1) const {
        const uint32_t I = (uint32_t)a.interleave;
        *w1 = (ch.of(off, I) + kTok - 1) / kTok;
        *sg = *w0 = 0;
        if (ends) {
            const int lo = cl.of(off, I), hi = ch.of(off, I);
            *sg = (cs.of(off, I) + kTok - 1) / kTok;
            *w0 = max(lo / kTok, *sg);
            *w1 = lo == hi ? *w0 : max(*w0, *w1);  // a shard may own none of the window: nothing of it is read
        }
    }
    // all groups of shards [lo, hi)
    __device__ __forceinline__ int count(int lo, int hi, const StreamArgs& a) const {
        int g = 0;
        uint64_t off = (uint64_t)(uint32_t)lo * (uint32_t)a.interleave;  // saturated as a.in is
        for (int n = lo; n < hi; n++) {
            int sg, w0, w1;
            groups(off > 0xffffffffu ? 0xffffffffu : (uint32_t)off, a, &sg, &w0, &w1);
            g += sg + w1 - w0;
            off += (uint32_t)a.interleave;
        }
        return g;
    }
};

__device__ __forceinline__ int length_of(const StreamArgs& a, int b) { return max(0, __ldg(a.seq_lens + b)); }

// groups of base (block of shards, request); at least 1, so that every row is written
__device__ __forceinline__ int base_groups(const StreamArgs& a, int base) {
    const int blk = a.per_shard ? base / a.batch : 0;
    const Visible v(length_of(a, base - blk * a.batch), a);
    const int lo = a.shard_lo + blk, hi = a.per_shard ? lo + 1 : a.shard_hi;
    return max(v.count(lo, hi, a), 1);
}

// A group: byte offset of its first row's codes in the pools (4-bit) or its index
// page * hkv + head (bf16), -1: no page; position of its first token; which tokens some
// row sees (all when every row sees the whole group); its first row in the page.
struct __align__(16) Desc {
    int64_t off;
    int32_t p0;
    uint16_t live, sub;
};

// Position of token e of a group whose first token's is p0: one further for each token,
// and past the other shards' runs where this shard's run ends.
__device__ __forceinline__ int64_t position_in(const StreamArgs& a, int p0, int e) {
    const uint32_t I = (uint32_t)a.interleave;
    const uint32_t runs = ((uint32_t)p0 % I + (uint32_t)e) / I;
    return (int64_t)p0 + e + (int64_t)runs * ((int64_t)a.in - I);
}

__device__ __forceinline__ bool sees(const StreamArgs& a, int64_t p, int at) {
    return p <= at && (p < a.sinks || at - p < a.window);
}

// Where group i of the visible groups of shards [lo, hi) lies (shard < 0: nowhere).
struct Place {
    int shard, t0;
};
__device__ __forceinline__ Place place_of(const StreamArgs& a, const Visible& v, int lo, int hi, int i) {
    uint64_t off = (uint64_t)(uint32_t)lo * (uint32_t)a.interleave;
    for (int n = lo; n < hi; n++) {
        int sg, w0, w1;
        v.groups(off > 0xffffffffu ? 0xffffffffu : (uint32_t)off, a, &sg, &w0, &w1);
        if (i < sg + w1 - w0) return Place{n, kTok * (i < sg ? i : w0 + i - sg)};
        i -= sg + w1 - w0;
        off += (uint32_t)a.interleave;
    }
    return Place{-1, 0};
}

// Its block-table entry; -1 past the table.
__device__ __forceinline__ int page_at(const StreamArgs& a, const Place& at, int b) {
    const int j = at.t0 >> (a.page_size == 16 ? 4 : 6);
    if (at.shard < 0 || j >= a.max_local_pages) return -1;
    return __ldg(a.block_tables + ((int64_t)(at.shard - a.bt_shard0) * a.batch + b) * a.max_local_pages + j);
}

// Its descriptor for KV head g; *full: every query token sees all of it.  block: bytes
// of a KV head's block (4-bit), or 0.
__device__ __forceinline__ Desc describe(const StreamArgs& a, const Visible& v, const Place& at, int pg, int g,
                                         int block, int row_bytes, bool* full) {
    Desc d{-1, 0, 0, 0};
    if (at.shard < 0) return d;
    if (pg < 0 || pg >= a.num_pages) {
        record_status(a.status, DCP_ERR_UNALLOCATED_PAGE);
        return d;
    }
    d.sub = (uint16_t)(at.t0 & (a.page_size - 1));
    d.off = (int64_t)pg * a.hkv + g;
    if (block) d.off = d.off * block + d.sub * row_bytes;
    const uint32_t I = (uint32_t)a.interleave;
    const uint32_t q = (uint32_t)at.t0 / I;
    uint32_t r = (uint32_t)at.t0 - q * I;
    int64_t p = (int64_t)q * a.in + (int64_t)at.shard * I + r;
    d.p0 = (int)p;  // a group has a token that counts, so its first one's position is below the length
    const int64_t p1 = p + (kTok - 1) + (int64_t)((r + kTok - 1) / I) * ((int64_t)a.in - I);
    *full = p1 <= v.first && (p1 < a.sinks || (int64_t)v.L - 1 - p < a.window);
    if (*full) {
        d.live = 0xffffu;
        return d;
    }
    for (int e = 0; e < kTok; e++) {
        if (p < v.L && (p < a.sinks || v.first - p < a.window)) d.live |= (uint16_t)(1u << e);
        p++;
        if (++r == I) {  // on to the shard's next run of positions
            r = 0;
            p += (int64_t)a.in - I;
        }
    }
    return d;
}

// Equal shares of the flat list of all segments' groups (each segment with a.lead
// groups before its own, what it costs beside them).
struct Share {
    long long total, r0, r1;  // all, and this team's [r0, r1)
    int active;               // teams that have a share
    int base, sub, x0;        // where r0 lies: base (block of shards, request), segment of the base, place in it
};

template <int WARPS>
struct ShareScratch {
    long long scan[WARPS];
    int base[WARPS], sub[WARPS], x0[WARPS];
};

// Executed by all WARPS warps of a block that holds `teams` teams; `least` groups to a share.
template <int WARPS>
__device__ __forceinline__ Share find_share(const StreamArgs& a, int nb, int per_base, int teams, int team,
                                            long long least, ShareScratch<WARPS>& sm) {
    constexpr int kN = 32 * WARPS;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int worker = blockIdx.x * teams + team;
    // every block sums all bases' groups, a run of consecutive bases for each thread
    const int each = (nb + kN - 1) / kN;
    const int b0 = min(nb, (int)threadIdx.x * each), b1 = min(nb, b0 + each);
    long long mine = 0;
    int first_groups = 0;  // of base b0
    for (int b = b0; b < b1; b++) {
        const int g = base_groups(a, b);
        if (b == b0) first_groups = g;
        mine += (long long)(g + a.lead) * per_base;
    }
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long t = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += t;
    }
    if (lane == 31) sm.scan[warp] = incl;
    __syncthreads();
    Share s{0, 0, 0, 0, 0, 0, 0};
    for (int w = 0; w < WARPS; w++) {
        if (w < warp) incl += sm.scan[w];
        s.total += sm.scan[w];
    }
    s.active = (int)min((long long)a.workers, (s.total + least - 1) / least);
    for (int t = 0; t < teams; t++) {
        const int w = blockIdx.x * teams + t;
        if (w >= s.active) break;
        long long at = s.total * w / s.active - (incl - mine);
        if (at < 0 || at >= mine) continue;
        for (int b = b0; b < b1; b++) {
            const int g = (b == b0 ? first_groups : base_groups(a, b)) + a.lead;
            const long long size = (long long)g * per_base;
            if (at < size) {
                sm.base[t] = b;
                sm.sub[t] = (int)(at / g);
                sm.x0[t] = (int)(at % g);
                break;
            }
            at -= size;
        }
    }
    __syncthreads();
    if (worker < s.active) {
        s.r0 = s.total * worker / s.active;
        s.r1 = s.total * (worker + 1) / s.active;
        s.base = sm.base[team];
        s.sub = sm.sub[team];
        s.x0 = sm.x0[team];
    }
    return s;
}

// The worker whose share holds the last group of a segment that ends (exclusively) at `end`.
__device__ __forceinline__ int last_worker(const Share& s, long long end) {
    return (int)((end * s.active + s.total - 1) / s.total) - 1;
}

// Lengths that cannot be: reported once (a length below 0 counts as 0, and query tokens
// before the first position see nothing).
__device__ __forceinline__ void check_lengths(const StreamArgs& a) {
    if (blockIdx.x != 0) return;
    for (int b = threadIdx.x; b < a.batch; b += blockDim.x) {
        const int L = __ldg(a.seq_lens + b);
        if (L < 0 || (L > 0 && L < a.q_len)) record_status(a.status, DCP_ERR_INVALID_ARG);
    }
}

// Where a row of a segment goes.
struct Row {
    float* o;
    float* lse;
};

// Output row r of segment (base, g, tile): the caller's tensors.
__device__ __forceinline__ Row out_row(const StreamArgs& a, int base, int g, int tile, int r, int D) {
    const int rr = tile * kRows + r, j = rr / a.group, h = rr - j * a.group;
    const int64_t at = ((int64_t)base * a.q_len + j) * a.hq + g * a.group + h;
    return Row{a.out + at * D, a.lse + at};
}

__device__ __forceinline__ void record_finish(const StreamArgs& a, int b) {
    const uint64_t dt = global_timer_ns() - (uint64_t)*a.t_start;
    atomicMax(reinterpret_cast<unsigned long long*>(a.finish_ns + b), (unsigned long long)dt);
}

// 4-bit operands
__device__ __forceinline__ void e2m1x8(uint32_t w, uint32_t* h) {  // four bytes, two values each -> four f16x2
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}
__device__ __forceinline__ uint32_t e4m3x2(uint32_t w) {  // low two bytes -> f16x2, exact
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)w, __NV_E4M3);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// Power of two that brings a row whose largest magnitude is amax into [1, 2), and its inverse.
__device__ __forceinline__ float2 row_power(float amax) {
    int e = (int)(__float_as_uint(amax) >> 23) - 127;
    e = (e > 127 || amax == 0.f) ? 0 : min(126, max(-126, e));
    return make_float2(__uint_as_float((uint32_t)(127 - e) << 23), __uint_as_float((uint32_t)(127 + e) << 23));
}

}  // namespace dcp
