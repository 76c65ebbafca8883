"""64-bit references of the cache operators (4-bit cache, windowed attention, norm and
rotation), written from their definitions in numpy, and a small sharded cache that is
filled without the library: a paging, packing or masking mistake cannot cancel out."""
from __future__ import annotations

import math

import numpy as np
import torch

import sequence_sharded_paged_b200 as dcp

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
_c = np.arange(127)
_e = _c // 8
E4M3 = np.where(_e == 0, _c * 2.0 ** -9, 2.0 ** (_e - 7.0) * (1 + (_c - 8 * _e) / 8))  # code c's magnitude


def bf16(x) -> np.ndarray:
    """float64 values rounded to bf16 (nearest even), as float64."""
    return torch.as_tensor(np.asarray(x, np.float64)).to(torch.float32).to(torch.bfloat16).double().numpy()


def nearest(a, grid) -> np.ndarray:
    """Index of the nearest grid value, ties to the even index, saturating."""
    a = np.asarray(a, np.float64)
    hi = np.clip(np.searchsorted(grid, a), 1, len(grid) - 1)
    down, up = a - grid[hi - 1], grid[hi] - a
    return np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, hi - 1)


def quantise4(x, factor=1.0, nudge=0.0):
    """Rows [..][d] -> (codes [..][d] in 0..15, scale bytes [..][d/16], values [..][d]).
    nudge: relative shift of every quotient before it is rounded to the grid."""
    x = np.asarray(x, np.float64)
    r = x.reshape(*x.shape[:-1], x.shape[-1] // 16, 16)
    with np.errstate(invalid="ignore"):
        amax = np.abs(r).max(-1)                      # a NaN stays
        nan = np.isnan(amax)
        sb = np.where(nan, 0x7F, nearest(np.where(nan, 0.0, amax / (6 * factor) * (1 + nudge)), E4M3))
        scale = np.where(nan, np.nan, E4M3[np.where(nan, 0, sb)] * factor)[..., None]
        ok = scale > 0
        y = np.where(ok, np.abs(r) / np.where(ok, scale, 1.0) * (1 + nudge), 0.0)
        code = np.where(ok, nearest(y, E2M1), 0)
        val = np.where(r < 0, -1.0, 1.0) * E2M1[code] * scale
    code = code | np.where(ok & (r < 0), 8, 0)
    return code.reshape(x.shape).astype(np.uint8), sb.astype(np.uint8), val.reshape(x.shape)


class Cache:
    """A sharded GQA cache of B requests whose rows are `k`, `v` (lists of float64
    [L_b][hkv][d]); whatever is not a stored row holds NaN (bf16) or NaN scales (4-bit)."""

    def __init__(self, dtype, k, v, *, hq, hkv, d, page, n, i, scale=None, factor=None, seed=0, spare=3, only=None,
                 room=0, drop=None):
        self.dtype, self.hq, self.hkv, self.d, self.page, self.n, self.i = dtype, hq, hkv, d, page, n, i
        self.k, self.v = [np.array(x) for x in k], [np.array(x) for x in v]
        self.scale = 1 / math.sqrt(d) if scale is None else scale
        self.factor = factor or (1.0, 1.0)
        B = len(k)
        L = np.array([len(x) for x in k], np.int64)
        self.lengths = L
        rng = np.random.default_rng(seed)
        shards = range(n) if only is None else [only]
        counts = np.array([[sum(1 for p in range(L[b]) if (p // i) % n == s) for b in range(B)] for s in shards])
        need = -(-(counts + room) // page)
        self.num_pages = int(need.sum()) + spare
        perm = rng.permutation(self.num_pages)
        bt = np.full((len(counts), B, max(1, int(need.max(initial=1)))), -1, np.int32)
        at = 0
        for s in range(len(counts)):
            for b in range(B):
                bt[s, b, :need[s, b]] = perm[at:at + need[s, b]]
                at += need[s, b]
        P, blk = page, page * (d // 2 + d // 16)
        if dtype == "bf16":
            pools = [np.full((self.num_pages, hkv, P, d), np.nan) for _ in range(2)]
        else:
            pools = [np.full((self.num_pages, hkv, blk), 0xFF, np.uint8) for _ in range(2)]
            stored = []
        for which, rows in enumerate((self.k, self.v)):
            for b in range(B):
                if dtype == "fp4":
                    code, sb, val = quantise4(rows[b], self.factor[which])
                    rows[b] = val
                for p in range(L[b]):
                    s = (p // i) % n
                    if only is not None and s != only:
                        continue
                    loc = (p // (i * n)) * i + p % i
                    pg, off = bt[0 if only is not None else s, b, loc // P], loc % P
                    if drop is not None and drop(b, p):
                        continue
                    if dtype == "bf16":
                        pools[which][pg, :, off] = rows[b][p]
                    else:
                        packed = code[p][:, 0::2] | (code[p][:, 1::2] << 4)
                        pools[which][pg, :, off * (d // 2):(off + 1) * (d // 2)] = packed
                        pools[which][pg, :, P * (d // 2) + np.arange(d // 16) * P + off] = sb[p].T
        if drop is not None:  # pages that hold dropped rows only are given up
            kept = np.zeros(bt.shape, bool)
            for b in range(B):
                for p in range(L[b]):
                    s = (p // i) % n
                    if not drop(b, p) and (only is None or s == only):
                        kept[0 if only is not None else s, b, ((p // (i * n)) * i + p % i) // P] = True
            bt[~kept] = -1
        if dtype == "bf16":
            dev = [torch.as_tensor(x).to(torch.float32).to(torch.bfloat16).cuda() for x in pools]
        else:
            dev = [torch.as_tensor(x).cuda() for x in pools]
        self.k_pages, self.v_pages = dev
        self.bt = torch.as_tensor(bt).cuda()
        self.kv_scales = None if factor is None else torch.tensor(list(factor) + [0, 0], dtype=torch.float32).cuda()
        self.seq_lens = torch.as_tensor(L.astype(np.int32)).cuda()
        self.desc = self.make_desc()

    def make_desc(self):
        return dcp.make_cache_desc(
            kind=dcp.DCP_GQA, dtype=dcp.DCP_BF16 if self.dtype == "bf16" else dcp.DCP_FP4_E2M1, n_shards=self.n,
            interleave=self.i, page_size=self.page, num_pages=self.num_pages, hq=self.hq, hkv=self.hkv, dk=self.d,
            dv=self.d, scale=self.scale, batch=len(self.k), block_tables=self.bt, k_pages=self.k_pages,
            v_pages=self.v_pages, kv_scales=self.kv_scales)


def rows(rng, L, hkv, d, gain=1.0):
    """bf16 values [L][hkv][d] as float64."""
    return bf16(rng.standard_normal((L, hkv, d)) * gain)


def attention(cache, q, *, window=None, sinks=0, shard=None):
    """q float64 [B][q_len][hq][d] -> (out, lse) in float64; 0 and -inf where nothing is seen."""
    B, ql, hq, d = q.shape
    G = hq // cache.hkv
    out, lse = np.zeros((B, ql, hq, d)), np.full((B, ql, hq), -np.inf)
    for b in range(B):
        for j in range(ql):
            at = int(cache.lengths[b]) - ql + j
            pos = np.arange(max(0, at + 1))
            if window is not None:
                pos = pos[(pos < sinks) | (pos > at - window)]
            if shard is not None:
                pos = pos[(pos // cache.i) % cache.n == shard]
            if not len(pos):
                continue
            for h in range(hq):
                K, V = cache.k[b][pos, h // G], cache.v[b][pos, h // G]
                s = (K @ q[b, j, h]) * cache.scale
                m = s.max()
                if not np.isfinite(m):
                    if np.isneginf(m):
                        continue
                p = np.exp(s - m)
                out[b, j, h] = (p @ V) / p.sum()
                lse[b, j, h] = m + np.log(p.sum())
    return out, lse


# Error bounds of the streamed decode kernel against 64 bits, for the tests' sizes (head
# size <= 128, at most 4096 visible tokens, sum |q_i k_i| scale <= 16 nats):
#  - a score is at most D/16 = 8 accumulations of exact products, each cut off below
#    2^-23 of a partial sum that is at most 16 nats: 8 * 16 * 2^-23 = 1.6e-5 nats; the
#    scaled argument of the exponential (|x| <= 64 in log2) is rounded to 2^-24 * 64 =
#    3.9e-6; the exponential itself to 2^-22: together under 2.1e-5 of a weight;
#  - a weight's terms leave out under 2^-21; the accumulation over n <= 3 * 256 / 4 steps
#    for each warp cuts off under 192 * 2^-23 = 2.3e-5 of O, and as much of the sum of the
#    weights;
#  - LSE carries the score's 1.6e-5, the weights' 2.1e-5, and its own rounding, 2^-23 of
#    at most 32.
# So |O - O_ref| <= (2 * 2.1e-5 + 2 * 2.3e-5) max|V| < 1e-4 max|V|, |LSE - ref| < 5e-5.
TOL_O, TOL_LSE = 1e-4, 5e-5


def check(name, out, lse, O, L, vmax):
    out, lse = out.double().cpu().numpy().reshape(O.shape), lse.double().cpu().numpy().reshape(L.shape)
    assert np.isfinite(out).all(), f"{name}: non-finite output"
    assert np.array_equal(np.isneginf(lse), np.isneginf(L)), f"{name}: which rows see nothing"
    none = np.isneginf(L)
    assert (out[none] == 0).all(), f"{name}: rows that see nothing are not 0"
    d_o = np.abs(out - O).max()
    d_l = np.abs(lse[~none] - L[~none]).max() if (~none).any() else 0.0
    assert d_o <= TOL_O * vmax, f"{name}: max|dO| = {d_o:.2e}, bound {TOL_O * vmax:.2e}"
    assert d_l <= TOL_LSE, f"{name}: max|dLSE| = {d_l:.2e}, bound {TOL_LSE:.2e}"


# ----------------------------------------------------------------------------
# norm and rotation
# ----------------------------------------------------------------------------

def frequencies(rot, theta, scaling="none", factor=1.0, original=0.0, low=1.0, high=32.0):
    """(radians per position of each pair, default factor on cosine and sine)."""
    f = []
    base = theta * factor ** (rot / (rot - 2)) if scaling == "base" else theta
    for k in range(rot // 2):
        w = base ** (-2 * k / rot)
        if scaling == "linear":
            w /= factor
        elif scaling == "yarn":
            def index(turns):
                return rot * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))
            lo, hi = max(math.floor(index(high)), 0), min(math.ceil(index(low)), rot - 1)
            r = min(max((k - lo) / max(hi - lo, 0.001), 0.0), 1.0)
            w = w * (1 - r) + w / factor * r
        elif scaling == "smooth":
            r = min(max((original * w / (2 * math.pi) - low) / (high - low), 0.0), 1.0)
            w = w * r + w / factor * (1 - r)
        f.append(w)
    return np.array(f), (0.1 * math.log(factor) + 1 if scaling == "yarn" else 1.0)


def rotate(x, pos, f, factor, layout):
    """x [T][heads][rot] -> rotated, in float64 (angles reduced with 128-bit fractions)."""
    from fractions import Fraction
    T, _, rot = x.shape
    # p * f modulo a turn, exactly from the double f: f / (2 pi) as a fraction of 2^-128
    two_pi = Fraction(6283185307179586476925286766559005768394, 10 ** 39)
    turns = [int(Fraction(w) / two_pi * 2 ** 128) for w in f]
    ang = np.array([[((int(p) * t) % 2 ** 128) / 2 ** 128 * 2 * math.pi for t in turns] for p in pos])
    c, s = np.cos(ang)[:, None] * factor, np.sin(ang)[:, None] * factor
    if layout == "half":
        a, z = x[..., :rot // 2], x[..., rot // 2:]
        return np.concatenate((a * c - z * s, z * c + a * s), -1)
    a, z = x[..., 0::2], x[..., 1::2]
    return np.stack((a * c - z * s, z * c + a * s), -1).reshape(x.shape)


def norm(x, w, eps):
    return x if w is None else x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
