"""What is measured of the cache operators: cases, inputs, plain forms and 64-bit results.

Four operators around one decode step over a sequence-sharded paged KV cache:

* ``decode4``  decode attention over a cache held in 4 bits (e2m1 codes, one e4m3 scale for each 16
  values), every shard merged;
* ``window``   decode attention that sees a sliding window and a few first tokens (sinks), over a bf16
  or a 4-bit cache;
* ``rope``     norms of queries and keys for each head and the rotation of their positions, in one pass
  that writes the keys and values into their owners' pages;
* ``append4``  rows quantised into the 4-bit cache and read back from it.

``own`` chooses between the plain form (elementary torch operations in 32 bits) and the calls of
``sequence_sharded_paged_b200``.  Lengths and positions follow from the case alone, values from the seed.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

# e2m1: bit 3 the sign, bits 2..0 the magnitude
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DEV = "cuda"


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------

def listed():
    return [
        # the tiny GQA workload (head size 64, page 16, two shards), with its cache in 4 bits: a call's latency
        _decode4("4-bit decode, two short requests", B=2, lo=300, hi=1000, hq=8, hkv=2, d=64, page=16, n=2, i=1),
        # a serving batch of chat-like lengths, from a few tokens to a few thousand, eight heads a group
        _decode4("4-bit decode, mixed short batch", B=48, lo=1, hi=16000, hq=64, hkv=8, d=128, page=64, n=4, i=16),
        # the long-context GQA workload (64 / 4 heads, page 16, eight shards, interleave 128), fewer requests
        _decode4("4-bit decode, long batch", B=24, lo=32000, hi=128000, hq=64, hkv=4, d=128, page=16, n=8, i=128),
        # one conversation behind a narrow window: a call's latency
        _window("window 128, one request", "bf16", B=1, lo=1000, hi=1000, window=128, sinks=4, hq=8, hkv=2, d=64,
                page=16, n=2, i=1),
        # the long-context GQA batch of a layer with a window
        _window("window 4096, long batch", "bf16", B=128, lo=32000, hi=128000, window=4096, sinks=4, hq=64, hkv=4,
                d=128, page=16, n=8, i=128),
        # four tokens to verify for each request (speculative decoding), 4-bit cache, odd window
        _window("window 1021, four tokens, 4-bit", "fp4", B=64, lo=200, hi=40000, window=1021, sinks=3, q_len=4,
                hq=32, hkv=8, d=128, page=64, n=4, i=64),
        # one long document behind a wide window: few heads, so the length has to be split
        _window("window 65536, one request", "bf16", B=1, lo=200000, hi=200000, window=65536, sinks=16, hq=64,
                hkv=4, d=128, page=16, n=8, i=128),
        # the new token of each request of the long-context GQA batch
        _rope("norm and rotate, one token each", "gqa", T=128, B=128, far=128000, hq=64, hkv=4, d=128, page=16, n=8,
              i=128, rot=128, layout="half", norm=True),
        # chunks of prompts
        _rope("norm and rotate, prompt chunks", "gqa", T=16384, B=13, far=1000000, hq=64, hkv=4, d=128, page=16, n=8,
              i=128, rot=64, layout="half", norm=True, scaling="smooth"),
        # latent rows and absorbed queries of the MLA workload, long-context frequencies
        _rope("latent norm and rotate, prompt chunk", "mla", T=4001, B=3, far=120000, hq=64, hkv=1, d=576, page=64,
              n=8, i=1, rot=64, layout="interleaved", norm=True, scaling="yarn"),
        # a decode step's rows
        _append4("4-bit append and read, one token each", T=128, B=128, far=128000, hkv=4, d=128, page=16, n=8, i=128),
        # prompt rows
        _append4("4-bit append and read, prompts", T=50021, B=7, far=30000, hkv=8, d=128, page=64, n=4, i=16),
    ]


def _decode4(name, B, lo, hi, hq, hkv, d, page, n, i, q_len=1, lens=11):
    return {"name": name, "op": "decode4", "dtype": "fp4", "B": B, "lo": lo, "hi": hi, "q_len": q_len, "window": 0,
            "sinks": 0, "hq": hq, "hkv": hkv, "d": d, "page": page, "n": n, "i": i, "lens": lens}


def _window(name, dtype, B, lo, hi, window, sinks, hq, hkv, d, page, n, i, q_len=1, lens=12):
    return {"name": name, "op": "window", "dtype": dtype, "B": B, "lo": lo, "hi": hi, "q_len": q_len,
            "window": window, "sinks": sinks, "hq": hq, "hkv": hkv, "d": d, "page": page, "n": n, "i": i, "lens": lens}


def _rope(name, kind, T, B, far, hq, hkv, d, page, n, i, rot, layout, norm, scaling="none", lens=13):
    return {"name": name, "op": "rope", "kind": kind, "T": T, "B": B, "far": far, "hq": hq, "hkv": hkv, "d": d,
            "page": page, "n": n, "i": i, "rot": rot, "layout": layout, "norm": norm, "scaling": scaling, "lens": lens}


def _append4(name, T, B, far, hkv, d, page, n, i, lens=14):
    return {"name": name, "op": "append4", "T": T, "B": B, "far": far, "hkv": hkv, "d": d, "page": page, "n": n,
            "i": i, "lens": lens}


def _log(rng, lo, hi):
    """A whole number from lo to hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["decode4", "window", "rope", "append4"])
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 8])
    page = rng.choice([16, 64])
    n = rng.choice([1, 2, 3, 4, 8])
    i = rng.choice([1, 16, 64, 128, rng.randint(2, 150)])
    lens = rng.randint(1, 1 << 20)
    if op in ("decode4", "window"):
        group = rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 12, 16])
        q_len = rng.choice([1, 1, 1, 2, 4])
        B = _log(rng, 1, 160)
        if op == "decode4":
            most = max(1, min(128000, int(1.9e6 * 4 * 128 / (B * hkv * d * q_len))))  # tokens of a request
            hi = max(q_len, _log(rng, 1, most))
            lo = max(q_len, _log(rng, 1, hi))
            c = _decode4("", B, lo, hi, hkv * group, hkv, d, page, n, i, q_len, lens)
        else:
            most = max(1, min(65536, int(128 * 4096 * 4 * 128 / (B * hkv * d * q_len))))  # visible tokens of a request
            window = _log(rng, 1, most)
            sinks = rng.choice([0, 1, 4, rng.randint(0, 64)])
            hi = max(q_len, _log(rng, 1, min(128000, int(1.2e7 * 4 * 128 / (B * hkv * d)))))
            lo = max(q_len, _log(rng, 1, hi))
            c = _window("", rng.choice(["bf16", "fp4"]), B, lo, hi, window, sinks, hkv * group, hkv, d, page, n, i,
                        q_len, lens)
    elif op == "rope":
        if rng.random() < 0.35:
            T = _log(rng, 1, 8000)
            c = _rope("", "mla", T, rng.randint(1, min(T, 64)), _log(rng, 64, 1000000), rng.choice([16, 32, 64]), 1,
                      576, 64, n, i, 64, rng.choice(["half", "interleaved"]), rng.random() < 0.7,
                      rng.choice(["none", "linear", "base", "yarn", "smooth"]), lens)
        else:
            group = rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 12, 16])
            T = _log(rng, 1, max(1, 16384 * 72 * 128 // (hkv * (group + 2) * d)) // 2)
            rot = rng.choice([d, d // 2, d // 4])
            c = _rope("", "gqa", T, rng.randint(1, min(T, 64)), _log(rng, 64, 1000000), hkv * group, hkv, d, page, n,
                      i, rot, rng.choice(["half", "interleaved"]), rng.random() < 0.7,
                      rng.choice(["none", "linear", "base", "yarn", "smooth"]), lens)
    else:
        T = _log(rng, 1, 50000 * 8 * 128 // (hkv * d) // 2)
        c = _append4("", T, rng.randint(1, min(T, 64)), _log(rng, 64, 60000), hkv, d, page, n, i, lens)
    del c["name"]
    return c


# ----------------------------------------------------------------------------
# lengths, positions and block tables (from the case alone)
# ----------------------------------------------------------------------------

def _lengths(case):
    r = np.random.RandomState(case["lens"])
    lo, hi = case["lo"], case["hi"]
    if hi < 4 * lo:
        return r.randint(lo, hi + 1, case["B"]).astype(np.int64)
    u = r.uniform(math.log(lo), math.log(hi), case["B"])
    return np.clip(np.round(np.exp(u)), lo, hi).astype(np.int64)


def _new_tokens(case):
    """(request, position) of the T new tokens: a run of consecutive positions for each request."""
    r = np.random.RandomState(case["lens"])
    T, B = case["T"], case["B"]
    cut = np.sort(r.choice(np.arange(1, T), B - 1, replace=False)) if B > 1 else np.zeros(0, np.int64)
    each = np.diff(np.concatenate([[0], cut, [T]])).astype(np.int64)
    start = r.randint(0, case["far"], B).astype(np.int64)
    req = np.repeat(np.arange(B), each)
    at = np.arange(T) - np.repeat(np.cumsum(each) - each, each)
    return req.astype(np.int32), (start[req] + at).astype(np.int32), start, each


def _counts(x, n, i):
    """Positions p < x_b that shard s owns, [n][B]."""
    x = np.asarray(x, np.int64)
    s = np.arange(n, dtype=np.int64)[:, None]
    return (x // (i * n)) * i + np.clip(x % (i * n) - s * i, 0, i)


def _tables(case, r, first, last):
    """Block tables [n][B][pages] for the positions [first_b, last_b) of each request; -1 elsewhere."""
    n, i, page = case["n"], case["i"], case["page"]
    a, z = _counts(first, n, i) // page, -(-_counts(last, n, i) // page)
    need = np.maximum(z - a, 0)
    total = int(need.sum())
    perm = r.permutation(total).astype(np.int32)
    bt = np.full((n, len(first), max(1, int(z.max()))), -1, np.int32)
    at = 0
    for s in range(n):
        for b in range(len(first)):
            k = int(need[s, b])
            bt[s, b, a[s, b]:a[s, b] + k] = perm[at:at + k]
            at += k
    return bt, max(1, total)


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------

def _normal(g, shape, gain=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * gain).to(torch.bfloat16)


def _block_bytes(case):
    return case["page"] * (case["d"] // 2 + case["d"] // 16)


def _fill4(g, case, pages):
    """Pages [pages][hkv][bytes] of quantised normal values."""
    hkv, page, d = case["hkv"], case["page"], case["d"]
    out = torch.empty((pages, hkv, _block_bytes(case)), dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 26) // (hkv * page * d))
    for a in range(0, pages, step):
        z = min(pages, a + step)
        x = torch.randn((z - a, hkv, page, d), generator=g, device=DEV)
        codes, scales = _quantise4(x)
        out[a:z, :, :page * d // 2] = codes.reshape(z - a, hkv, -1)
        out[a:z, :, page * d // 2:] = scales.transpose(2, 3).reshape(z - a, hkv, -1)
    return out


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    r = np.random.RandomState(case["lens"] + 1)
    s = {"case": case}
    if case["op"] in ("decode4", "window"):
        L = _lengths(case)
        first = np.zeros_like(L)
        if case["op"] == "window":  # only pages that some token can see are kept, and the sinks'
            first = np.maximum(0, L - case["q_len"] - case["window"] + 1)
        bt, pages = _tables(case, r, first, L)
        if case["op"] == "window" and case["sinks"]:
            sink_bt, more = _tables(case, r, np.zeros_like(L), np.minimum(case["sinks"], L))
            w = min(bt.shape[2], sink_bt.shape[2])
            free = (bt[:, :, :w] < 0) & (sink_bt[:, :, :w] >= 0)
            bt[:, :, :w][free] = sink_bt[:, :, :w][free] + pages
            pages += more
        s["lens"] = torch.as_tensor(L.astype(np.int32), device=DEV)
        s["most"] = int(L.max())
        s["q"] = _normal(g, (case["B"], case["q_len"], case["hq"], case["d"]), 1.5)
        if case["dtype"] == "fp4":
            s["k"], s["v"] = _fill4(g, case, pages), _fill4(g, case, pages)
        else:
            shape = (pages, case["hkv"], case["page"], case["d"])
            s["k"], s["v"] = _normal(g, shape), _normal(g, shape)
        s["out"] = torch.empty((case["B"], case["q_len"], case["hq"], case["d"]), device=DEV)
        s["lse"] = torch.empty((case["B"], case["q_len"], case["hq"]), device=DEV)
    else:
        req, pos, start, each = _new_tokens(case)
        bt, pages = _tables(case, r, start, start + each)
        s["req"], s["pos"] = torch.as_tensor(req, device=DEV), torch.as_tensor(pos, device=DEV)
        T, hkv, d = case["T"], case["hkv"], case["d"]
        if case["op"] == "append4":
            s["k_new"], s["v_new"] = _normal(g, (T, hkv, d)), _normal(g, (T, hkv, d))
            s["k"] = torch.zeros((pages, hkv, _block_bytes(case)), dtype=torch.uint8, device=DEV)
            s["v"] = torch.zeros_like(s["k"])
            s["k_out"], s["v_out"] = torch.empty_like(s["k_new"]), torch.empty_like(s["v_new"])
        elif case["kind"] == "gqa":
            # one projection's output, as a model has it: queries, keys and values of a token side by side
            hq = case["hq"]
            rows = _normal(g, (T, hq + 2 * hkv, d), 2.0)
            s["q"], s["k_new"], s["v_new"] = rows[:, :hq], rows[:, hq:hq + hkv], rows[:, hq + hkv:]
            s["k"] = torch.zeros((pages, hkv, case["page"], d), dtype=torch.bfloat16, device=DEV)
            s["v"] = torch.zeros_like(s["k"])
            s["qw"] = _normal(g, (d,), 0.2) + 1 if case["norm"] else None
            s["kw"] = _normal(g, (d,), 0.2) + 1 if case["norm"] else None
        else:
            s["q"] = _normal(g, (T, case["hq"], d))
            s["k_new"], s["v_new"] = _normal(g, (T, d), 2.0), None
            s["k"] = torch.zeros((pages, case["page"], d), dtype=torch.bfloat16, device=DEV)
            s["v"] = None
            s["qw"], s["kw"] = None, _normal(g, (512,), 0.2) + 1 if case["norm"] else None
        if case["op"] == "rope":
            s["q_out"] = torch.empty((T, case["hq"], d), dtype=torch.bfloat16, device=DEV)
    s["bt"] = torch.as_tensor(bt, device=DEV)
    s["pages"] = pages
    if own:
        import sequence_sharded_paged_b200 as dcp
        mla = case.get("kind") == "mla"
        four = case["op"] in ("decode4", "append4") or case.get("dtype") == "fp4"
        s["desc"] = dcp.make_cache_desc(
            kind=dcp.DCP_MLA if mla else dcp.DCP_GQA, dtype=dcp.DCP_FP4_E2M1 if four else dcp.DCP_BF16,
            n_shards=case["n"], interleave=case["i"], page_size=case["page"], num_pages=pages,
            hq=case.get("hq", case["hkv"]), hkv=case["hkv"], dk=case["d"], dv=512 if mla else case["d"],
            scale=1.0 / math.sqrt(192 if mla else case["d"]), batch=bt.shape[1], block_tables=s["bt"], k_pages=s["k"],
            v_pages=s["v"])
        if case["op"] == "decode4":
            size = dcp.dcp_decode_workspace_size_ex(s["desc"], case["B"], case["q_len"], dcp.DCP_DECODE_MERGED)
            s["ws"] = torch.empty(size, dtype=torch.uint8, device=DEV)
        elif case["op"] == "window":
            size = dcp.dcp_decode_window_workspace_size(s["desc"], case["B"], case["q_len"], case["window"],
                                                        case["sinks"])
            s["ws"] = torch.empty(size, dtype=torch.uint8, device=DEV)
        elif case["op"] == "rope":
            s["rope"] = dcp.make_rope(case["rot"], layout=case["layout"], **SCALING[case["scaling"]])
    return s


SCALING = {
    "none": {"theta": 1e6},
    "linear": {"theta": 1e4, "scaling": "linear", "factor": 4.0},
    "base": {"theta": 1e4, "scaling": "base", "factor": 8.0},
    "yarn": {"theta": 5e4, "scaling": "yarn", "factor": 32.0, "original": 4096, "low": 1.0, "high": 32.0},
    "smooth": {"theta": 5e5, "scaling": "smooth", "factor": 8.0, "original": 8192, "low": 1.0, "high": 4.0},
}


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------

def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import sequence_sharded_paged_b200 as dcp
    case = s["case"]
    if case["op"] == "decode4":
        dcp.dcp_decode_merged(s["desc"], s["q"], s["lens"], s["out"], s["lse"], s["ws"])
        return {"out": s["out"], "lse": s["lse"]}
    if case["op"] == "window":
        dcp.dcp_decode_window(s["desc"], s["q"], s["lens"], case["window"], case["sinks"], s["out"], s["lse"], s["ws"])
        return {"out": s["out"], "lse": s["lse"]}
    if case["op"] == "rope":
        dcp.dcp_norm_rope_append(s["desc"], s["rope"], s["req"], s["pos"], s["q"], s["k_new"], s["v_new"], s["qw"],
                                 s["kw"], 1e-6, s["q_out"])
        return {"q": s["q_out"], "k": s["k"], "v": s["v"]}
    dcp.dcp_kv_append(s["desc"], s["req"], s["pos"], s["k_new"], s["v_new"])
    dcp.dcp_kv_gather(s["desc"], s["req"], s["pos"], s["k_out"], s["v_out"])
    return {"k": s["k_out"], "v": s["v_out"]}


def _run_plain(s):
    case = s["case"]
    if case["op"] in ("decode4", "window"):
        return _plain_attention(s)
    if case["op"] == "rope":
        return _plain_rope(s)
    page, off = _place(s, s["req"].long(), s["pos"].long())
    got = {}
    for name in ("k", "v"):
        codes, scales = _split4(case, s[name])
        c, e = _quantise4(s[name + "_new"].float())
        codes[page, :, off] = c
        scales[page, :, :, off] = e
        got[name] = _read4(case, s[name], page, off).to(torch.bfloat16)
    return got


def _place(s, req, pos):
    """Page and offset of each position (clamped where a table has no page)."""
    n, i, P = s["case"]["n"], s["case"]["i"], s["case"]["page"]
    local = pos // (i * n) * i + pos % i
    j = (local // P).clamp(max=s["bt"].shape[2] - 1)
    return s["bt"][pos // i % n, req, j].long().clamp(min=0), local % P


def _split4(case, pages):
    """Views of 4-bit pages: codes [pages][hkv][P][d/2] and scales [pages][hkv][d/16][P]."""
    P, d = case["page"], case["d"]
    codes, scales = pages.split([P * d // 2, P * d // 16], dim=2)
    return codes.unflatten(2, (P, d // 2)), scales.unflatten(2, (d // 16, P))


def _quantise4(x):
    """Rows [..][d] in 32 bits -> codes [..][d/2] (two a byte, the first low) and e4m3 scale bytes [..][d/16]."""
    x = x.unflatten(-1, (-1, 16))
    scale = (x.abs().amax(-1, keepdim=True) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    f = scale.float()
    y = torch.where(f > 0, x / f, torch.zeros_like(x))
    a = y.abs()  # to the nearest of E2M1, ties to the even code
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75).to(torch.uint8) + (a > 1.25).to(torch.uint8) +
            (a >= 1.75).to(torch.uint8) + (a > 2.5).to(torch.uint8) + (a >= 3.5).to(torch.uint8) +
            (a > 5.0).to(torch.uint8)) | ((y < 0).to(torch.uint8) << 3)
    code = code.flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale.view(torch.uint8).flatten(-2)


def _read4(case, pages, page, off):
    """Values [..][hkv][d] in 32 bits of the rows at (page, off)."""
    codes, scales = _split4(case, pages)
    c = codes[page, :, off]
    lut = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=c.device)
    x = torch.stack((lut[(c & 15).int()], lut[(c >> 4).int()]), -1).flatten(-2)
    f = scales[page, :, :, off].contiguous().view(torch.float8_e4m3fn).float()
    return (x.unflatten(-1, (-1, 16)) * f.unsqueeze(-1)).flatten(-2)


def _plain_attention(s):
    case = s["case"]
    B, ql, hq, hkv, d = case["B"], case["q_len"], case["hq"], case["hkv"], case["d"]
    L = s["lens"].long()[:, None]
    b = torch.arange(B, device=DEV)[:, None]
    if case["op"] == "window":  # the sinks, then what the first token's window begins with
        k = torch.arange(min(s["most"], case["sinks"] + case["window"] + ql - 1), device=DEV)[None]
        start = (L - ql - case["window"] + 1).clamp(min=case["sinks"])
        pos = torch.where(k < case["sinks"], k, start + k - case["sinks"])
    else:
        pos = torch.arange(s["most"], device=DEV)[None].expand(B, -1)
    page, off = _place(s, b, pos)
    if case["dtype"] == "fp4":
        K, V = _read4(case, s["k"], page, off), _read4(case, s["v"], page, off)
    else:
        K, V = s["k"][page, :, off].float(), s["v"][page, :, off].float()
    q = s["q"].float().view(B, ql, hkv, hq // hkv, d).transpose(1, 2).reshape(B, hkv, -1, d)
    x = q @ K.permute(0, 2, 3, 1) / math.sqrt(d)                     # [B][hkv][ql * group][M]
    at = (L - ql + torch.arange(ql, device=DEV))[:, :, None]         # each query token's own position
    sees = (pos[:, None] <= at) & (pos[:, None] < L[:, :, None])
    if case["op"] == "window":
        sees &= (pos[:, None] < case["sinks"]) | (pos[:, None] > at - case["window"])
    sees = sees.repeat_interleave(hq // hkv, 1)[:, None]
    x = x.masked_fill(~sees, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - m.masked_fill(m == -math.inf, 0.0))
    total = p.sum(-1, keepdim=True)
    o = p @ V.transpose(1, 2) / total.clamp(min=1e-30)
    lse = m + torch.log(total)
    back = lambda t: t.view(B, hkv, ql, hq // hkv, -1).transpose(1, 2).reshape(B, ql, hq, -1)  # noqa: E731
    return {"out": back(o), "lse": back(lse).squeeze(-1)}


def _frequencies(case):
    """Radians per position of each rotated pair, in 64 bits, and the factor on cosine and sine."""
    c, rot = SCALING[case["scaling"]], case["rot"]
    k = torch.arange(rot // 2, dtype=torch.float64, device=DEV)
    theta, kind = c["theta"], c.get("scaling", "none")
    if kind == "base":
        theta *= c["factor"] ** (rot / (rot - 2))
    f = theta ** (-2 * k / rot)
    if kind == "linear":
        return f / c["factor"], 1.0
    if kind == "yarn":  # pairs that turn often keep their frequency, those that turn seldom are stretched
        edge = lambda turns: rot * math.log(c["original"] / (turns * 2 * math.pi)) / (2 * math.log(theta))  # noqa: E731
        lo, hi = max(math.floor(edge(c["high"])), 0), min(math.ceil(edge(c["low"])), rot - 1)
        ramp = ((k - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        return f / c["factor"] * ramp + f * (1 - ramp), 0.1 * math.log(c["factor"]) + 1
    if kind == "smooth":  # by how often a pair turns within the original length
        turns = c["original"] * f / (2 * math.pi)
        keep = ((turns - c["low"]) / (c["high"] - c["low"])).clamp(0, 1)
        return f * keep + f / c["factor"] * (1 - keep), 1.0
    return f, 1.0


def _plain_rotate(case, x, pos):
    """Rows [T][heads][rot] rotated by their positions."""
    f, factor = _frequencies(case)
    angle = pos.double()[:, None] * f
    cos, sin = (torch.cos(angle) * factor).float()[:, None], (torch.sin(angle) * factor).float()[:, None]
    if case["layout"] == "half":
        a, z = x.chunk(2, -1)
        return torch.cat((a * cos - z * sin, z * cos + a * sin), -1)
    a, z = x[..., 0::2], x[..., 1::2]
    return torch.stack((a * cos - z * sin, z * cos + a * sin), -1).flatten(-2)


def _plain_norm(x, w):
    return x if w is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.float()


def _plain_rope(s):
    case, pos = s["case"], s["pos"].long()
    rot = case["rot"]
    page, off = _place(s, s["req"].long(), pos)
    if case["kind"] == "gqa":
        q, k = _plain_norm(s["q"].float(), s["qw"]), _plain_norm(s["k_new"].float(), s["kw"])
        q = torch.cat((_plain_rotate(case, q[..., :rot], pos), q[..., rot:]), -1)
        k = torch.cat((_plain_rotate(case, k[..., :rot], pos), k[..., rot:]), -1)
        s["k"][page, :, off] = k.to(torch.bfloat16)
        s["v"][page, :, off] = s["v_new"]
    else:
        x = s["k_new"].float()
        q = s["q"].float()
        q = torch.cat((q[..., :512], _plain_rotate(case, q[..., 512:], pos)), -1)
        k = _plain_rotate(case, x[:, None, 512:], pos)[:, 0]
        s["k"][page, off] = torch.cat((_plain_norm(x[:, :512], s["kw"]), k), -1).to(torch.bfloat16)
    return {"q": q.to(torch.bfloat16), "k": s["k"], "v": s["v"]}


# ----------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------

def work(case):
    d, hkv = case["d"], case["hkv"]
    if case["op"] in ("decode4", "window"):
        L, ql, hq = _lengths(case), case["q_len"], case["hq"]
        seen = L if case["op"] == "decode4" else np.minimum(L, case["sinks"] + case["window"] + ql - 1)
        tokens = int(seen.sum())
        row = 2 * (d // 2 + d // 16) if case["dtype"] == "fp4" else 4 * d
        return {"bytes": tokens * hkv * row + case["B"] * ql * hq * (6 * d + 4) + 4 * tokens // case["page"],
                "flops": 4 * tokens * ql * hq * d}
    T = case["T"]
    if case["op"] == "append4":
        return {"bytes": T * (2 * hkv * (2 * 2 * d + 2 * (d // 2 + d // 16)) + 8), "flops": 8 * T * hkv * d}
    rows = case["hq"] + 2 * hkv if case["kind"] == "gqa" else case["hq"] + 1
    return {"bytes": T * (rows * d * 4 + 8), "flops": 8 * T * rows * d}


# ----------------------------------------------------------------------------
# the definition in 64 bits
# ----------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("decode4", "window"):
        return _exact_attention(case, s)
    return _exact_rope(case, s) if case["op"] == "rope" else _exact_append4(case, s)


def _exact_rows(case, s, name, b, pos):
    """Values [len(pos)][hkv][d] in 64 bits of request b's positions, read from its owners' pages."""
    n, i, P, d = case["n"], case["i"], case["page"], case["d"]
    pos = np.asarray(pos, np.int64)
    shard = (pos // i) % n
    within = (pos // (i * n)) * i + pos % i
    table = s["bt"].cpu().numpy()
    page = torch.as_tensor(table[shard, b, within // P].astype(np.int64), device=DEV)
    off = torch.as_tensor(within % P, device=DEV)
    if s[name].dtype == torch.bfloat16:
        return s[name][page, :, off].double()
    raw = s[name]
    byte = off[:, None] * (d // 2) + torch.arange(d // 2, device=DEV)
    two = raw[page[:, None, None], torch.arange(case["hkv"], device=DEV)[None, :, None], byte[:, None]].to(torch.int32)
    nibble = torch.stack((two % 16, two // 16), -1).flatten(-2)
    e, m = (nibble // 2) % 4, nibble % 2
    mag = torch.where(e == 0, 0.5 * m.double(), torch.exp2(e.double() - 1) * (1 + 0.5 * m.double()))
    at = P * d // 2 + torch.arange(d // 16, device=DEV)[None] * P + off[:, None]
    sb = raw[page[:, None, None], torch.arange(case["hkv"], device=DEV)[None, :, None], at[:, None]].to(torch.int32)
    se, sm = sb // 8, (sb % 8).double()
    scale = torch.where(se == 0, sm * 2.0 ** -9, torch.exp2(se.double() - 7) * (1 + sm / 8))
    return torch.where(nibble >= 8, -mag, mag) * scale.repeat_interleave(16, -1)


def _exact_attention(case, s):
    L, ql, hq, hkv, d = _lengths(case), case["q_len"], case["hq"], case["hkv"], case["d"]
    out = torch.zeros((case["B"], ql, hq, d), dtype=torch.float64, device=DEV)
    lse = torch.full((case["B"], ql, hq), -math.inf, dtype=torch.float64, device=DEV)
    for b in range(case["B"]):
        for j in range(ql):
            at = int(L[b]) - ql + j
            if at < 0:
                continue
            pos = np.arange(at + 1)
            if case["op"] == "window":
                pos = pos[(pos < case["sinks"]) | (pos > at - case["window"])]
            K, V = _exact_rows(case, s, "k", b, pos), _exact_rows(case, s, "v", b, pos)
            q = s["q"][b, j].double().view(hkv, hq // hkv, d)
            x = torch.einsum("ghd,mgd->ghm", q, K) / math.sqrt(d)
            lse[b, j] = torch.logsumexp(x, -1).flatten()
            out[b, j] = torch.einsum("ghm,mgd->ghd", torch.softmax(x, -1), V).reshape(hq, d)
    return {"out": out, "lse": lse}


def _exact_turn(case, x, pos):
    """x [T][heads][rot] in 64 bits, each pair turned as a complex number."""
    c, rot, factor = SCALING[case["scaling"]], case["rot"], 1.0
    f = []
    for k in range(rot // 2):
        base, kind = c["theta"], c.get("scaling", "none")
        if kind == "base":
            base = base * c["factor"] ** (rot / (rot - 2.0))
        w = math.exp(-2.0 * k / rot * math.log(base))
        if kind == "linear":
            w = w / c["factor"]
        elif kind == "yarn":
            lo = math.floor(rot * math.log(c["original"] / (c["high"] * 2 * math.pi)) / (2 * math.log(base)))
            hi = math.ceil(rot * math.log(c["original"] / (c["low"] * 2 * math.pi)) / (2 * math.log(base)))
            lo, hi = max(lo, 0), min(hi, rot - 1)
            share = min(max((k - lo) / max(hi - lo, 0.001), 0.0), 1.0)
            w = w * (1 - share + share / c["factor"])
            factor = 1 + 0.1 * math.log(c["factor"])
        elif kind == "smooth":
            share = min(max((c["original"] * w / (2 * math.pi) - c["low"]) / (c["high"] - c["low"]), 0.0), 1.0)
            w = w * (share + (1 - share) / c["factor"])
        f.append(w)
    angle = pos.double()[:, None] * torch.tensor(f, dtype=torch.float64, device=DEV)
    turn = torch.polar(torch.full_like(angle, factor), angle)[:, None]
    if case["layout"] == "half":
        z = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:].contiguous()) * turn
        return torch.cat((z.real, z.imag), -1)
    return torch.view_as_real(torch.view_as_complex(x.unflatten(-1, (-1, 2)).contiguous()) * turn).flatten(-2)


def _exact_rope(case, s):
    pos, rot, P = s["pos"], case["rot"], case["page"]

    def norm(x, w):
        return x if w is None else x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + 1e-6) * w.double()

    n, i = case["n"], case["i"]
    p = pos.cpu().numpy().astype(np.int64)
    within = (p // (i * n)) * i + p % i
    page = torch.as_tensor(s["bt"].cpu().numpy()[(p // i) % n, s["req"].cpu().numpy(), within // P].astype(np.int64),
                           device=DEV)
    row = page * P + torch.as_tensor(within % P, device=DEV)
    q = s["q"].double()
    if case["kind"] == "mla":
        q[..., 512:] = _exact_turn(case, q[..., 512:], pos)
        x = s["k_new"].double()
        x = torch.cat((norm(x[:, :512], s["kw"]), _exact_turn(case, x[:, None, 512:], pos)[:, 0]), -1)
        k = s["k"].double().view(-1, 576)
        k[row] = x
        return {"q": q, "k": k.view(s["k"].shape), "v": None}
    q, x = norm(q, s["qw"]), norm(s["k_new"].double(), s["kw"])
    q[..., :rot], x[..., :rot] = _exact_turn(case, q[..., :rot].clone(), pos), _exact_turn(case, x[..., :rot].clone(), pos)
    k, v = (s[name].double().transpose(1, 2).reshape(-1, case["hkv"], case["d"]) for name in ("k", "v"))
    k[row], v[row] = x, s["v_new"].double()
    back = lambda t: t.view(-1, P, case["hkv"], case["d"]).transpose(1, 2)  # noqa: E731
    return {"q": q, "k": back(k), "v": back(v)}


def _exact_append4(case, s):
    grid = torch.tensor(E2M1, dtype=torch.float64, device=DEV)
    # e4m3's 127 finite magnitudes, in order: code c's is grid8[c]
    c = torch.arange(127, dtype=torch.float64, device=DEV)
    e = torch.floor(c / 8)
    grid8 = torch.where(e == 0, c * 2.0 ** -9, torch.exp2(e - 7) * (1 + (c - 8 * e) / 8))

    def nearest(a, values):  # ties to the even code
        hi = torch.searchsorted(values, a.contiguous()).clamp(1, len(values) - 1)
        down, up = a - values[hi - 1], values[hi] - a
        return torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, hi - 1)

    got = {}
    for name in ("k", "v"):
        x = s[name + "_new"].double().unflatten(-1, (-1, 16))
        scale = grid8[nearest(x.abs().amax(-1, keepdim=True) / 6, grid8)]
        safe = torch.where(scale > 0, scale, torch.ones_like(scale))
        mag = grid[nearest(x.abs() / safe, grid)] * scale
        got[name] = torch.where(x < 0, -mag, mag).flatten(-2)
    return got
