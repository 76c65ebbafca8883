"""Decode attention under a sliding window with sinks (marked gpu) against 64 bits."""
import math

import numpy as np
import pytest
import torch

import sequence_sharded_paged_b200 as dcp

from op_ref import Cache, attention, bf16, check, rows

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clear_status():
    dcp.dcp_get_device_status()
    yield
    assert dcp.dcp_get_device_status() == dcp.DCP_OK


def to_bf16(x):
    return torch.as_tensor(x).to(torch.float32).to(torch.bfloat16).cuda()


def run(c, q, window, sinks, rank=None, ws=None, stream=None):
    B, ql, hq, d = q.shape
    out = torch.full((B, ql, hq, d), float("nan"), device="cuda")
    lse = torch.full((B, ql, hq), float("nan"), device="cuda")
    if ws is None:
        size = dcp.dcp_decode_window_workspace_size(c.desc, B, ql, window, sinks, rank=rank)
        assert size > 0
        ws = torch.full((size,), 0xCD, dtype=torch.uint8, device="cuda")
    dcp.dcp_decode_window(c.desc, q, c.seq_lens, window, sinks, out, lse, ws, rank=rank, stream=stream)
    return out, lse


SHAPES = [  # hq, hkv, d, page, n, i, lengths
    (8, 2, 64, 16, 2, 1, [300, 1000]),
    (8, 8, 64, 64, 1, 1, [1, 0, 130]),
    (6, 2, 128, 16, 3, 5, [77, 16, 15, 17]),
    (40, 8, 128, 64, 4, 16, [200, 65, 5]),
    (64, 4, 128, 16, 8, 128, [1500, 129, 0, 7]),
    (16, 1, 64, 64, 5, 3, [700, 64]),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp4"])
@pytest.mark.parametrize("q_len", [1, 4])
@pytest.mark.parametrize("window,sinks", [(1, 0), (16, 4), (33, 1), (100, 70), (2 ** 31 - 1, 0), (64, 2 ** 31 - 1)])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"hq{s[0]}-hkv{s[1]}-d{s[2]}-P{s[3]}-N{s[4]}-I{s[5]}")
def test_against_64_bits(shape, window, sinks, q_len, dtype):
    hq, hkv, d, page, n, i, L = shape
    L = [x if x == 0 else max(x, q_len) for x in L]
    rng = np.random.default_rng(hq + window % 1000 + q_len)

    def behind(b, p):  # rows that no query token sees: not stored, their pages given up where they can be
        return not (p < sinks or p > L[b] - q_len - window)

    c = Cache(dtype, [rows(rng, x, hkv, d) for x in L], [rows(rng, x, hkv, d) for x in L], hq=hq, hkv=hkv, d=d,
              page=page, n=n, i=i, drop=behind, scale=-0.1 if hq == 6 else None)
    q = bf16(rng.standard_normal((len(L), q_len, hq, d)))
    out, lse = run(c, to_bf16(q), window, sinks)
    vmax = max(np.abs(x).max(initial=0) for x in c.v)
    check("window", out, lse, *attention(c, q, window=window, sinks=sinks), vmax)


@pytest.mark.parametrize("dtype", ["bf16", "fp4"])
def test_rank_partials_merge_to_the_whole(dtype):
    hq, hkv, d, page, n, i, L, window, sinks = 8, 2, 128, 16, 4, 2, [300, 3, 90], 50, 5
    rng = np.random.default_rng(8)
    k, v = [rows(rng, x, hkv, d) for x in L], [rows(rng, x, hkv, d) for x in L]
    q = bf16(rng.standard_normal((3, 2, hq, d)))
    outs, lses = [], []
    for r in range(n):
        c = Cache(dtype, k, v, hq=hq, hkv=hkv, d=d, page=page, n=n, i=i, only=r)
        o, l = run(c, to_bf16(q), window, sinks, rank=r)
        vmax = max(np.abs(x).max() for x in c.v)
        check(f"rank {r}", o, l, *attention(c, q, window=window, sinks=sinks, shard=r), vmax)
        outs.append(o.view(3, 2 * hq, d))
        lses.append(l.view(3, 2 * hq))
    out, lse = torch.empty((3, 2 * hq, d), device="cuda"), torch.empty((3, 2 * hq), device="cuda")
    dcp.dcp_merge(torch.stack(outs), torch.stack(lses), out, lse)
    check("merged", out, lse, *attention(c, q, window=window, sinks=sinks), 2 * vmax)


@pytest.mark.parametrize("hq,q_len", [(2, 3), (16, 4)])
@pytest.mark.parametrize("dtype", ["bf16", "fp4"])
def test_non_finite_rows_reach_only_the_tokens_that_see_them(dtype, hq, q_len):
    """Among the new tokens, a later one's NaN or infinite key or value stays out of the earlier ones; behind the
    window nothing matters."""
    hkv, d, L, window = 2, 64, 60, 20
    rng = np.random.default_rng(1)
    k, v = rows(rng, L, hkv, d), rows(rng, L, hkv, d)
    v[L - 1, :, 3] = np.inf if dtype == "bf16" else np.nan
    k[L - 1, 1, 5] = np.nan
    v[L - window - q_len] = np.nan       # just behind the first token's window
    k[5] = np.nan
    c = Cache(dtype, [k], [v], hq=hq, hkv=hkv, d=d, page=16, n=1, i=1)
    q = bf16(rng.standard_normal((1, q_len, hq, d)))
    out, lse = run(c, to_bf16(q), window, 0)
    with np.errstate(invalid="ignore"):
        O, LSE = attention(c, q, window=window, sinks=0)
    clean = np.nan_to_num(c.v[0], posinf=0, neginf=0)
    check("earlier tokens", out[:, :-1], lse[:, :-1], O[:, :-1], LSE[:, :-1], np.abs(clean).max())
    last = out[0, -1].cpu().numpy()
    head = np.arange(hq) // (hq // hkv)
    assert np.isnan(last[head == 1]).all()                     # the NaN key
    assert not np.isfinite(last[head == 0][:, 3]).any()        # the value's dimension
    run_dims = [x for x in range(d) if not (dtype == "fp4" and x < 16) and x != 3]
    assert np.abs(last[head == 0][:, run_dims] - O[0, -1][head == 0][:, run_dims]).max() <= 1e-4 * np.abs(clean).max()


def test_masked_infinite_scores_and_empty_rows():
    """A visible key of -inf scores weighs nothing; a row of nothing but those is empty."""
    hkv, d, L = 1, 64, 40
    rng = np.random.default_rng(2)
    k, v = np.abs(rows(rng, L, hkv, d)) + 1, rows(rng, L, hkv, d)
    k[L - 3:] = -np.inf
    c = Cache("bf16", [bf16(k)], [v], hq=2, hkv=hkv, d=d, page=16, n=2, i=4)
    q = np.abs(bf16(rng.standard_normal((1, 1, 2, d)))) + 1
    q = bf16(q)
    for window, sinks in ((3, 0), (30, 0), (2, 1)):
        out, lse = run(c, to_bf16(q), window, sinks)
        O, LSE = attention(c, q, window=window, sinks=sinks)
        check(f"window {window}", out, lse, O, LSE, np.abs(v).max())


def test_short_request_with_more_query_tokens_than_positions_is_reported():
    hkv, d = 2, 64
    rng = np.random.default_rng(6)
    c = Cache("bf16", [rows(rng, 2, hkv, d)], [rows(rng, 2, hkv, d)], hq=4, hkv=hkv, d=d, page=16, n=1, i=1)
    q = bf16(rng.standard_normal((1, 4, 4, d)))
    out, lse = run(c, to_bf16(q), 8, 0)
    torch.cuda.synchronize()
    assert dcp.dcp_get_device_status() == dcp.DCP_ERR_INVALID_ARG
    check("rows before the first position are empty", out, lse, *attention(c, q, window=8), np.abs(c.v[0]).max())


@pytest.mark.parametrize("window", [40, 3000])
def test_streams_graphs_and_shared_workspace(window):
    """On another stream, captured and replayed with new lengths, two graphs on one workspace one after the other."""
    hq, hkv, d, L = 16, 2, 64, [3500, 20, 1700]
    rng = np.random.default_rng(7)
    c = Cache("bf16", [rows(rng, x, hkv, d) for x in L], [rows(rng, x, hkv, d) for x in L], hq=hq, hkv=hkv, d=d,
              page=64, n=2, i=16)
    q = bf16(rng.standard_normal((3, 1, hq, d)))
    qt = to_bf16(q)
    vmax = max(np.abs(x).max() for x in c.v)
    ws = torch.full((dcp.dcp_decode_window_workspace_size(c.desc, 3, 1, window, 2),), 0xEE, dtype=torch.uint8,
                    device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out, lse = run(c, qt, window, 2, ws=ws)
    s.synchronize()
    check("stream", out, lse, *attention(c, q, window=window, sinks=2), vmax)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        o, l = torch.empty_like(out), torch.empty_like(lse)
        with torch.cuda.graph(g):
            dcp.dcp_decode_window(c.desc, qt, c.seq_lens, window, 2, o, l, ws)
        graphs.append((g, o, l))
    for cut in (0, 5):
        c.lengths = np.maximum(np.array(L) - cut, 0)
        c.seq_lens.copy_(torch.as_tensor(c.lengths.astype(np.int32)))
        for g, o, l in graphs:
            g.replay()
        torch.cuda.synchronize()
        for _, o, l in graphs:
            check(f"replay {cut}", o, l, *attention(c, q, window=window, sinks=2), vmax)
    assert torch.equal(graphs[0][1], graphs[1][1])  # the same work twice: the same bits


@pytest.mark.parametrize("dtype", ["bf16", "fp4"])
def test_pools_past_four_gigabytes(dtype):
    """Pages whose byte offset does not fit 32 bits."""
    hq, hkv, d, P = 8, 8, 128, 64
    block = P * d * 2 if dtype == "bf16" else P * (d // 2 + d // 16)
    pages = (2 ** 32 + 2 ** 28) // (hkv * block) + 4
    rng = np.random.default_rng(10)
    L = 150
    c = Cache(dtype, [rows(rng, L, hkv, d)], [rows(rng, L, hkv, d)], hq=hq, hkv=hkv, d=d, page=P, n=1, i=1, spare=0)
    big = []
    for pool in (c.k_pages, c.v_pages):
        x = torch.zeros((pages,) + tuple(pool.shape[1:]), dtype=pool.dtype, device="cuda")
        x[pages - c.num_pages:] = pool
        big.append(x)
    c.k_pages, c.v_pages = big
    c.bt += pages - c.num_pages
    c.num_pages = pages
    c.desc = c.make_desc()
    q = bf16(rng.standard_normal((1, 1, hq, d)))
    out, lse = run(c, to_bf16(q), 100, 3)
    check("far pages", out, lse, *attention(c, q, window=100, sinks=3), np.abs(c.v[0]).max())
    pos = torch.tensor([0, 149], dtype=torch.int32, device="cuda")
    ko, vo = (torch.empty((2, hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    dcp.dcp_kv_gather(c.desc, torch.zeros_like(pos), pos, ko, vo)
    np.testing.assert_array_equal(ko.double().cpu().numpy(), c.k[0][[0, 149]])
    dcp.dcp_kv_append(c.desc, torch.zeros_like(pos), pos, ko, vo)
    k2 = torch.empty_like(ko)
    dcp.dcp_kv_gather(c.desc, torch.zeros_like(pos), pos, k2)
    if dtype == "bf16":
        assert torch.equal(k2, ko)


@pytest.mark.parametrize("d,group,q_len", [(64, 2, 1), (64, 3, 4), (128, 4, 2), (128, 16, 1)])
@pytest.mark.parametrize("dtype", ["bf16", "fp4"])
@pytest.mark.parametrize("window", [130, 1000])
def test_more_segments_than_blocks(window, dtype, d, group, q_len):
    """400 segments on 148 SMs: whole segments, of a lone warp (short window) or of a team of two (longer)."""
    B, hkv, page, n, i, sinks = 80, 5, 16, 2, 16, 3
    hq, g = hkv * group, torch.Generator("cuda").manual_seed(d + group)
    lens = torch.randint(q_len, 2200, (B,), generator=torch.Generator().manual_seed(5)).to(torch.int32)
    lens[7] = 0
    each = 2200 // n // page + 1
    pages = n * B * each
    bt = torch.randperm(pages, generator=torch.Generator().manual_seed(6)).to(torch.int32).view(n, B, each).cuda()
    shape, dt = ((pages, hkv, page, d), torch.bfloat16) if dtype == "bf16" else \
        ((pages, hkv, page * (d // 2 + d // 16)), torch.uint8)
    kp, vp = (torch.empty(shape, dtype=dt, device="cuda") for _ in range(2))
    for p in (kp, vp):  # rows that are not written: NaN
        p.view(torch.uint8).fill_(0xFF)
    desc = dcp.make_cache_desc(kind=dcp.DCP_GQA, dtype=dcp.DCP_BF16 if dtype == "bf16" else dcp.DCP_FP4_E2M1,
                               n_shards=n, interleave=i, page_size=page, num_pages=pages, hq=hq, hkv=hkv, dk=d, dv=d,
                               scale=d ** -0.5, batch=B, block_tables=bt, k_pages=kp, v_pages=vp)
    ks, vs = [], []
    for b, L in enumerate(lens.tolist()):
        k, v = (torch.randn((L, hkv, d), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
        pos = torch.arange(L, dtype=torch.int32, device="cuda")
        req = torch.full_like(pos, b)
        dcp.dcp_kv_append(desc, req, pos, k, v)
        dcp.dcp_kv_gather(desc, req, pos, k, v)
        ks.append(k), vs.append(v)
    q = torch.randn((B, q_len, hq, d), generator=g, device="cuda").to(torch.bfloat16)
    out, lse = torch.empty((B, q_len, hq, d), device="cuda"), torch.empty((B, q_len, hq), device="cuda")
    size = dcp.dcp_decode_window_workspace_size(desc, B, q_len, window, sinks)
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
    dcp.dcp_decode_window(desc, q, lens.cuda(), window, sinks, out, lse, ws)
    O = torch.zeros((B, q_len, hq, d), dtype=torch.float64, device="cuda")
    ref = torch.full((B, q_len, hq), -math.inf, dtype=torch.float64, device="cuda")
    for b, L in enumerate(lens.tolist()):
        for j in range(q_len):
            at = L - q_len + j
            p = torch.arange(max(0, at + 1), device="cuda")
            p = p[(p < sinks) | (p > at - window)]
            if not len(p):
                continue
            kd, vd = (x[b][p].double().repeat_interleave(group, 1) for x in (ks, vs))
            s = torch.einsum("hd,phd->hp", q[b, j].double(), kd) * d ** -0.5
            O[b, j] = torch.einsum("hp,phd->hd", s.softmax(-1), vd)
            ref[b, j] = s.logsumexp(-1)
    check("many segments", out, lse, O.cpu().numpy(), ref.cpu().numpy(), max(float(x.abs().max()) for x in vs if len(x)))
