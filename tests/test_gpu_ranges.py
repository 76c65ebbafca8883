"""Sizes at the far ends of what the streamed decode documents (marked gpu), against 64 bits:
64 query tokens, interleaves whose round of all shards passes 32 bits, windows and 4-bit
shares long enough for every plan, tables much wider than their requests, missing pages."""
import numpy as np
import pytest
import torch

import sequence_sharded_paged_b200 as dcp

from op_ref import Cache, attention, bf16, check, rows
from test_gpu_edges import attend, decode, shared_pages, to_bf16

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clear_status():
    dcp.dcp_get_device_status()
    yield
    assert dcp.dcp_get_device_status() == dcp.DCP_OK


def cache(dtype, L, hq, hkv, d, page, n, i, seed, **kw):
    rng = np.random.default_rng(seed)
    return Cache(dtype, [rows(rng, x, hkv, d) for x in L], [rows(rng, x, hkv, d) for x in L], hq=hq, hkv=hkv, d=d,
                 page=page, n=n, i=i, **kw), rng


def widen(c, pages):
    """The same cache with block tables of `pages` local pages, -1 past the requests' own."""
    bt = torch.full(tuple(c.bt.shape[:2]) + (pages,), -1, dtype=torch.int32, device="cuda")
    bt[:, :, :c.bt.shape[2]] = c.bt
    c.bt = bt
    c.desc = c.make_desc()


@pytest.mark.parametrize("q_len,hq,hkv,d", [(64, 4, 2, 64), (64, 2, 2, 128), (17, 6, 2, 128), (33, 16, 1, 64)])
@pytest.mark.parametrize("dtype,window,sinks", [("bf16", 70, 5), ("fp4", 70, 5), ("bf16", 2 ** 31 - 1, 0), ("fp4", None, 0)])
def test_many_query_tokens(dtype, window, sinks, q_len, hq, hkv, d):
    c, rng = cache(dtype, [q_len, 300, 0, 701], hq, hkv, d, 16, 2, 16, q_len)
    q = bf16(rng.standard_normal((4, q_len, hq, d)))
    out, lse = decode(c, to_bf16(q), window, sinks)
    check("many tokens", out, lse, *attention(c, q, window=window, sinks=sinks), max(np.abs(x).max(initial=0) for x in c.v))


@pytest.mark.parametrize("n,i", [(8, 2 ** 30), (2, 3 * 2 ** 29), (7, 2 ** 31 - 1), (2 ** 20, 2 ** 12)])
@pytest.mark.parametrize("dtype,window,sinks", [("bf16", 70, 5), ("bf16", 2 ** 31 - 1, 0), ("fp4", 70, 5)])
@pytest.mark.parametrize("q_len", [1, 3])
def test_rounds_of_all_shards_past_32_bits(n, i, dtype, window, sinks, q_len):
    """interleave * n_shards at and above 2^31 and 2^32: as a rank, which holds all of the requests or nothing."""
    hq, hkv, d, L = 8, 2, 64, [300, 41]
    q = bf16(np.random.default_rng(1).standard_normal((2, q_len, hq, d)))
    for rank in (0, 1, n - 1):
        c, _ = cache(dtype, L, hq, hkv, d, 16, n, i, 3, only=rank)
        out, lse = (torch.full(s, float("nan"), device="cuda") for s in (q.shape, q.shape[:3]))
        ws = torch.empty(dcp.dcp_decode_window_workspace_size(c.desc, 2, q_len, window, sinks, rank=rank), dtype=torch.uint8,
                         device="cuda")
        dcp.dcp_decode_window(c.desc, to_bf16(q), c.seq_lens, window, sinks, out, lse, ws, rank=rank)
        check(f"rank {rank}", out, lse, *attention(c, q, window=window, sinks=sinks, shard=rank),
              max(np.abs(x).max() for x in c.v))
        if rank == 0:  # rows back by the same arithmetic
            pos = torch.arange(300, dtype=torch.int32, device="cuda")
            k = torch.empty((300, hkv, d), dtype=torch.bfloat16, device="cuda")
            dcp.dcp_kv_gather(c.desc, torch.zeros_like(pos), pos, k, rank=0)
            np.testing.assert_array_equal(k.double().cpu().numpy(), c.k[0])


@pytest.mark.parametrize("dtype", ["bf16", "fp4"])
@pytest.mark.parametrize("group,d,q_len", [(16, 128, 1), (8, 64, 3)])
def test_long_windows_are_split(dtype, group, d, q_len):
    """A window of 40000 positions of two requests among few heads: parts of every length, summed."""
    hkv, L, window, sinks = 2, 50021, 40000, 7
    g = torch.Generator("cuda").manual_seed(d)
    desc, k, v, keep = shared_pages(g, dtype, 2, hkv, group, d, 16, L)
    q = torch.randn((2, q_len, hkv * group, d), generator=g, device="cuda").to(torch.bfloat16)
    lens = torch.tensor([L, 33333], dtype=torch.int32, device="cuda")
    out, lse = torch.empty(q.shape, device="cuda"), torch.empty(q.shape[:3], device="cuda")
    ws = torch.full((dcp.dcp_decode_window_workspace_size(desc, 2, q_len, window, sinks),), 0xFF, dtype=torch.uint8, device="cuda")
    assert ws.numel() > 1 << 20  # in parts
    dcp.dcp_decode_window(desc, q, lens, window, sinks, out, lse, ws)
    # the bounds of op_ref: a part has fewer groups than its 4096 tokens
    for b in range(2):
        O, ref = attend(q[b], k, v, int(lens[b]), window, sinks)
        check(f"request {b}", out[b], lse[b], O.cpu().numpy(), ref.cpu().numpy(), float(v.abs().max()))


def test_4bit_shares_of_many_groups_of_128_dimensions():
    """Equal shares in which a warp's part of a segment is longer than what it sums before O goes to memory."""
    B, hkv, group, d, L = 96, 8, 16, 128, 32 * 1024 + 5
    g = torch.Generator("cuda").manual_seed(8)
    desc, k, v, keep = shared_pages(g, "fp4", B, hkv, group, d, 64, L)
    q = torch.randn((B, 1, hkv * group, d), generator=g, device="cuda").to(torch.bfloat16)
    lens = torch.full((B,), L, dtype=torch.int32, device="cuda")
    lens[3], lens[-1] = 1, L - 4096
    out, lse = torch.empty(q.shape, device="cuda"), torch.empty(q.shape[:3], device="cuda")
    size = dcp.dcp_decode_workspace_size_ex(desc, B, 1, dcp.DCP_DECODE_MERGED)
    dcp.dcp_decode_merged(desc, q, lens, out, lse, torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda"))
    # 768 segments of 2049 groups over at least 1184 warps, under 1400 groups a warp: between two stores O and
    # the sum of the weights are cut off 512 times each, 2^-23 of at most max|V|; 2.1e-5 of every weight twice
    # (op_ref).  The sum of the weights in LSE takes 700 steps of 2^-24 each, beside op_ref's 5e-5.
    tol_o = (2 * 1400 * 2.0 ** -23 + 2 * 2.1e-5) * float(v.abs().max())
    for b in range(0, B, 5):
        O, ref = attend(q[b], k, v, int(lens[b]), 2 ** 31 - 1, 0)
        assert (out[b] - O).abs().max() <= tol_o and (lse[b] - ref).abs().max() <= 5e-5 + 700 * 2.0 ** -24


@pytest.mark.parametrize("dtype,window,sinks", [("bf16", 50, 5), ("bf16", 2 ** 31 - 1, 0), ("fp4", 50, 5), ("fp4", None, 0)])
@pytest.mark.parametrize("pages", [64, 8192])
@pytest.mark.parametrize("hq,q_len", [(8, 1), (32, 1), (8, 4)])
def test_tables_wider_than_their_requests(dtype, window, sinks, pages, hq, q_len):
    """A server's tables have one width whatever the requests: other plans, the same results."""
    L = [300, 1000, 0, 5, 77]
    c, rng = cache(dtype, L, hq, 2, 64, 16, 2, 16, hq)
    widen(c, pages)
    q = bf16(rng.standard_normal((len(L), q_len, hq, 64)))
    out, lse = decode(c, to_bf16(q), window, sinks)
    check("wide tables", out, lse, *attention(c, q, window=window, sinks=sinks), max(np.abs(x).max(initial=0) for x in c.v))


@pytest.mark.parametrize("pages", [None, 4096])
def test_many_requests_and_shards(pages):
    """1200 (shard, request) pairs, more than a block has threads, most of them short or empty."""
    rng = np.random.default_rng(6)
    L = [int(x) for x in rng.integers(0, 41, 300)]
    L[17], L[299] = 900, 333
    c, rng = cache("fp4", L, 2, 1, 64, 16, 4, 2, 7)
    if pages:
        widen(c, pages)
    q = bf16(rng.standard_normal((300, 1, 2, 64)))
    part, plse = torch.full((4, 300, 1, 2, 64), float("nan"), device="cuda"), torch.full((4, 300, 1, 2), float("nan"), device="cuda")
    ws = torch.full((dcp.dcp_decode_workspace_size_ex(c.desc, 300, 1, dcp.DCP_DECODE_PARTIAL),), 0xAB, dtype=torch.uint8, device="cuda")
    dcp.dcp_decode_partial_multi(c.desc, to_bf16(q), c.seq_lens, part, plse, ws)
    vmax = max(np.abs(x).max(initial=0) for x in c.v)
    for s in range(4):
        check(f"shard {s}", part[s], plse[s], *attention(c, q, shard=s), vmax)
    out, lse = decode(c, to_bf16(q))
    check("merged", out, lse, *attention(c, q), vmax)


@pytest.mark.parametrize("dtype", ["bf16", "fp4"])
@pytest.mark.parametrize("hq,q_len", [(8, 1), (32, 1), (8, 3)])
def test_missing_pages_in_a_window_are_reported_and_skipped(dtype, hq, q_len):
    hkv, d, L, window, sinks = 2, 64, [200, 40], 90, 20
    c, rng = cache(dtype, L, hq, hkv, d, 16, 2, 1, hq)
    c.bt[0, 0, 5] = c.num_pages + 5     # positions 160, 162, .. 190
    c.bt[1, 0, 0] = -1                  # 1, 3, .. 31: of the sinks
    q = bf16(rng.standard_normal((2, q_len, hq, d)))
    O, LSE = attention(c, q, window=window, sinks=sinks)
    lost = [p for p in range(200) if (p % 2 == 0 and 160 <= p < 192) or (p % 2 == 1 and p < 32)]
    for j in range(q_len):
        at = 200 - q_len + j
        p = np.setdiff1d([x for x in range(at + 1) if x < sinks or x > at - window], lost)
        for h in range(hq):
            s = c.k[0][p, h // (hq // hkv)] @ q[0, j, h] * c.scale
            w = np.exp(s - s.max())
            O[0, j, h], LSE[0, j, h] = w @ c.v[0][p, h // (hq // hkv)] / w.sum(), s.max() + np.log(w.sum())
    out, lse = decode(c, to_bf16(q), window, sinks)
    torch.cuda.synchronize()
    assert dcp.dcp_get_device_status() == dcp.DCP_ERR_UNALLOCATED_PAGE
    check("missing pages", out, lse, O, LSE, max(np.abs(x).max() for x in c.v))
