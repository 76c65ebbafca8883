"""Ends of the ranges of the operators around the decode (marked gpu), against 64 bits."""
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


def decode(c, q, window=None, sinks=0):
    """dcp_decode_merged, or dcp_decode_window with a window."""
    B, ql, hq, d = q.shape
    out = torch.full((B, ql, hq, d), float("nan"), device="cuda")
    lse = torch.full((B, ql, hq), float("nan"), device="cuda")
    size = (dcp.dcp_decode_workspace_size_ex(c.desc, B, ql, dcp.DCP_DECODE_MERGED) if window is None else
            dcp.dcp_decode_window_workspace_size(c.desc, B, ql, window, sinks))
    assert size > 0
    ws = torch.full((size,), 0xCD, dtype=torch.uint8, device="cuda")
    if window is None:
        dcp.dcp_decode_merged(c.desc, q, c.seq_lens, out, lse, ws)
    else:
        dcp.dcp_decode_window(c.desc, q, c.seq_lens, window, sinks, out, lse, ws)
    return out, lse


# ---- a softmax scale of zero, and products of scales that 32 bits take for zero: every visible
# position weighs the same, and a masked one still weighs nothing.  The bounds of op_ref hold:
# all scores are 0 there, and what a product leaves of one is below 2^-100.

@pytest.mark.parametrize("hq,q_len", [(4, 1), (4, 3), (32, 1), (32, 2)])
@pytest.mark.parametrize("dtype,window,sinks", [("bf16", 40, 3), ("bf16", 2 ** 31 - 1, 0), ("fp4", 40, 3),
                                                ("fp4", None, 0)])
@pytest.mark.parametrize("scale", [0.0, -0.0, 1e-45])
def test_scale_of_zero(dtype, window, sinks, hq, q_len, scale):
    hkv, d, L = 2, 64, [77, 0, 16, 203]
    rng = np.random.default_rng(hq + q_len)
    c = Cache(dtype, [rows(rng, x, hkv, d) for x in L], [rows(rng, x, hkv, d) for x in L], hq=hq, hkv=hkv, d=d,
              page=16, n=2, i=5, scale=scale)
    q = bf16(rng.standard_normal((4, q_len, hq, d)))
    out, lse = decode(c, to_bf16(q), window, sinks)
    check("scale 0", out, lse, *attention(c, q, window=window, sinks=sinks), max(np.abs(x).max(initial=0) for x in c.v))


@pytest.mark.parametrize("hq", [4, 32])
@pytest.mark.parametrize("window", [None, 40])
def test_scales_whose_product_is_below_32_bits(hq, window):
    """A small key factor and small queries: 1e-30 of the keys' factor times 2^-67 of the query's row."""
    hkv, d, L = 2, 128, [77, 9]
    rng = np.random.default_rng(hq)
    c = Cache("fp4", [rows(rng, x, hkv, d, 1e-30) for x in L], [rows(rng, x, hkv, d) for x in L], hq=hq, hkv=hkv,
              d=d, page=16, n=2, i=1, factor=(1e-30, 1.0))
    assert np.abs(c.k[0]).max() > 0
    q = bf16(rng.standard_normal((2, 1, hq, d)) * 1e-20)
    out, lse = decode(c, to_bf16(q), window, 0)
    check("tiny scales", out, lse, *attention(c, q, window=window), max(np.abs(x).max() for x in c.v))


# ---- requests in parts: the sum's kernel is on the SMs before the parts are written

@pytest.mark.parametrize("dtype", ["bf16", "fp4"])
def test_parts_of_one_call_are_not_taken_for_the_next_ones(dtype):
    """Calls back to back on one workspace, each with other queries, eagerly and in a replayed graph: every one
    returns, bit for bit, what it returns by itself."""
    hq, hkv, d, L = 16, 1, 128, 3500
    rng = np.random.default_rng(12)
    c = Cache(dtype, [rows(rng, L, hkv, d)], [rows(rng, L, hkv, d)], hq=hq, hkv=hkv, d=d, page=64, n=2, i=64)
    qs = [to_bf16(bf16(rng.standard_normal((1, 1, hq, d)) * (1 + k))) for k in range(4)]
    alone = [decode(c, q, 3000, 1) for q in qs]
    for k, q in enumerate(qs):
        check(f"alone {k}", *alone[k], *attention(c, q.double().cpu().numpy(), window=3000, sinks=1), np.abs(c.v[0]).max())
    ws = torch.empty(dcp.dcp_decode_window_workspace_size(c.desc, 1, 1, 3000, 1), dtype=torch.uint8, device="cuda")
    assert ws.numel() > 4096  # in parts
    got = [(torch.empty_like(o), torch.empty_like(l)) for o, l in alone]

    def calls():
        for q, (o, l) in zip(qs, got):
            dcp.dcp_decode_window(c.desc, q, c.seq_lens, 3000, 1, o, l, ws)

    calls()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    first = [(o.clone(), l.clone()) for o, l in got]
    with torch.cuda.graph(graph):
        calls()
    for o, l in got:
        o.fill_(float("nan")), l.fill_(float("nan"))
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for (o, l), (fo, fl), (ro, rl) in zip(alone, first, got):
        assert torch.equal(fo, o) and torch.equal(fl, l) and torch.equal(ro, o) and torch.equal(rl, l)


# ---- workspace sizes

def windowed_desc(B, hkv, group, d, tokens, dtype=dcp.DCP_FP4_E2M1):
    """A descriptor for sizes only: tables of `tokens` positions on one shard."""
    bt = torch.zeros((1, B, -(-tokens // 64)), dtype=torch.int32, device="cuda")
    pool = torch.zeros(64, dtype=torch.uint8, device="cuda")
    return dcp.make_cache_desc(kind=dcp.DCP_GQA, dtype=dtype, n_shards=1, interleave=1, page_size=64, num_pages=1,
                               hq=hkv * group, hkv=hkv, dk=d, dv=d, scale=1.0, batch=B, block_tables=bt, k_pages=pool,
                               v_pages=pool), bt, pool


def test_sums_in_memory_take_room_only_where_a_warp_needs_them():
    """One segment for each pair of warps: whole segments in teams of two, no parts, so that the workspace is its
    header and, for more groups than a warp adds up without a store, 8704 bytes for each of the 8 warps of an SM."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    size = lambda d, w: dcp.dcp_decode_window_workspace_size(d, d.batch, 1, w, 0)  # noqa: E731
    B, hkv = sms, 4
    desc, *keep = windowed_desc(B, hkv, 16, 128, 1 << 17)
    assert size(desc, 300 * 16) == 256                            # 151 groups a warp
    assert 256 < size(desc, 600 * 16) <= 256 + 8 * sms * 8704     # 301
    few, *keep2 = windowed_desc(B, hkv, 8, 128, 1 << 17)
    assert size(few, 600 * 16) == 256                             # 8 rows: sums stay in registers


@pytest.mark.parametrize("B,hkv,group,q_len", [(1, 1, 1, 1), (1, 4, 16, 1), (3, 2, 16, 4), (48, 8, 8, 1), (74, 8, 16, 1),
                                               (512, 4, 16, 1), (2, 1, 16, 64)])
@pytest.mark.parametrize("d", [64, 128])
def test_4bit_workspaces_keep_to_the_stated_bound(B, hkv, group, q_len, d):
    W = 8 * torch.cuda.get_device_properties(0).multi_processor_count
    up = lambda x: -(-x // 256) * 256  # noqa: E731
    parts, sums = up(16 * W) + up(128 * W) + up(128 * d * W), up(8704 * W)
    for tokens in (64, 5000, 1 << 15, 1 << 20):
        desc, *keep = windowed_desc(B, hkv, group, d, tokens)
        sizes = [dcp.dcp_decode_workspace_size_ex(desc, B, q_len, m)
                 for m in (dcp.DCP_DECODE_PARTIAL, dcp.DCP_DECODE_MERGED, dcp.DCP_DECODE_RANK)]
        sizes += [dcp.dcp_decode_window_workspace_size(desc, B, q_len, w, 4) for w in (16, 1000, 9600, 1 << 17)]
        assert all(256 <= s <= 256 + parts + sums for s in sizes)
        assert sizes[0] <= dcp.DCP_STATIC_SCRATCH_BYTES


def shared_pages(g, dtype, B, hkv, group, d, page, L):
    """A cache of L positions on one shard whose pages all B requests read: small, whatever B."""
    pages = -(-L // page)
    bt = torch.arange(pages, dtype=torch.int32, device="cuda").expand(1, B, pages).contiguous()
    shape, dt = ((pages, hkv, page, d), torch.bfloat16) if dtype == "bf16" else \
        ((pages, hkv, page * (d // 2 + d // 16)), torch.uint8)
    kp, vp = (torch.zeros(shape, dtype=dt, device="cuda") for _ in range(2))
    desc = dcp.make_cache_desc(kind=dcp.DCP_GQA, dtype=dcp.DCP_BF16 if dtype == "bf16" else dcp.DCP_FP4_E2M1, n_shards=1,
                               interleave=1, page_size=page, num_pages=pages, hq=hkv * group, hkv=hkv, dk=d, dv=d,
                               scale=d ** -0.5, batch=B, block_tables=bt, k_pages=kp, v_pages=vp)
    k, v = (torch.randn((L, hkv, d), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    v += 0.25  # a mean apart from 0: O moves on all the way
    pos = torch.arange(L, dtype=torch.int32, device="cuda")
    req = torch.zeros_like(pos)
    dcp.dcp_kv_append(desc, req, pos, k, v)
    dcp.dcp_kv_gather(desc, req, pos, k, v)
    return desc, k, v, (bt, kp, vp)


def attend(q, k, v, L, window, sinks):
    """One request of attention in 64 bits on the GPU: q [q_len][hq][d], k and v [..][hkv][d]."""
    ql, hq, d = q.shape
    hkv = k.shape[1]
    kd, vd = k[:L].double(), v[:L].double()
    s = torch.einsum("jghd,pgd->jghp", q.double().view(ql, hkv, hq // hkv, d), kd) * d ** -0.5
    p, at = torch.arange(L, device="cuda"), (L - ql + torch.arange(ql, device="cuda"))[:, None]
    s = s.masked_fill(~((p <= at) & ((p < sinks) | (p > at - window)))[:, None, None], -float("inf"))
    return torch.einsum("jghp,pgd->jghd", s.softmax(-1), vd).reshape(ql, hq, d), s.logsumexp(-1).reshape(ql, hq)


def test_sums_in_memory_of_teams_of_two():
    """The plan of the sizes above with 301 groups a warp: O goes to memory once and comes back."""
    B, hkv, group, d, window, L = torch.cuda.get_device_properties(0).multi_processor_count, 4, 16, 128, 9600, 9733
    g = torch.Generator("cuda").manual_seed(4)
    desc, k, v, keep = shared_pages(g, "fp4", B, hkv, group, d, 64, L)
    q = torch.randn((B, 1, hkv * group, d), generator=g, device="cuda").to(torch.bfloat16)
    lens = torch.randint(9000, L + 1, (B,), generator=torch.Generator().manual_seed(4)).to(torch.int32)
    lens[5], lens[6] = 3, L
    out, lse = torch.empty((B, 1, hkv * group, d), device="cuda"), torch.empty((B, 1, hkv * group), device="cuda")
    ws = torch.full((dcp.dcp_decode_window_workspace_size(desc, B, 1, window, 2),), 0xFF, dtype=torch.uint8, device="cuda")
    guard = torch.full((ws.numel() + 4096,), 0xEE, dtype=torch.uint8, device="cuda")  # nothing is written behind the workspace
    dcp.dcp_decode_window(desc, q, lens.cuda(), window, 2, out, lse, guard[:ws.numel()])
    assert (guard[ws.numel():] == 0xEE).all()
    # between two stores O is cut off 2 * 256 times, 2^-23 of at most max|V| each, the sum of the
    # weights as often, and every weight is off by 2.1e-5 (op_ref); LSE sums 151 steps in 32 bits
    tol_o = (2 * 512 * 2.0 ** -23 + 2 * 2.1e-5) * float(v.abs().max())
    for b in range(B):
        O, ref = attend(q[b], k, v, int(lens[b]), window, 2)
        assert (out[b] - O).abs().max() <= tol_o
        assert (lse[b] - ref).abs().max() <= 5e-5 + 151 * 2.0 ** -24


# ---- lengths past the block table

@pytest.mark.parametrize("dtype,window,sinks", [("fp4", None, 0), ("fp4", 40, 3), ("bf16", 40, 3), ("bf16", 2 ** 31 - 1, 0),
                                                ("fp4", 2 ** 30, 0)])
@pytest.mark.parametrize("L", [130, 70000, 2 ** 31 - 1])
@pytest.mark.parametrize("hq,q_len", [(4, 1), (32, 1), (4, 3)])
def test_lengths_past_the_table_are_reported_and_cost_what_the_table_does(hq, q_len, L, dtype, window, sinks):
    """Positions without a table entry count as absent; the work does not grow with a length that cannot be."""
    hkv, d, have = 2, 64, 128  # four whole pages for each of two shards
    rng = np.random.default_rng(hq)
    c = Cache(dtype, [rows(rng, x, hkv, d) for x in (have, 33)], [rows(rng, x, hkv, d) for x in (have, 33)], hq=hq,
              hkv=hkv, d=d, page=16, n=2, i=16)
    q = bf16(rng.standard_normal((2, q_len, hq, d)))
    O, LSE = attention(c, q, window=window, sinks=sinks)
    for j in range(q_len):  # query token j of request 0 stands at L - q_len + j
        p, at = np.arange(have), L - q_len + j
        p = p if window is None else p[(p < sinks) | (p > at - window)]
        p = p[p <= at]
        for h in range(hq):
            O[0, j, h], LSE[0, j, h] = 0, -np.inf
            if len(p):
                s = c.k[0][p, h // (hq // hkv)] @ q[0, j, h] * c.scale
                w = np.exp(s - s.max())
                O[0, j, h], LSE[0, j, h] = w @ c.v[0][p, h // (hq // hkv)] / w.sum(), s.max() + np.log(w.sum())
    c.seq_lens[0] = L
    out, lse = decode(c, to_bf16(q), window, sinks)
    torch.cuda.synchronize()
    assert dcp.dcp_get_device_status() == dcp.DCP_ERR_UNALLOCATED_PAGE
    check("past the table", out, lse, O, LSE, max(np.abs(x).max() for x in c.v))


@pytest.mark.parametrize("dtype", ["fp4", "bf16"])
@pytest.mark.parametrize("q_len", [1, 2])
def test_a_window_past_a_page_that_is_not_there_reports_nothing(dtype, q_len):
    """Tables that end inside a run of positions: position 124 has no entry, but it lies behind the window."""
    hq, hkv, d, L, window = 4, 2, 64, 129, 3
    rng = np.random.default_rng(21)
    c = Cache(dtype, [rows(rng, x, hkv, d) for x in (L, 20)], [rows(rng, x, hkv, d) for x in (L, 20)], hq=hq, hkv=hkv, d=d,
              page=16, n=2, i=5)
    assert c.bt.shape[2] == 5      # shard 0 owns 65 of the 129 positions, the last of them 124
    c.bt = c.bt[:, :, :4].contiguous()
    c.desc = c.make_desc()
    q = bf16(rng.standard_normal((2, q_len, hq, d)))
    out, lse = decode(c, to_bf16(q), window, 0)
    check("behind the window", out, lse, *attention(c, q, window=window), max(np.abs(x).max() for x in c.v))
    torch.cuda.synchronize()
    assert dcp.dcp_get_device_status() == dcp.DCP_OK
    c.seq_lens[0] = 131            # 129, 130, .. : shard 1's 65th and shard 0's 66th are past the tables
    decode(c, to_bf16(q), window, 0)
    torch.cuda.synchronize()
    assert dcp.dcp_get_device_status() == dcp.DCP_ERR_UNALLOCATED_PAGE
