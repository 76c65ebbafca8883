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
