"""Norm, rotation and append into quantised caches (marked gpu): what they store is what
dcp_kv_append stores of the bf16 rows that the same call puts into a bf16 cache."""
import numpy as np
import pytest
import torch

import sequence_sharded_paged_b200 as dcp

from op_ref import bf16, quantise4

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clear_status():
    dcp.dcp_get_device_status()
    yield
    assert dcp.dcp_get_device_status() == dcp.DCP_OK


def to_bf16(x):
    return torch.as_tensor(x).to(torch.float32).to(torch.bfloat16).cuda()


def pools(kind, dtype, num_pages, hkv, page, d):
    """(k_pages, v_pages, kv_scales), every byte 0xA5."""
    if kind == dcp.DCP_MLA:
        k = torch.empty((num_pages, page, 576), dtype=torch.bfloat16 if dtype == dcp.DCP_BF16 else torch.uint8, device="cuda")
        both = [k, None]
        scales = torch.zeros((num_pages, page), device="cuda") if dtype == dcp.DCP_FP8_E4M3 else None
    else:
        shape, dt = ((num_pages, hkv, page, d), torch.bfloat16) if dtype == dcp.DCP_BF16 else \
            ((num_pages, hkv, page * (d // 2 + d // 16)), torch.uint8)
        both, scales = [torch.empty(shape, dtype=dt, device="cuda") for _ in range(2)], None
    for p in both:
        if p is not None:
            p.view(torch.uint8).fill_(0xA5)
    return both[0], both[1], scales


def caches(kind, quantised, *, hq, hkv, d, dv, page, n, i, B, each, factors=None):
    """A bf16 cache and two quantised ones with the same tables."""
    bt = torch.as_tensor(np.random.default_rng(0).permutation(n * B * each).astype(np.int32).reshape(n, B, each)).cuda()
    out = []
    for dtype in (dcp.DCP_BF16, quantised, quantised):
        k, v, s = pools(kind, dtype, n * B * each, hkv, page, d)
        s = factors if dtype == dcp.DCP_FP4_E2M1 else s
        out.append((dcp.make_cache_desc(kind=kind, dtype=dtype, n_shards=n, interleave=i, page_size=page,
                                        num_pages=n * B * each, hq=hq, hkv=hkv, dk=d, dv=dv, scale=1.0, batch=B,
                                        block_tables=bt, k_pages=k, v_pages=v, kv_scales=s), k, v, s))
    return out, bt


def places(rng, T, B, n, i, page, each):
    room = each * page // i * i * n
    flat = rng.permutation(B * room)[:T]
    return [torch.as_tensor(x.astype(np.int32)).cuda() for x in (flat // room, flat % room)]


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("d,rot,hq,hkv,page,n,i,normed,factors", [
    (64, 64, 8, 2, 16, 2, 1, False, None), (128, 48, 5, 5, 64, 3, 7, False, (0.75, 3.0)), (128, 128, 16, 4, 16, 2, 16, False, None),
    (64, 16, 3, 1, 64, 1, 1, True, None), (128, 128, 64, 4, 16, 8, 128, True, None), (128, 32, 14, 2, 16, 2, 16, True, (0.5, 2.0)),
    (128, None, 4, 2, 16, 1, 1, False, None)])
def test_4bit_rows_are_the_appended_bf16_rows(d, rot, hq, hkv, page, n, i, normed, factors, layout):
    rng = np.random.default_rng(d + hq)
    T, B, each = 301, 3, 256 // page
    fs = None if factors is None else torch.tensor(list(factors) + [0, 0], dtype=torch.float32, device="cuda")
    (plain, direct, appended), bt = caches(dcp.DCP_GQA, dcp.DCP_FP4_E2M1, hq=hq, hkv=hkv, d=d, dv=d, page=page, n=n, i=i,
                                           B=B, each=each, factors=fs)
    req, pos = places(rng, T, B, n, i, page, each)
    qkv = to_bf16(rng.standard_normal((T, hq + 2 * hkv, d)) * np.exp(rng.standard_normal((T, 1, 1)) * 3))
    w = to_bf16(rng.standard_normal(d) * 0.3 + 1) if normed else None
    rope = None if rot is None else dcp.make_rope(rot, layout=layout, theta=1e4)
    for desc, *_ in (plain, direct):
        q_out = torch.empty((T, hq, d), dtype=torch.bfloat16, device="cuda")
        dcp.dcp_norm_rope_append(desc, rope, req, pos, qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], w, w, 1e-6, q_out)
    k, v = (torch.empty((T, hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    dcp.dcp_kv_gather(plain[0], req, pos, k, v)
    assert torch.equal(v, qkv[:, hq + hkv:])
    dcp.dcp_kv_append(appended[0], req, pos, k, v)
    assert torch.equal(direct[2], appended[2])  # values: whole pool, untouched bytes among them
    if not normed:  # the same operations in the same order
        assert torch.equal(direct[1], appended[1])
        return
    # the sum of squares is taken in another order: the factor differs in the last bits of 32, and a
    # row's value may lie one bf16 step away.  Where a run is not the appended one, it is that of a row
    # with one such step (two in one run of 16 are rarer than 1 in 10^6).
    got, want = (torch.empty((T, hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    dcp.dcp_kv_gather(direct[0], req, pos, got)
    dcp.dcp_kv_gather(appended[0], req, pos, want)
    runs = lambda x: x.double().cpu().numpy().reshape(-1, 16)  # noqa: E731
    got, want, row = runs(got), runs(want), runs(k)
    off = np.flatnonzero((got != want).any(-1))
    assert len(off) <= 0.02 * len(got)
    factor = factors[0] if factors else 1.0
    for r in off:
        near = []
        for e in range(16):
            for way in (-np.inf, np.inf):
                x = torch.tensor(row[r], dtype=torch.float64).to(torch.bfloat16)
                x[e] = torch.nextafter(x[e], torch.tensor(way, dtype=torch.bfloat16))
                near.append(x.double().numpy())
        values = bf16(quantise4(np.array(near), factor)[2])
        assert (values == got[r]).all(-1).any(), f"run {r}: {row[r]} stored as {got[r]}"


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("normed", [False, True])
@pytest.mark.parametrize("hq", [16, 48])
def test_fp8_latent_rows_are_the_appended_bf16_rows(layout, normed, hq):
    rng = np.random.default_rng(hq)
    T, B, n, i, page, each = 203, 2, 2, 3, 64, 3
    (plain, direct, appended), bt = caches(dcp.DCP_MLA, dcp.DCP_FP8_E4M3, hq=hq, hkv=1, d=576, dv=512, page=page, n=n, i=i,
                                           B=B, each=each)
    req, pos = places(rng, T, B, n, i, page, each)
    x = rng.standard_normal((T, 576)) * np.exp(rng.standard_normal((T, 1)) * 3)
    x[7] = 0.0
    lat = to_bf16(x)
    w = to_bf16(rng.standard_normal(512) * 0.3 + 1) if normed else None
    rope = dcp.make_rope(64, layout=layout, theta=1e4)
    for desc, *_ in (plain, direct):
        dcp.dcp_norm_rope_append(desc, rope, req, pos, None, lat, None, None, w, 1e-6, None)
    k = torch.empty((T, 576), dtype=torch.bfloat16, device="cuda")
    dcp.dcp_kv_gather(plain[0], req, pos, k)
    dcp.dcp_kv_append(appended[0], req, pos, k)
    assert torch.equal(direct[1], appended[1]) and torch.equal(direct[3], appended[3])  # one kernel, one order
