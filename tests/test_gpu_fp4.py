"""The 4-bit cache (marked gpu): append, read-back and every decode call against the
64-bit reference of its definition."""
import numpy as np
import pytest
import torch

import sequence_sharded_paged_b200 as dcp

from op_ref import Cache, attention, bf16, check, quantise4, rows

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clear_status():
    dcp.dcp_get_device_status()
    yield
    assert dcp.dcp_get_device_status() == dcp.DCP_OK


def empty_cache(rng, L, **kw):
    """A cache with room for the lengths L whose stored bytes are garbage."""
    c = Cache("fp4", [np.zeros((n, kw["hkv"], kw["d"])) for n in L], [np.zeros((n, kw["hkv"], kw["d"])) for n in L],
              hq=kw["hkv"], **kw)
    c.k_pages.fill_(0xFF)
    c.v_pages.fill_(0xFF)
    return c


def to_bf16(x):
    return torch.as_tensor(x).to(torch.float32).to(torch.bfloat16).cuda()


def nasty(rng, T, hkv, d):
    """Rows that cover the format's corners: zeros, ties, values past the largest scale, scales that round
    to zero, infinities and NaN."""
    x = rng.standard_normal((T, hkv, d)) * 10.0 ** rng.uniform(-4, 4, (T, hkv, 1))
    x = x.reshape(T, hkv, d // 16, 16)
    x[0] = 0.0
    if T > 1:
        x[1, :, :, :8] = np.array([6, 0.25, 0.75, 1.25, -1.75, 2.5, -3.5, 5.0])  # scale 1: borders, to the even code
    if T > 2:
        x[2] *= 1e-9
    if T > 3:
        x[3, :, 0, 3] = np.inf
    if T > 4:
        x[4, :, -1, 15] = np.nan
    if T > 5:
        x[5, :, 0, :] = 3e38
    return bf16(x.reshape(T, hkv, d))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hkv,page,n,i,L", [(1, 16, 1, 1, [1]), (2, 16, 2, 1, [33, 0, 5]), (3, 64, 3, 7, [150, 64]),
                                            (8, 64, 4, 16, [130, 1, 77])])
@pytest.mark.parametrize("factor", [None, (0.5, 0.01)])
def test_append_and_gather_are_exact(d, hkv, page, n, i, L, factor):
    rng = np.random.default_rng(d + hkv)
    c = empty_cache(rng, L, hkv=hkv, d=d, page=page, n=n, i=i, factor=factor)
    T = sum(L)
    req = np.repeat(np.arange(len(L)), L).astype(np.int32)
    pos = np.concatenate([np.arange(x) for x in L]).astype(np.int32)
    order = rng.permutation(T)
    req, pos = torch.as_tensor(req[order]).cuda(), torch.as_tensor(pos[order]).cuda()
    k, v = nasty(rng, T, hkv, d), nasty(rng, T, hkv, d)
    dcp.dcp_kv_append(c.desc, req, pos, to_bf16(k), to_bf16(v))
    ko, vo = (torch.full((T, hkv, d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    dcp.dcp_kv_gather(c.desc, req, pos, ko, vo)
    fk, fv = (np.float64(np.float32(f)) for f in (factor or (1.0, 1.0)))
    for got, x, f in ((ko, k, fk), (vo, v, fv)):
        want = quantise4(x, f)[2]
        got = got.double().cpu().numpy()
        if factor is None or f in (0.5,):  # a power of two keeps 6 significant bits: exact in bf16
            np.testing.assert_array_equal(got, want)
        else:
            # A quotient by the factor is two 32-bit roundings (2^-24 each) away from the 64-bit one, so at a border
            # of the grid it may fall on either side; the value read back is rounded to 32 bits and to bf16 (half a
            # step, 2^-8 of it).  Every run has to be one of the three.
            ok = np.zeros(got.shape, bool)
            for nudge in (0.0, 2.0 ** -22, -2.0 ** -22):
                w = quantise4(x, f, nudge)[2]
                ok |= np.abs(got - w) <= np.abs(w) * (2.0 ** -8 + 2.0 ** -22)
                ok |= np.isnan(got) & np.isnan(w)
            assert ok.all()
    # only values, keys alone, an index listed twice
    idx = torch.zeros(3, dtype=torch.int32, device="cuda")
    if L[0] > 0:
        k3 = torch.empty((3, hkv, d), dtype=torch.bfloat16, device="cuda")
        dcp.dcp_kv_gather(c.desc, idx, idx, k3)
        first = int(np.where((req.cpu().numpy() == 0) & (pos.cpu().numpy() == 0))[0][0])
        assert torch.equal(k3, ko[first].expand(3, -1, -1)) or torch.isnan(ko[first]).any()


@pytest.mark.parametrize("kind", ["gqa", "mla-bf16", "mla-fp8"])
def test_gather_of_the_other_caches(kind):
    """bf16 rows come back bit for bit; fp8 rows as code * scale, rounded once."""
    rng = np.random.default_rng(5)
    n, i, P, L = 2, 3, 64, [70, 9]
    T = sum(L)
    req = torch.as_tensor(np.repeat(np.arange(2), L).astype(np.int32)).cuda()
    pos = torch.as_tensor(np.concatenate([np.arange(x) for x in L]).astype(np.int32)).cuda()
    bt = torch.arange(2 * 2 * 2, dtype=torch.int32, device="cuda").view(2, 2, 2)
    mla = kind != "gqa"
    shape = (8, P, 576) if mla else (8, 2, P, 64)
    dt = torch.uint8 if kind == "mla-fp8" else torch.bfloat16
    kp, vp = torch.zeros(shape, dtype=dt, device="cuda"), torch.zeros(shape, dtype=dt, device="cuda")
    sc = torch.zeros((8, P), device="cuda")
    desc = dcp.make_cache_desc(kind=dcp.DCP_MLA if mla else dcp.DCP_GQA,
                               dtype=dcp.DCP_FP8_E4M3 if kind == "mla-fp8" else dcp.DCP_BF16, n_shards=n, interleave=i,
                               page_size=P, num_pages=8, hq=16, hkv=1 if mla else 2, dk=576 if mla else 64,
                               dv=512 if mla else 64, scale=1.0, batch=2, block_tables=bt, k_pages=kp,
                               v_pages=None if mla else vp, kv_scales=sc if kind == "mla-fp8" else None)
    row = (576,) if mla else (2, 64)
    k, v = to_bf16(rng.standard_normal((T,) + row)), to_bf16(rng.standard_normal((T,) + row))
    dcp.dcp_kv_append(desc, req, pos, k, None if mla else v)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    dcp.dcp_kv_gather(desc, req, pos, ko, None if mla else vo)
    if kind != "mla-fp8":
        assert torch.equal(ko, k) and (mla or torch.equal(vo, v))
        return
    x = k.double().cpu().numpy()
    scale = (np.abs(x).max(-1, keepdims=True) / 448).astype(np.float32).astype(np.float64)
    from op_ref import E4M3, nearest
    got, ok = ko.double().cpu().numpy(), False
    for nudge in (0.0, 2.0 ** -23, -2.0 ** -23):  # the quotient is rounded to 32 bits: at a border, either code
        want = np.sign(x) * E4M3[nearest(np.abs(x) / scale * (1 + nudge), E4M3)] * scale
        # rounded to bf16 once (half a step, 2^-8 of the value), after a product in 32 bits (2^-24)
        ok |= np.abs(got - want) <= np.abs(want) * (2.0 ** -8 + 2.0 ** -23)
    assert ok.all()


SHAPES = [  # hq, hkv, d, page, n, i, lengths
    (8, 2, 64, 16, 2, 1, [300, 1000]),
    (8, 8, 64, 64, 1, 1, [1, 0, 130]),          # one query head for each KV head
    (6, 2, 128, 16, 3, 5, [77, 16, 15, 17]),    # groups of three
    (40, 8, 128, 64, 4, 16, [200, 65, 3]),      # groups of five
    (16, 1, 128, 64, 2, 64, [513]),             # a full tile
    (64, 4, 128, 16, 8, 128, [1500, 129, 0, 7]),
    (48, 2, 64, 16, 2, 2, [90, 91]),            # 24 rows: two tiles
]


@pytest.mark.parametrize("q_len", [1, 2, 5])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"hq{s[0]}-hkv{s[1]}-d{s[2]}-P{s[3]}-N{s[4]}-I{s[5]}")
def test_every_decode_call(shape, q_len):
    hq, hkv, d, page, n, i, L = shape
    L = [x if x == 0 else max(x, q_len) for x in L]
    rng = np.random.default_rng(hq * d + q_len)
    c = Cache("fp4", [rows(rng, x, hkv, d) for x in L], [rows(rng, x, hkv, d) for x in L], hq=hq, hkv=hkv, d=d,
              page=page, n=n, i=i, factor=(0.5, 2.0) if hq == 6 else None, seed=q_len)
    B = len(L)
    q = bf16(rng.standard_normal((B, q_len, hq, d)))
    qt = to_bf16(q)
    vmax = max(np.abs(x).max(initial=0) for x in c.v)
    O, LSE = attention(c, q)
    new = lambda *s: torch.full(s, float("nan"), device="cuda")  # noqa: E731

    def ws(mode):
        size = dcp.dcp_decode_workspace_size_ex(c.desc, B, q_len, mode)
        assert size > 0
        return torch.full((size,), 0xAB, dtype=torch.uint8, device="cuda")

    out, lse = new(B, q_len, hq, d), new(B, q_len, hq)
    fin = torch.full((B,), -1, dtype=torch.int64, device="cuda")
    w = ws(dcp.DCP_DECODE_MERGED)
    for again in range(2):
        dcp.dcp_decode_merged(c.desc, qt, c.seq_lens, out, lse, w, finish_ns=fin if again else None)
        check(f"merged {again}", out, lse, O, LSE, vmax)
    assert (fin >= 0).all() and (fin < 10 ** 9).all()
    part, plse = new(n, B, q_len, hq, d), new(n, B, q_len, hq)
    dcp.dcp_decode_partial_multi(c.desc, qt, c.seq_lens, part, plse, ws(dcp.DCP_DECODE_PARTIAL))
    for s in range(n):
        Os, Ls = attention(c, q, shard=s)
        check(f"shard {s}", part[s], plse[s], Os, Ls, vmax)
    dcp.dcp_merge(part.view(n, B, q_len * hq, d), plse.view(n, B, q_len * hq), out.view(B, q_len * hq, d),
                  lse.view(B, q_len * hq))
    check("partials merged", out, lse, O, LSE, 2 * vmax)  # two kernels' errors
    if q_len == 1:
        p2, l2 = new(n, B, hq, d), new(n, B, hq)
        dcp.dcp_decode_partial(c.desc, qt[:, 0].contiguous(), c.seq_lens, p2, l2, ws(dcp.DCP_DECODE_PARTIAL))
        assert torch.equal(p2, part[:, :, 0]) and torch.equal(l2, plse[:, :, 0])
        p2.fill_(float("nan"))
        dcp.dcp_decode_partial_noalloc(c.desc, qt[:, 0].contiguous(), c.seq_lens, p2, l2)
        assert torch.equal(p2, part[:, :, 0]) and torch.equal(l2, plse[:, :, 0])


def test_rank_partials():
    hq, hkv, d, page, n, i, L = 12, 4, 128, 16, 3, 4, [100, 1, 37]
    rng = np.random.default_rng(3)
    k, v = [rows(rng, x, hkv, d) for x in L], [rows(rng, x, hkv, d) for x in L]
    q = bf16(rng.standard_normal((3, 1, hq, d)))
    for r in range(n):
        c = Cache("fp4", k, v, hq=hq, hkv=hkv, d=d, page=page, n=n, i=i, only=r)
        o, l = torch.empty((3, 1, hq, d), device="cuda"), torch.empty((3, 1, hq), device="cuda")
        w = torch.empty(dcp.dcp_decode_workspace_size_ex(c.desc, 3, 1, dcp.DCP_DECODE_RANK), dtype=torch.uint8,
                        device="cuda")
        dcp.dcp_decode_rank(c.desc, r, to_bf16(q), c.seq_lens, o, l, w)
        check(f"rank {r}", o, l, *attention(c, q, shard=r), max(np.abs(x).max() for x in c.v))


def test_long_requests_are_split():
    """One request among few heads: its length is shared by many blocks and the parts are summed."""
    hq, hkv, d, L = 16, 1, 128, 40000
    rng = np.random.default_rng(9)
    g = torch.Generator().manual_seed(1)
    c = Cache("fp4", [np.zeros((0, hkv, d))], [np.zeros((0, hkv, d))], hq=hq, hkv=hkv, d=d, page=64, n=2, i=64,
              room=20000)
    c.lengths = np.array([L])
    c.seq_lens.fill_(L)
    k = torch.randn((L, hkv, d), generator=g).to(torch.bfloat16)
    v = torch.randn((L, hkv, d), generator=g).to(torch.bfloat16)
    req, pos = torch.zeros(L, dtype=torch.int32, device="cuda"), torch.arange(L, dtype=torch.int32, device="cuda")
    dcp.dcp_kv_append(c.desc, req, pos, k.cuda(), v.cuda())
    c.k, c.v = [quantise4(k.double().numpy())[2]], [quantise4(v.double().numpy())[2]]
    q = bf16(rng.standard_normal((1, 1, hq, d)) * 2)
    out, lse = torch.empty((1, 1, hq, d), device="cuda"), torch.empty((1, 1, hq), device="cuda")
    w = torch.empty(dcp.dcp_decode_workspace_size_ex(c.desc, 1, 1, 1), dtype=torch.uint8, device="cuda")
    dcp.dcp_decode_merged(c.desc, to_bf16(q), c.seq_lens, out, lse, w)
    check("split", out, lse, *attention(c, q), np.abs(c.v[0]).max())


def test_bad_pages_are_reported_and_skipped():
    hq, hkv, d, page, n, i, L = 8, 2, 64, 16, 2, 1, [200, 40]
    rng = np.random.default_rng(4)
    c = Cache("fp4", [rows(rng, x, hkv, d) for x in L], [rows(rng, x, hkv, d) for x in L], hq=hq, hkv=hkv, d=d,
              page=page, n=n, i=i)
    c.bt[0, 0, 1] = c.num_pages + 5
    c.bt[1, 0, 0] = -1
    q = bf16(rng.standard_normal((2, 1, hq, d)))
    O, LSE = attention(c, q)
    out, lse = torch.empty((2, 1, hq, d), device="cuda"), torch.empty((2, 1, hq), device="cuda")
    w = torch.empty(dcp.dcp_decode_workspace_size_ex(c.desc, 2, 1, 1), dtype=torch.uint8, device="cuda")
    dcp.dcp_decode_merged(c.desc, to_bf16(q), c.seq_lens, out, lse, w)
    torch.cuda.synchronize()
    assert dcp.dcp_get_device_status() == dcp.DCP_ERR_UNALLOCATED_PAGE
    assert torch.isfinite(out).all()
    check("the other request", out[1:], lse[1:], O[1:], LSE[1:], np.abs(c.v[1]).max())
    # request 0 as if the two pages' tokens did not exist
    lost = [p for p in range(L[0]) if (p % 2 == 0 and 16 <= p // 2 < 32) or (p % 2 == 1 and p // 2 < 16)]
    keep = np.setdiff1d(np.arange(L[0]), lost)
    for h in range(hq):
        s = (c.k[0][keep, h // 4] @ q[0, 0, h]) * c.scale
        p = np.exp(s - s.max())
        want = p @ c.v[0][keep, h // 4] / p.sum()
        assert np.abs(out[0, 0, h].double().cpu().numpy() - want).max() <= 1e-4 * np.abs(c.v[0]).max()
    ko = torch.full((3, hkv, d), 5.0, dtype=torch.bfloat16, device="cuda")
    pos = torch.tensor([1, 33, 0], dtype=torch.int32, device="cuda")
    dcp.dcp_kv_gather(c.desc, torch.zeros_like(pos), pos, ko)
    assert dcp.dcp_get_device_status() == dcp.DCP_ERR_UNALLOCATED_PAGE
    assert (ko[0] == 5).all()                                  # position 1: shard 1, page 0 (-1)
    np.testing.assert_array_equal(ko[2].double().cpu().numpy(), c.k[0][0])
