"""Norms of queries and keys, position rotation and append in one pass (marked gpu)
against 64 bits."""
import numpy as np
import pytest
import torch

import sequence_sharded_paged_b200 as dcp

from op_ref import bf16, frequencies, norm, quantise4, rotate

pytestmark = pytest.mark.gpu

# A stored value is the 64-bit one rounded to bf16 (half a step, 2^-8 of it) after 32-bit
# arithmetic: the norm's sum of up to 512 squares, its root, two products and the pair's
# two products and sum, under 32 roundings of 2^-24 of the pair's magnitude, and cosine
# and sine of an angle that is within 2^-33 turns (7.4e-10 rad) and 2 units of 2^-24.
# The pair's magnitude can exceed a cancelled result, so that part is absolute.
REL, ABS = 2.0 ** -8, 40 * 2.0 ** -24

SCALINGS = [dict(theta=1e4), dict(theta=5e5, scaling="linear", factor=4.0), dict(theta=1e4, scaling="base", factor=8.0),
            dict(theta=5e4, scaling="yarn", factor=32.0, original=4096.0, low=1.0, high=32.0),
            dict(theta=5e5, scaling="smooth", factor=8.0, original=8192.0, low=1.0, high=4.0)]


@pytest.fixture(autouse=True)
def _clear_status():
    dcp.dcp_get_device_status()
    yield
    assert dcp.dcp_get_device_status() == dcp.DCP_OK


def to_bf16(x):
    return torch.as_tensor(x).to(torch.float32).to(torch.bfloat16).cuda()


def near(name, got, want, mag):
    """|got - want| within the bound for values of pairs of magnitude mag."""
    got = got.double().cpu().numpy()
    bound = np.abs(want) * REL + mag * ABS + 1e-30
    bad = np.abs(got - want) > bound
    assert not bad.any(), f"{name}: {bad.sum()} of {bad.size}, worst {np.abs(got - want)[bad].max()}"


def tables(n, B, pages_each):
    return torch.as_tensor(np.random.default_rng(0).permutation(n * B * pages_each).astype(np.int32)
                           .reshape(n, B, pages_each)).cuda()


def tokens(rng, T, B, n, i, page, pages_each, far=0):
    """T distinct (request, position) pairs whose pages exist."""
    room = pages_each * page // i * i * n  # positions that fit
    flat = rng.permutation(B * room)[:T]
    return (flat // room).astype(np.int32), (flat % room).astype(np.int32)


@pytest.mark.parametrize("scaling", range(len(SCALINGS)))
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("d,rot,hq,hkv,page,n,i", [(64, 64, 8, 2, 16, 2, 1), (128, 32, 5, 5, 64, 3, 7), (128, 128, 64, 4, 16, 8, 128),
                                                   (64, 16, 3, 1, 64, 1, 1), (128, 48, 14, 2, 16, 2, 16)])
@pytest.mark.parametrize("dtype", ["bf16", "fp4"])
def test_gqa(d, rot, hq, hkv, page, n, i, layout, scaling, dtype):
    rng = np.random.default_rng(d + rot + scaling)
    T, B, each = 37, 3, 4 if i < 100 else 8
    req, pos = tokens(rng, T, B, n, i, page, each)
    bt = tables(n, B, each)
    pages = bt.numel()
    block = page * (d // 2 + d // 16)
    shape, dt = ((pages, hkv, page, d), torch.bfloat16) if dtype == "bf16" else ((pages, hkv, block), torch.uint8)
    kp, vp = torch.zeros(shape, dtype=dt, device="cuda"), torch.zeros(shape, dtype=dt, device="cuda")
    desc = dcp.make_cache_desc(kind=dcp.DCP_GQA, dtype=dcp.DCP_BF16 if dtype == "bf16" else dcp.DCP_FP4_E2M1,
                               n_shards=n, interleave=i, page_size=page, num_pages=pages, hq=hq, hkv=hkv, dk=d, dv=d,
                               scale=1.0, batch=B, block_tables=bt, k_pages=kp, v_pages=vp)
    qkv = bf16(rng.standard_normal((T, hq + 2 * hkv, d)) * 3)
    t = to_bf16(qkv)
    q, k, v = t[:, :hq], t[:, hq:hq + hkv], t[:, hq + hkv:]
    qw, kw = bf16(rng.standard_normal(d) * 0.3 + 1), bf16(rng.standard_normal(d) * 0.3 + 1)
    rope = dcp.make_rope(rot, layout=layout, **SCALINGS[scaling])
    q_out = torch.full((T, hq, d), 9.0, dtype=torch.bfloat16, device="cuda")
    dreq, dpos = torch.as_tensor(req).cuda(), torch.as_tensor(pos).cuda()
    use_norm = scaling != 1
    dcp.dcp_norm_rope_append(desc, rope, dreq, dpos, q, k, v, to_bf16(qw) if use_norm else None,
                             to_bf16(kw) if use_norm else None, 1e-6, q_out)
    ko, vo = (torch.empty((T, hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    dcp.dcp_kv_gather(desc, dreq, dpos, ko, vo)
    f, factor = frequencies(rot, **SCALINGS[scaling])

    def want(x, w):
        y = norm(x, w if use_norm else None, 1e-6)
        r = rotate(y[..., :rot], pos, f, factor, layout)
        mag = np.abs(y)
        a, z = (r[..., :rot // 2], r[..., rot // 2:]) if layout == "half" else (r[..., 0::2], r[..., 1::2])
        m = np.hypot(a, z)
        mag[..., :rot] = np.concatenate((m, m), -1) if layout == "half" else np.repeat(m, 2, -1)
        return np.concatenate((r, y[..., rot:]), -1), mag

    near("q", q_out, *want(qkv[:, :hq], qw))
    kref, kmag = want(qkv[:, hq:hq + hkv], kw)
    if dtype == "bf16":
        near("k", ko, kref, kmag)
        assert torch.equal(vo, v)
        return
    np.testing.assert_array_equal(vo.double().cpu().numpy(), quantise4(qkv[:, hq + hkv:])[2])
    # what the cache holds is the quantised bf16 row: where the row's bf16 rounding is the
    # reference's, the values are equal; a row value one bf16 step off moves the code or
    # the run's scale by one step at most
    got, ref = ko.double().cpu().numpy(), quantise4(bf16(kref))[2]
    assert (got == ref).mean() > 0.98
    run = np.abs(kref).reshape(T, hkv, d // 16, 16).max(-1).repeat(16, -1).reshape(kref.shape)
    assert (np.abs(got - ref) <= run * 0.45).all()  # the widest step, 4 to 6, is a third of the largest value; scales step 1/8


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("hq", [16, 48])
def test_mla(layout, dtype, in_place, hq):
    rng = np.random.default_rng(hq)
    T, B, n, i, page, each = 19, 2, 2, 3, 64, 3
    req, pos = tokens(rng, T, B, n, i, page, each)
    bt = tables(n, B, each)
    kp = torch.zeros((bt.numel(), page, 576), dtype=torch.bfloat16 if dtype == "bf16" else torch.uint8, device="cuda")
    sc = torch.zeros((bt.numel(), page), device="cuda")
    desc = dcp.make_cache_desc(kind=dcp.DCP_MLA, dtype=dcp.DCP_BF16 if dtype == "bf16" else dcp.DCP_FP8_E4M3, n_shards=n,
                               interleave=i, page_size=page, num_pages=bt.numel(), hq=hq, hkv=1, dk=576, dv=512, scale=1.0,
                               batch=B, block_tables=bt, k_pages=kp, kv_scales=sc if dtype == "fp8" else None)
    x, kx = bf16(rng.standard_normal((T, hq, 576))), bf16(rng.standard_normal((T, 600)) * 2)
    q, lat = to_bf16(x), to_bf16(kx)[:, :576]
    w = bf16(rng.standard_normal(512) * 0.3 + 1)
    sg = SCALINGS[3]
    rope = dcp.make_rope(64, layout=layout, **sg)
    q_out = q if in_place else torch.empty_like(q)
    dreq, dpos = torch.as_tensor(req).cuda(), torch.as_tensor(pos).cuda()
    dcp.dcp_norm_rope_append(desc, rope, dreq, dpos, q, lat, None, None, to_bf16(w), 1e-5, q_out)
    f, factor = frequencies(64, **sg)
    r = rotate(x[..., 512:], pos, f, factor, layout)
    np.testing.assert_array_equal(q_out[..., :512].double().cpu().numpy(), x[..., :512])
    near("q", q_out[..., 512:], r, np.abs(x[..., 512:]).max() * 2)
    ref = np.concatenate((norm(kx[:, :512], w, 1e-5), rotate(kx[:, None, 512:576], pos, f, factor, layout)[:, 0]), -1)
    ko = torch.empty((T, 576), dtype=torch.bfloat16, device="cuda")
    dcp.dcp_kv_gather(desc, dreq, dpos, ko)
    if dtype == "bf16":
        near("latent", ko, ref, np.abs(ref).max())
    else:  # e4m3 against the row's largest value: half a step, 2^-4 of a value, or half the smallest step of the scale
        got, amax = ko.double().cpu().numpy(), np.abs(ref).max(-1, keepdims=True)
        assert (np.abs(got - ref) <= np.abs(ref) * (2.0 ** -4 + 2.0 ** -7) + amax / 448 * 2.0 ** -9).all()


def gqa_desc(hq=4, hkv=2, d=64, B=2, n=1, i=1, each=2, page=16):
    bt = tables(n, B, each)
    kp, vp = (torch.zeros((bt.numel(), hkv, page, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    desc = dcp.make_cache_desc(kind=dcp.DCP_GQA, dtype=dcp.DCP_BF16, n_shards=n, interleave=i, page_size=page,
                               num_pages=bt.numel(), hq=hq, hkv=hkv, dk=d, dv=d, scale=1.0, batch=B, block_tables=bt,
                               k_pages=kp, v_pages=vp)
    return desc, kp, vp, bt


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_far_positions(layout):
    """Angles of the largest positions keep their fraction of a turn."""
    desc, *_ = gqa_desc(hq=2, d=128)
    rng = np.random.default_rng(0)
    pos = np.array([0, 1, 131071, 10 ** 6, 2 ** 24 + 1, 2 ** 31 - 1, 123456789], np.int32)
    T = len(pos)
    x = bf16(rng.standard_normal((T, 2, 128)))
    q_out = torch.empty((T, 2, 128), dtype=torch.bfloat16, device="cuda")
    dpos, dreq = torch.as_tensor(pos).cuda(), torch.zeros(T, dtype=torch.int32, device="cuda")
    dcp.dcp_norm_rope_append(desc, dcp.make_rope(128, layout=layout, theta=1e4), dreq, dpos, to_bf16(x), None, None,
                             None, None, 0.0, q_out)
    # the double frequencies themselves are off by 2^-53 of their value, times the position: 2.4e-7 rad at 2^31
    f, _ = frequencies(128, 1e4)
    near("q", q_out, rotate(x, pos, f, 1.0, layout), np.abs(x).max() * 2)


def test_padding_ranks_and_parts():
    desc, kp, vp, bt = gqa_desc(n=2, i=1)
    rng = np.random.default_rng(1)
    T = 5
    q, k, v = (to_bf16(rng.standard_normal((T, h, 64))) for h in (4, 2, 2))
    req = torch.tensor([0, 1, 0, 0, 1], dtype=torch.int32, device="cuda")
    pos = torch.tensor([3, -1, 4, -7, 0], dtype=torch.int32, device="cuda")
    rope = dcp.make_rope(64)
    q_out = torch.full((T, 4, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    dcp.dcp_norm_rope_append(desc, rope, req, pos, q, k, v, None, None, 0.0, q_out)
    torch.cuda.synchronize()
    assert dcp.dcp_get_device_status() == dcp.DCP_OK             # padding is no error
    assert (q_out[[1, 3]] == 9).all() and not (q_out[[0, 2, 4]] == 9).all(-1).any()
    assert (kp != 0).any(-1).sum() == 3 * 2                      # three tokens' heads, nothing else
    whole = kp.clone(), vp.clone(), q_out.clone()
    # queries alone; keys and values alone; the same without rotation is the append
    kp.zero_(), vp.zero_(), q_out.fill_(9.0)
    dcp.dcp_norm_rope_append(desc, rope, req, pos, q, None, None, None, None, 0.0, q_out)
    assert torch.equal(q_out, whole[2]) and not kp.any()
    dcp.dcp_norm_rope_append(desc, rope, req, pos, None, k, v, None, None, 0.0, None)
    assert torch.equal(kp, whole[0]) and torch.equal(vp, whole[1])
    # in place
    q2 = q.clone()
    dcp.dcp_norm_rope_append(desc, rope, req, pos, q2, None, None, None, None, 0.0, q2)
    assert torch.equal(q2[[0, 2, 4]], whole[2][[0, 2, 4]]) and torch.equal(q2[[1, 3]], q[[1, 3]])
    # a rank stores what it owns: tables of its shard only
    for r in range(2):
        kp.zero_(), vp.zero_()
        mine = dcp.make_cache_desc(kind=dcp.DCP_GQA, dtype=dcp.DCP_BF16, n_shards=2, interleave=1, page_size=16,
                                   num_pages=bt.numel(), hq=4, hkv=2, dk=64, dv=64, scale=1.0, batch=2,
                                   block_tables=bt[r:r + 1].contiguous(), k_pages=kp, v_pages=vp)
        q_out.fill_(9.0)
        dcp.dcp_norm_rope_append(mine, rope, req, pos, q, k, v, None, None, 0.0, q_out, rank=r)
        torch.cuda.synchronize()
        owned = [i for i, p in enumerate(pos.tolist()) if p >= 0 and p % 2 == r]
        assert torch.equal(q_out, whole[2]) and (kp != 0).any(-1).sum() == 2 * len(owned)


def test_without_rotation_and_norm_rows_pass_bit_for_bit():
    desc, kp, vp, bt = gqa_desc()
    bits = torch.randint(0, 1 << 16, (3, 8, 64), dtype=torch.int32, device="cuda").to(torch.int16)
    x = bits.view(torch.bfloat16)
    pos = torch.tensor([0, 17, 5], dtype=torch.int32, device="cuda")
    req = torch.tensor([0, 0, 1], dtype=torch.int32, device="cuda")
    q_out = torch.empty((3, 4, 64), dtype=torch.bfloat16, device="cuda")
    dcp.dcp_norm_rope_append(desc, None, req, pos, x[:, :4], x[:, 4:6], x[:, 6:], None, None, 1.0, q_out)
    ko, vo = (torch.empty((3, 2, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    dcp.dcp_kv_gather(desc, req, pos, ko, vo)
    assert torch.equal(q_out.view(torch.int16), bits[:, :4])
    assert torch.equal(ko.view(torch.int16), bits[:, 4:6]) and torch.equal(vo.view(torch.int16), bits[:, 6:])


def test_unallocated_pages_are_reported():
    desc, kp, vp, bt = gqa_desc()
    bt[0, 0, 1] = -1
    bt[0, 1, 0] = bt.numel()
    q, k, v = (torch.ones((3, h, 64), dtype=torch.bfloat16, device="cuda") for h in (4, 2, 2))
    req = torch.tensor([0, 1, 0], dtype=torch.int32, device="cuda")
    pos = torch.tensor([20, 2, 33], dtype=torch.int32, device="cuda")  # -1, past the pool, past the table
    q_out = torch.zeros((3, 4, 64), dtype=torch.bfloat16, device="cuda")
    dcp.dcp_norm_rope_append(desc, None, req, pos, q, k, v, None, None, 0.0, q_out)
    torch.cuda.synchronize()
    assert dcp.dcp_get_device_status() == dcp.DCP_ERR_UNALLOCATED_PAGE
    assert not kp.any() and not vp.any() and (q_out == 1).all()


@pytest.mark.parametrize("T", [1, 300, 5000])
def test_many_tokens_and_graphs(T):
    """Block sizes change with the number of tokens; a captured call reads its inputs anew."""
    hq, hkv, d = 6, 2, 128
    desc, kp, vp, bt = gqa_desc(hq=hq, hkv=hkv, d=d, B=1, n=2, i=4, each=200, page=16)
    rng = np.random.default_rng(T)
    pos = rng.permutation(6400)[:T].astype(np.int32)
    x = bf16(rng.standard_normal((T, hq + 2 * hkv, d)))
    t = to_bf16(x)
    dpos, req = torch.as_tensor(pos).cuda(), torch.zeros(T, dtype=torch.int32, device="cuda")
    w = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    q_out = torch.empty((T, hq, d), dtype=torch.bfloat16, device="cuda")
    rope = dcp.make_rope(d, theta=1e6)
    args = (desc, rope, req, dpos, t[:, :hq], t[:, hq:hq + hkv], t[:, hq + hkv:], w, w, 1e-6, q_out)
    dcp.dcp_norm_rope_append(*args)
    f, _ = frequencies(d, 1e6)
    ko, vo = (torch.empty((T, hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    dcp.dcp_kv_gather(desc, req, dpos, ko, vo)
    y = norm(x, 1.0, 1e-6)
    near("q", q_out, rotate(y[:, :hq], pos, f, 1.0, "half"), np.abs(y).max() * 2)
    near("k", ko, rotate(y[:, hq:hq + hkv], pos, f, 1.0, "half"), np.abs(y).max() * 2)
    assert torch.equal(vo, t[:, hq + hkv:])
    first = q_out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dcp.dcp_norm_rope_append(*args)
    t.mul_(-1)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(q_out, -first)
