"""Host side of the cache operators, without a GPU: refusals with the status that
include/dcp.h names, the rotation's frequencies, and the binding's argument checks."""
import ctypes
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import sequence_sharded_paged_b200 as dcp

from op_ref import frequencies

A = 1024  # a 16-byte-aligned placeholder device address


def gqa(dtype=dcp.DCP_FP4_E2M1, **kw):
    d = dcp.CacheDesc()
    d.kind, d.dtype, d.n_shards, d.interleave, d.page_size = dcp.DCP_GQA, dtype, 2, 1, 64
    d.num_pages, d.hq, d.hkv, d.dk, d.dv, d.batch, d.max_local_pages = 10, 16, 4, 128, 128, 3, 4
    d.k_pages, d.v_pages, d.block_tables, d.scale = 256, 768, 16, 1.0
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def mla(**kw):
    return gqa(dcp.DCP_BF16, kind=dcp.DCP_MLA, hq=16, hkv=1, dk=576, dv=512, v_pages=None, **kw)


INVALID, UNSUPPORTED, MISALIGNED = dcp.DCP_ERR_INVALID_ARG, dcp.DCP_ERR_UNSUPPORTED, dcp.DCP_ERR_MISALIGNED


@pytest.mark.parametrize("change,status", [
    (dict(kind=dcp.DCP_MLA, hkv=1, dk=576, dv=512), UNSUPPORTED),   # 4 bits are for GQA caches
    (dict(dv=64), UNSUPPORTED), (dict(dk=96, dv=96), UNSUPPORTED), (dict(page_size=32), UNSUPPORTED),
    (dict(k_pages=264), MISALIGNED), (dict(kv_scales=520), MISALIGNED), (dict(v_pages=None), INVALID),
    (dict(hq=18), INVALID), (dict(n_shards=0), INVALID),
])
def test_4bit_descriptors(change, status):
    L, d = dcp.lib(), gqa(**change)
    assert L.dcp_kv_append(ctypes.byref(d), 1, A, A, A, A, None) == status
    assert L.dcp_kv_gather(ctypes.byref(d), -1, 1, A, A, A, A, None) == status
    assert L.dcp_decode_merged(ctypes.byref(d), 3, 1, A, A, A, A, None, A, 1 << 30, None) == status
    assert L.dcp_decode_window(ctypes.byref(d), -1, 3, 1, 8, 0, A, A, A, A, A, 1 << 30, None) == status


def test_gather_refusals():
    L, d = dcp.lib(), gqa()
    call = lambda rank=-1, n=1, pos=A, k=A, v=A, desc=d: L.dcp_kv_gather(ctypes.byref(desc), rank, n, None, pos, k, v, None)  # noqa: E731
    assert call(rank=-2) == INVALID and call(rank=2) == INVALID and call(n=-1) == INVALID
    assert call(pos=None) == INVALID and call(k=None) == INVALID
    assert call(k=A + 8) == MISALIGNED and call(v=A + 2) == MISALIGNED
    assert call(n=0, pos=None, k=None) == dcp.DCP_OK
    assert call(desc=mla()) == INVALID  # a latent cache has no values of its own


def test_window_refusals():
    L = dcp.lib()

    def call(d=None, rank=-1, B=3, q_len=1, window=8, sinks=0, q=A, lens=A, out=A, lse=A, ws=A):
        d = gqa(dcp.DCP_BF16) if d is None else d
        return L.dcp_decode_window(ctypes.byref(d), rank, B, q_len, window, sinks, q, lens, out, lse, ws, 1 << 30, None)

    for bad in (dict(rank=2), dict(rank=-2), dict(B=2), dict(q_len=0), dict(window=0), dict(window=-5), dict(sinks=-1),
                dict(q=None), dict(lens=None), dict(out=None), dict(lse=None), dict(ws=None)):
        assert call(**bad) == INVALID, bad
    assert call(q_len=65) == UNSUPPORTED and call(d=mla()) == UNSUPPORTED
    for bad in (dict(q=A + 8), dict(out=A + 4), dict(lse=A + 4), dict(ws=A + 8)):
        assert call(**bad) == MISALIGNED, bad
    assert L.dcp_decode_window(None, -1, 3, 1, 8, 0, A, A, A, A, A, 1, None) == INVALID
    d = gqa()
    assert L.dcp_decode_window_workspace_size(ctypes.byref(d), -1, 3, 1, 0, 0) == 0
    assert L.dcp_decode_window_workspace_size(ctypes.byref(mla()), -1, 3, 1, 8, 0) == 0


def test_norm_rope_refusals():
    L = dcp.lib()
    rope = dcp.make_rope(128)

    def call(d=None, rank=-1, rope=rope, n=2, pos=A, q=A, qs=16 * 128, k=A, ks=512, v=A, vs=512, qw=A, kw=A, eps=1e-6,
             q_out=1 << 20):
        d = gqa() if d is None else d
        r = None if rope is None else ctypes.byref(rope)
        return L.dcp_norm_rope_append(ctypes.byref(d), rank, r, n, None, pos, q, qs, k, ks, v, vs, qw, kw, eps, q_out, None)

    for bad in (dict(rank=2), dict(n=-1), dict(eps=-1.0), dict(eps=float("nan")), dict(pos=None), dict(q_out=None),
                dict(q=None), dict(q=None, k=None, v=None, qw=None, kw=None, q_out=None), dict(v=None), dict(k=None),
                dict(q=None, q_out=None), dict(k=None, v=None), dict(qs=100), dict(ks=100), dict(vs=0),
                dict(q_out=A + 64, qs=16 * 128), dict(q_out=A, qs=16 * 128 + 64), dict(rope=dcp.Rope())):
        assert call(**bad) == INVALID, bad
    assert call(qs=16 * 128 + 4) == MISALIGNED
    for name in ("q", "k", "v", "qw", "kw", "q_out"):
        assert call(**{name: (1 << 20) + 8}) == MISALIGNED, name
    assert call(d=gqa(dk=64, dv=64)) == UNSUPPORTED               # 128 rotated dimensions of 64
    assert call(n=0, pos=None, q=None, k=None, v=None) == dcp.DCP_OK
    m = dict(d=mla(), qs=16 * 576, ks=576, v=None, qw=None)
    assert call(**m) == UNSUPPORTED                               # a latent row rotates its last 64
    r64 = dcp.make_rope(64)
    assert call(**{**m, "rope": r64, "v": A}) == INVALID and call(**{**m, "rope": r64, "qw": A}) == INVALID


@pytest.mark.parametrize("which", ["q", "k", "v", "qw", "kw"])
def test_norm_rope_refuses_an_output_that_overlaps_an_input(which):
    L = dcp.lib()
    rope = dcp.make_rope(128)
    far = dict(q=1 << 30, k=2 << 30, v=3 << 30, qw=4 << 30, kw=5 << 30)
    size = dict(q=2 * 2 * 16 * 128, k=2 * (1024 + 512), v=2 * (1024 + 512), qw=256, kw=256)[which]  # bytes read

    def call(out):
        p = far
        return L.dcp_norm_rope_append(ctypes.byref(gqa()), 0, ctypes.byref(rope), 2, A, A, p["q"], 2048, p["k"], 1024,
                                      p["v"], 1024, p["qw"], p["kw"], 1e-6, out, None)

    out_bytes = 2 * 2 * 16 * 128
    assert call(far[which] + size - 16) == INVALID
    assert call(far[which] - out_bytes + 16) == INVALID
    # next to it: passes the checks (and fails for want of a GPU, or is not reached on one)
    if not torch.cuda.is_available():
        assert call(far[which] + size) == dcp.DCP_ERR_CUDA and call(far[which] - out_bytes) == dcp.DCP_ERR_CUDA


def test_rope_refusals():
    L, r = dcp.lib(), dcp.Rope()
    call = lambda rot=64, layout=0, theta=1e4, kind=0, factor=1.0, original=0.0, low=0.0, high=0.0, attn=0.0: L.dcp_rope_init(  # noqa: E731
        ctypes.byref(r), rot, layout, theta, kind, factor, original, low, high, attn)
    assert call() == dcp.DCP_OK
    for bad in (dict(rot=0), dict(layout=2), dict(theta=1.0), dict(theta=math.inf), dict(theta=math.nan), dict(kind=5),
                dict(kind=1, factor=0.5), dict(kind=2, factor=math.nan), dict(kind=3, factor=2.0),
                dict(kind=3, factor=2.0, original=10.0, low=2.0, high=2.0), dict(attn=-1.0), dict(attn=math.nan)):
        assert call(**bad) == INVALID, bad
    for rot in (8, 24, 130, 144, 256):
        assert call(rot=rot) == UNSUPPORTED, rot
    assert L.dcp_rope_init(None, 64, 0, 1e4, 0, 1.0, 0.0, 0.0, 0.0, 0.0) == INVALID
    with pytest.raises(ValueError):
        dcp.make_rope(64, layout="other")
    with pytest.raises(dcp.DcpError):
        dcp.make_rope(20)


@pytest.mark.parametrize("rot", [16, 64, 128])
@pytest.mark.parametrize("kw", [dict(theta=1e4), dict(theta=1e6, scaling="linear", factor=3.0),
                                dict(theta=1e4, scaling="base", factor=8.0),
                                dict(theta=1e5, scaling="yarn", factor=40.0, original=4096.0, low=1.0, high=32.0),
                                dict(theta=5e5, scaling="smooth", factor=8.0, original=8192.0, low=1.0, high=4.0)])
def test_rope_frequencies(rot, kw):
    """turns[] are the frequencies in 2^-64 turns: within the doubles' own rounding of the definition."""
    r = dcp.make_rope(rot, layout="interleaved", **kw)
    f, factor = frequencies(rot, **kw)
    two_pi = Fraction(6283185307179586476925286766559005768394, 10 ** 39)
    for k in range(rot // 2):
        want = Fraction(float(f[k])) / two_pi * 2 ** 64
        assert abs(Fraction(r.turns[k]) - want) <= want * Fraction(1, 2 ** 45) + 1
    assert all(t == 0 for t in r.turns[rot // 2:])
    assert (r.rot_dim, r.layout) == (rot, dcp.DCP_ROPE_INTERLEAVED)
    assert abs(r.attn_factor - factor) <= factor * 2.0 ** -23
    assert dcp.make_rope(rot, attn_factor=0.5, **kw).attn_factor == 0.5


def test_rope_struct_matches_the_header():
    assert ctypes.sizeof(dcp.Rope) == 16 + 8 * 64
    assert dcp.Rope.turns.offset == 16


def test_binding_refuses_host_tensors():
    d = gqa()
    q = torch.zeros((3, 16, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="not on the current CUDA device"):
        dcp.dcp_decode_window(d, q, torch.zeros(3, dtype=torch.int32), 8, 0, torch.zeros((3, 16, 128)),
                              torch.zeros((3, 16)), torch.zeros(256, dtype=torch.uint8))
    with pytest.raises(ValueError, match="not on the current CUDA device"):
        dcp.dcp_kv_gather(d, None, torch.zeros(2, dtype=torch.int32), torch.zeros((2, 4, 128), dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        dcp.dcp_norm_rope_append(d, None, None, torch.zeros(2, dtype=torch.int32), None, None, None, None, None, 0.0, None)


def test_reference_quantiser_against_brute_force():
    """The tests' own quantiser: every code is a nearest one, ties go to the even code."""
    from op_ref import E2M1, E4M3, quantise4
    rng = np.random.default_rng(0)
    x = rng.standard_normal((50, 32)) * 10.0 ** rng.uniform(-3, 3, (50, 1))
    code, sb, val = quantise4(x)
    for row in range(50):
        for run in range(2):
            part = slice(16 * run, 16 * run + 16)
            want = np.abs(x[row, part]).max() / 6
            scale = E4M3[sb[row, run]]
            assert np.abs(scale - want) <= np.abs(E4M3 - want).min()          # a nearest scale
            for v, c, back in zip(x[row, part], code[row, part], val[row, part]):
                if scale == 0:                                                # rounds away: nothing is kept
                    assert c == 0 and back == 0
                    continue
                away = np.abs(np.abs(v) / scale - E2M1)
                assert away[c & 7] == away.min()                              # a nearest code
                assert back == (-1.0 if c & 8 else 1.0) * E2M1[c & 7] * scale
                assert bool(c & 8) == (v < 0)
    ties = np.array([6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0] + [0.0] * 8)
    assert quantise4(ties[None])[2][0, :8].tolist() == [6.0, 0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0]
