"""The cache operators as they are used together (marked gpu): a prompt's queries and keys
normed, rotated and appended, then decode steps over the cache, windowed or not, on one
GPU and as a rank of a group."""
import math
import socket

import numpy as np
import pytest
import torch
import torch.distributed as dist

import oracle
import sequence_sharded_paged_b200 as dcp
import synth
from sequence_sharded_paged_b200 import parallel
from sequence_sharded_paged_b200 import workload as wl

from op_ref import Cache, attention, bf16, check, frequencies, norm, quantise4, rotate, rows

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clear_status():
    dcp.dcp_get_device_status()
    yield
    assert dcp.dcp_get_device_status() == dcp.DCP_OK


def to_bf16(x):
    return torch.as_tensor(x).to(torch.float32).to(torch.bfloat16).cuda()


@pytest.mark.parametrize("window,sinks", [(None, 0), (70, 3)])
@pytest.mark.parametrize("dtype", ["bf16", "fp4"])
def test_prompt_and_decode_steps(dtype, window, sinks):
    """Prompts of different lengths in one padded call, then three decode steps of two query tokens each; the
    rows that the library's own read-back returns are the reference's rows."""
    hq, hkv, d, page, n, i = 8, 2, 64, 16, 2, 16
    L = [90, 0, 151]
    rng = np.random.default_rng(31)
    empty = [np.zeros((0, hkv, d))] * 3
    c = Cache(dtype, empty, empty, hq=hq, hkv=hkv, d=d, page=page, n=n, i=i, room=100)
    if dtype == "bf16":  # nothing that was never written may be read: the pools stay NaN
        assert torch.isnan(c.k_pages).all()
    rope = dcp.make_rope(d, theta=1e4)
    f, factor = frequencies(d, 1e4)
    w = bf16(rng.standard_normal(d) * 0.2 + 1)
    lens = list(L)

    def tokens(req, pos):
        qkv = bf16(rng.standard_normal((len(req), hq + 2 * hkv, d)))
        t = to_bf16(qkv)
        q_out = torch.empty((len(req), hq, d), dtype=torch.bfloat16, device="cuda")
        dcp.dcp_norm_rope_append(c.desc, rope, torch.tensor(req, dtype=torch.int32).cuda(),
                                 torch.tensor(pos, dtype=torch.int32).cuda(), t[:, :hq], t[:, hq:hq + hkv],
                                 t[:, hq + hkv:], to_bf16(w), to_bf16(w), 1e-6, q_out)
        want = rotate(norm(qkv[:, :hq], w, 1e-6), np.maximum(pos, 0), f, factor, "half")
        live = np.array(pos) >= 0
        assert np.abs(q_out.double().cpu().numpy() - want)[live].max() <= 2 ** -8 * np.abs(want).max() + 1e-4
        return q_out

    # the prompts, padded to the longest
    tokens([b for b in range(3) for _ in range(max(L))], [p if p < L[b] else -1 for b in range(3) for p in range(max(L))])
    for _ in range(3):
        new = [(b, lens[b] + j) for b in range(3) for j in range(2)]
        q = tokens([b for b, _ in new], [p for _, p in new]).view(3, 2, hq, d)
        lens = [x + 2 for x in lens]
        c.lengths = np.array(lens)
        seq = torch.tensor(lens, dtype=torch.int32).cuda()
        out, lse = torch.empty((3, 2, hq, d), device="cuda"), torch.empty((3, 2, hq), device="cuda")
        if window is None and dtype == "bf16":  # several query tokens of 4 heads: the windowed call serves them
            size = dcp.dcp_decode_window_workspace_size(c.desc, 3, 2, 2 ** 31 - 1)
            dcp.dcp_decode_window(c.desc, q, seq, 2 ** 31 - 1, 0, out, lse, torch.empty(size, dtype=torch.uint8, device="cuda"))
        elif window is None:
            size = dcp.dcp_decode_workspace_size_ex(c.desc, 3, 2, dcp.DCP_DECODE_MERGED)
            dcp.dcp_decode_merged(c.desc, q, seq, out, lse, torch.empty(size, dtype=torch.uint8, device="cuda"))
        else:
            size = dcp.dcp_decode_window_workspace_size(c.desc, 3, 2, window, sinks)
            dcp.dcp_decode_window(c.desc, q, seq, window, sinks, out, lse, torch.empty(size, dtype=torch.uint8, device="cuda"))
        for b in range(3):
            pos = torch.arange(lens[b], dtype=torch.int32, device="cuda")
            k, v = (torch.empty((lens[b], hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
            dcp.dcp_kv_gather(c.desc, torch.full_like(pos, b), pos, k, v)
            c.k[b], c.v[b] = k.double().cpu().numpy(), v.double().cpu().numpy()
        check("step", out, lse, *attention(c, q.double().cpu().numpy(), window=window, sinks=sinks),
              max(np.abs(x).max() for x in c.v))


def test_fp4_workload():
    """The workload helper's 4-bit cache: its rows are the seeded rows after quantisation."""
    w = synth.Workload("gqa fp4", "gqa", "fp4", 2, 16, 2, 64, 64, 16, 2, 1, 1 / 8, 71, 1071)
    w.lengths = np.array([130, 33])
    assert w.kv_bytes_per_token == 2 * 2 * (32 + 4)
    dw = wl.build(w, oracle.shard_counts(w.lengths, 2, 1))
    assert dw.kv_bytes == 163 * w.kv_bytes_per_token
    pos = torch.arange(130, dtype=torch.int32, device="cuda")
    k, v = (torch.empty((130, 2, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    req = torch.zeros_like(pos)
    dcp.dcp_kv_gather(dw.desc, req, pos, k, v)
    ks, vs = synth.device.gqa_rows(w.seed_val, req, pos, 2, 64)
    np.testing.assert_array_equal(k.double().cpu().numpy(), quantise4(ks.double().cpu().numpy())[2])
    np.testing.assert_array_equal(v.double().cpu().numpy(), quantise4(vs.double().cpu().numpy())[2])


@pytest.mark.parametrize("dtype", ["bf16", "fp4"])
def test_windowed_decode_on_a_one_rank_nccl_group(dtype):
    hq, hkv, d = 16, 2, 64
    rng = np.random.default_rng(5)
    c = Cache(dtype, [rows(rng, n, hkv, d) for n in (200, 31)], [rows(rng, n, hkv, d) for n in (200, 31)], hq=hq,
              hkv=hkv, d=d, page=16, n=1, i=1)
    q = bf16(rng.standard_normal((2, 1, hq, d)))
    with socket.socket() as s:
        s.bind(("127.0.0.1", 0))
        port = s.getsockname()[1]
    store = dist.TCPStore("127.0.0.1", port, 1, True)
    dist.init_process_group("nccl", store=store, rank=0, world_size=1, device_id=torch.device("cuda", 0))
    try:
        ws = parallel.rank_workspace(c.desc, 2, device="cuda", rank=0, window=50, n_sinks=2)
        out, lse = parallel.decode_distributed(c.desc, 0, 1, to_bf16(q)[:, 0], c.seq_lens, ws, window=50, n_sinks=2)
        torch.cuda.synchronize()
    finally:
        dist.destroy_process_group()
    check("one-rank group", out, lse, *attention(c, q, window=50, sinks=2), max(np.abs(x).max() for x in c.v))


@pytest.mark.parametrize("group", [2, 16])
def test_4bit_shares_of_many_groups(group):
    """So many tokens that a warp's share is longer than what it sums before O goes to memory.  All requests
    read the same pages, so the cache itself is small."""
    B, hkv, d, page, L = 96, 8, 64, 64, 32 * 1024 + 5
    hq = hkv * group
    pages = -(-L // page)
    g = torch.Generator("cuda").manual_seed(3)
    bt = torch.arange(pages, dtype=torch.int32, device="cuda").expand(1, B, pages).contiguous()
    kp = torch.empty((pages, hkv, page * (d // 2 + d // 16)), dtype=torch.uint8, device="cuda")
    vp = torch.empty_like(kp)
    desc = dcp.make_cache_desc(kind=dcp.DCP_GQA, dtype=dcp.DCP_FP4_E2M1, n_shards=1, interleave=1, page_size=page,
                               num_pages=pages, hq=hq, hkv=hkv, dk=d, dv=d, scale=1 / math.sqrt(d), batch=B,
                               block_tables=bt, k_pages=kp, v_pages=vp)
    k, v = (torch.randn((L, hkv, d), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    # a mean apart from 0 and growing scores: both O and the reference move on all the way
    v += 0.25
    k *= torch.linspace(0.1, 1.5, L, device="cuda")[:, None, None].to(torch.bfloat16)
    pos = torch.arange(L, dtype=torch.int32, device="cuda")
    dcp.dcp_kv_append(desc, torch.zeros_like(pos), pos, k, v)
    dcp.dcp_kv_gather(desc, torch.zeros_like(pos), pos, k, v)
    q = torch.randn((B, hq, d), generator=g, device="cuda").to(torch.bfloat16)
    lens = torch.full((B,), L, dtype=torch.int32, device="cuda")
    lens[3], lens[-1] = 1, L - 4096
    out, lse = torch.empty((B, hq, d), device="cuda"), torch.empty((B, hq), device="cuda")
    size = dcp.dcp_decode_workspace_size_ex(desc, B, 1, dcp.DCP_DECODE_MERGED)
    dcp.dcp_decode_merged(desc, q, lens, out, lse, torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda"))
    O, lse_ref = torch.empty((B, hq, d), dtype=torch.float64), torch.empty((B, hq), dtype=torch.float64)
    for b in range(B):
        n = int(lens[b])
        kd, vd = k[:n].double(), v[:n].double()
        s = torch.einsum("gjd,pgd->gjp", q[b].double().view(hkv, group, d), kd) / math.sqrt(d)
        O[b] = torch.einsum("gjp,pgd->gjd", s.softmax(-1), vd).reshape(hq, d)
        lse_ref[b] = s.logsumexp(-1).reshape(hq)
    # 96 * 8 segments of 2049 groups over at least 1184 warps: under 1400 groups a warp, whose O
    # is cut off once a group (8 rows at most) or, between two stores, 512 times: 2^-23 of at
    # most max|V| each, and the sum of the weights as often; 2.1e-5 of every weight twice
    # (op_ref).  The sum of the weights in LSE takes 700 steps of 2^-24 each, beside op_ref's 5e-5.
    tol_o = (2 * 1400 * 2.0 ** -23 + 2 * 2.1e-5) * float(v.abs().max())
    assert (out.double().cpu() - O).abs().max() <= tol_o
    assert (lse.double().cpu() - lse_ref).abs().max() <= 5e-5 + 700 * 2.0 ** -24


@pytest.mark.parametrize("start,T", [(0, 4), (0, 130), (1, 7), (2, 3), (3, 61), (5, 200), (64, 1)])
@pytest.mark.parametrize("d,hkv,page,n,i", [(64, 3, 16, 2, 16), (128, 1, 64, 1, 1), (128, 2, 16, 3, 5)])
def test_4bit_append_of_consecutive_tokens(d, hkv, page, n, i, start, T):
    """Prompt rows from any first position: stored exactly, nothing beside them touched, and read back into
    tensors that begin on a 16-byte boundary only."""
    pages = 24
    rng = np.random.default_rng(T + d)
    bt = torch.as_tensor(rng.permutation(n * pages).astype(np.int32).reshape(n, 1, pages)).cuda()
    block = page * (d // 2 + d // 16)
    kp, vp = (torch.full((n * pages, hkv, block), 0xA5, dtype=torch.uint8, device="cuda") for _ in range(2))
    desc = dcp.make_cache_desc(kind=dcp.DCP_GQA, dtype=dcp.DCP_FP4_E2M1, n_shards=n, interleave=i, page_size=page,
                               num_pages=n * pages, hq=hkv, hkv=hkv, dk=d, dv=d, scale=1.0, batch=1, block_tables=bt,
                               k_pages=kp, v_pages=vp)
    pos = np.arange(start, start + T)
    k, v = (bf16(rng.standard_normal((T, hkv, d)) * 5) for _ in range(2))

    def at16(x):  # a copy of x that lies 16 bytes after a 32-byte boundary
        room = torch.empty(x.numel() + 8, dtype=torch.bfloat16, device="cuda")
        room[8:] = x.flatten()
        return room[8:].view(x.shape)

    dpos = torch.as_tensor(pos.astype(np.int32)).cuda()
    req = torch.zeros_like(dpos)
    dcp.dcp_kv_append(desc, req, dpos, at16(to_bf16(k)), at16(to_bf16(v)))
    for pool, x in ((kp, k), (vp, v)):
        code, sb, _ = quantise4(x)
        want = np.full((n * pages, hkv, block), 0xA5, np.uint8)
        for t, p in enumerate(pos):
            loc = (p // (i * n)) * i + p % i
            pg, off = int(bt[(p // i) % n, 0, loc // page]), loc % page
            want[pg, :, off * (d // 2):(off + 1) * (d // 2)] = code[t][:, 0::2] | (code[t][:, 1::2] << 4)
            want[pg, :, page * (d // 2) + np.arange(d // 16) * page + off] = sb[t].T
        np.testing.assert_array_equal(pool.cpu().numpy(), want)
    for shift in (0, 8):
        ko, vo = (torch.empty(T * hkv * d + 8, dtype=torch.bfloat16, device="cuda")[shift:shift + T * hkv * d]
                  .view(T, hkv, d) for _ in range(2))
        dcp.dcp_kv_gather(desc, req, dpos, ko, vo)
        np.testing.assert_array_equal(ko.double().cpu().numpy(), quantise4(k)[2])
        np.testing.assert_array_equal(vo.double().cpu().numpy(), quantise4(v)[2])


@pytest.mark.parametrize("q_len", [1, 3])
def test_4bit_decode_on_two_streams_and_in_a_graph(q_len):
    """Two calls at once with a workspace each, and a captured call replayed after the cache has grown."""
    hq, hkv, d = 16, 2, 128
    rng = np.random.default_rng(77)
    c = Cache("fp4", [rows(rng, L, hkv, d) for L in (700, 9, 3000)], [rows(rng, L, hkv, d) for L in (700, 9, 3000)],
              hq=hq, hkv=hkv, d=d, page=16, n=2, i=16, room=40)
    size = dcp.dcp_decode_workspace_size_ex(c.desc, 3, q_len, dcp.DCP_DECODE_MERGED)
    shape = (3, q_len, hq, d)
    q = [bf16(rng.standard_normal(shape)) for _ in range(2)]
    dq = [to_bf16(x) for x in q]
    out = [torch.empty(shape, device="cuda") for _ in range(2)]
    lse = [torch.empty(shape[:3], device="cuda") for _ in range(2)]
    ws = [torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for k, s in enumerate(streams):
            dcp.dcp_decode_merged(c.desc, dq[k], c.seq_lens, out[k], lse[k], ws[k], stream=s)
    torch.cuda.synchronize()
    vmax = max(np.abs(x).max() for x in c.v)
    for k in range(2):
        check(f"stream {k}", out[k], lse[k], *attention(c, q[k]), vmax)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dcp.dcp_decode_merged(c.desc, dq[0], c.seq_lens, out[0], lse[0], ws[0])
        dcp.dcp_decode_merged(c.desc, dq[1], c.seq_lens, out[1], lse[1], ws[0])  # in order: the same workspace
    new_k, new_v = rows(rng, 3, hkv, d), rows(rng, 3, hkv, d)
    dcp.dcp_kv_append(c.desc, None, c.seq_lens, to_bf16(new_k), to_bf16(new_v))
    c.seq_lens += 1
    for b in range(3):
        c.k[b] = np.concatenate((c.k[b], quantise4(new_k[b:b + 1])[2]))
        c.v[b] = np.concatenate((c.v[b], quantise4(new_v[b:b + 1])[2]))
    c.lengths = c.lengths + 1
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for k in range(2):
        check(f"replay {k}", out[k], lse[k], *attention(c, q[k]), vmax)
