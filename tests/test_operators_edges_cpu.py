"""Ends of the ranges of the operators around the decode, host side, without a GPU."""
import pytest
import torch

import sequence_sharded_paged_b200 as dcp

from test_operators_cpu import gqa


class OnDevice:
    """Stands for a tensor on GPU `index`, as far as the binding's checks look at one."""

    def __init__(self, shape, dtype, index=0, strides=None):
        self.host = torch.empty(shape, dtype=dtype)
        self.shape, self.dtype, self.device, self.index = self.host.shape, dtype, f"cuda:{index}", index
        self.strides = strides

    def get_device(self):
        return self.index

    def is_contiguous(self):
        return self.strides is None

    def stride(self):
        return self.strides or self.host.stride()

    def data_ptr(self):
        return 1024

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.host.numel()

    def element_size(self):
        return self.host.element_size()


def decode(name, desc, ws, q_len=1):
    q = OnDevice((3, q_len, 16, 128), torch.bfloat16)
    out, lse = OnDevice((3, q_len, 16, 128), torch.float32), OnDevice((3, q_len, 16), torch.float32)
    lens = OnDevice((3,), torch.int32)
    call = getattr(dcp, name)
    if name == "dcp_decode_window":
        call(desc, q, lens, 8, 0, out, lse, ws, stream=7)
    elif name == "dcp_decode_rank":
        call(desc, 0, q, lens, out, lse, ws, stream=7)
    else:
        call(desc, q, lens, out, lse, ws, stream=7)


@pytest.mark.parametrize("ws,why", [
    (torch.zeros(1 << 12, dtype=torch.uint8), "on cpu, not on the current CUDA device"),
    (OnDevice((1 << 12,), torch.uint8, index=1), "on cuda:1, not on the current CUDA device"),
    (OnDevice((1 << 12,), torch.uint8, strides=(2,)), "not contiguous"),
    (OnDevice((1 << 12,), torch.uint8), None),
], ids=["host", "another GPU", "strided view", "good"])
@pytest.mark.parametrize("name", ["dcp_decode_window", "dcp_decode_merged", "dcp_decode_partial",
                                  "dcp_decode_partial_multi", "dcp_decode_rank"])
def test_streamed_decode_checks_its_workspace(monkeypatch, name, ws, why):
    """The kernel writes partials through that pointer: what it could not write is refused before the call."""
    calls = []

    def entry(*args):
        calls.append(args)
        return dcp.DCP_OK

    monkeypatch.setattr(dcp, "_device", lambda: 0)
    monkeypatch.setattr(dcp, "_torch", torch)
    monkeypatch.setattr(dcp, "lib", lambda: type("Library", (), {name: staticmethod(entry)}))
    if why is None:
        decode(name, gqa(), ws)
        assert len(calls) == 1 and calls[0][-2] == 1 << 12
    else:
        with pytest.raises(ValueError, match=why):
            decode(name, gqa(), ws)
        assert not calls


@pytest.mark.parametrize("attn", [1e300, 3.5e38, 1e-60, 5e-324])
def test_rope_refuses_an_attention_factor_that_32_bits_do_not_hold(attn):
    """Stored in 32 bits it would be infinite or 0: every rotated value would be."""
    rope = dcp.Rope()
    with pytest.raises(dcp.DcpError) as e:
        dcp.dcp_rope_init(rope, 64, dcp.DCP_ROPE_HALF, 1e4, attn_factor=attn)
    assert e.value.status == dcp.DCP_ERR_INVALID_ARG
    assert rope.rot_dim == 0  # left as it was


@pytest.mark.parametrize("attn", [3e38, 1e-37, 1.0])
def test_rope_keeps_an_attention_factor_that_32_bits_hold(attn):
    assert abs(dcp.make_rope(64, attn_factor=attn).attn_factor - attn) <= attn * 2.0 ** -24
