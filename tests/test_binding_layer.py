"""The binding's training calls on the CPU: what they hand to the library, and what they refuse.  No kernel runs; where a
call has to get past its checks, the device check and the library call are stood in for."""
import ctypes
from types import SimpleNamespace

import pytest
import torch

import gated_delta_rule_129_b200 as gdn2


def _packed(*shape):
    return gdn2.PackedAct(torch.zeros(shape, dtype=torch.int8), torch.zeros((*shape[:-1], 1), dtype=torch.uint8))


def _x(*shape):
    return torch.zeros(shape)


T4 = (1, 4, 2, 64)
BY_KEYWORD = [
    ("act_pack", dict(out=None, x=_x(*T4))),
    ("act_unpack", dict(dtype=torch.float32, packed=_packed(*T4))),
    ("act_unpack", dict(packed=list(_packed(*T4)))),
    ("token_prologue_bwd", dict(cu_seqlens=None, conv_q=_x(128, 4), conv_k=_x(128, 4), conv_v=_x(128, 4), dq=_x(*T4),
                                dk=_x(*T4), dv=_x(*T4), q_raw=_packed(*T4), k_raw=_packed(*T4), v_raw=_packed(*T4))),
    ("token_epilogue_bwd", dict(workspace=None, o=_packed(*T4), gate=_x(*T4), norm_weight=_x(64), dout=_x(*T4))),
    ("token_path_bwd", dict(scale=None, h0=None, q_raw=_x(*T4), k_raw=_x(*T4), v_raw=_x(*T4), log_alpha=_x(*T4),
                            b=_x(*T4), w=_x(*T4), gate=_x(*T4), conv_q=_x(128, 4), conv_k=_x(128, 4),
                            conv_v=_x(128, 4), norm_weight=_x(64), dout=_x(*T4))),
    ("gated_scan_fwd", dict(h0=None, v=_x(*T4), log_alpha=_x(*T4), w=_x(*T4))),
    ("gated_scan_bwd", dict(cu_seqlens=None, dO=_x(*T4), v=_x(*T4), log_alpha=_x(*T4), w=_x(*T4))),
    ("gated_scan_step", dict(out=None, v=_x(4, 2, 64), log_alpha=_x(4, 2, 64), w=_x(4, 2, 64), state=_x(4, 2, 64))),
]


@pytest.mark.parametrize("name,kw", BY_KEYWORD, ids=[f"{i}-{n}" for i, (n, _) in enumerate(BY_KEYWORD)])
def test_stream_of_another_device_is_refused_by_keyword_too(name, kw):
    """The call's device is that of its leading argument, wherever and in whatever order it is given."""
    stream = SimpleNamespace(device=torch.device("cuda", 0))
    with pytest.raises(ValueError, match="stream is on"):
        getattr(gdn2, name)(**kw, stream=stream)


def test_a_missing_leading_argument_is_named():
    stream = SimpleNamespace(device=torch.device("cuda", 0))
    with pytest.raises(TypeError, match="x"):
        gdn2.act_pack(stream=stream)
    with pytest.raises(TypeError, match="v"):
        gdn2.gated_scan_step(log_alpha=_x(4, 2, 64), w=_x(4, 2, 64), state=_x(4, 2, 64), stream=stream)


@pytest.mark.parametrize("shape", [(2 ** 32 + 128,), (2 ** 31 + 128,), (3, 2 ** 32 + 256), (2, 5, 128), (7, 1001), (4, 128, 64)])
def test_checkpoints_describe_every_value(monkeypatch, shape):
    """Rows and columns that reach the library cover the tensor, however long its rows are."""
    calls = {}
    monkeypatch.setattr(gdn2, "_cuda_device", lambda name, t: t.device)
    monkeypatch.setattr(gdn2, "_call", lambda where, device, *args: calls.update({where: args}))
    x = torch.empty(shape, dtype=torch.bfloat16, device="meta")
    p = gdn2.act_pack(x)
    gdn2.act_unpack(p)
    _, _, rows, cols, _, _ = calls["gdn2_act_pack"]
    assert calls["gdn2_act_unpack"][2:4] == (rows, cols)
    assert rows * cols == x.numel() and cols < 2 ** 31
    assert rows * -(-cols // 128) == p.exps.numel()


@pytest.mark.parametrize("D", [2 ** 31, 2 ** 31 + 1, 2 ** 32 + 1])
def test_checkpoints_refuse_rows_past_the_library(monkeypatch, D):
    """Odd rows of 2^31 values and more (2^31 itself is whole blocks, and goes through)."""
    monkeypatch.setattr(gdn2, "_cuda_device", lambda name, t: t.device)
    monkeypatch.setattr(gdn2, "_call", lambda *a: None)
    x = torch.empty(2, D, dtype=torch.bfloat16, device="meta")
    p = gdn2.PackedAct(torch.empty(2, D, dtype=torch.int8, device="meta"),
                       torch.empty(2, -(-D // 128), dtype=torch.uint8, device="meta"))
    if D % 128 == 0:
        gdn2.act_pack(x), gdn2.act_unpack(p)
        return
    with pytest.raises(ValueError, match="D"):
        gdn2.act_pack(x)
    with pytest.raises(ValueError, match="D"):
        gdn2.act_unpack(p)


class _Library:
    """Stands in for the scan's calls: each writes the status it is told to the workspace's first word."""

    def __init__(self, monkeypatch, **status):
        monkeypatch.setattr(gdn2, "_cuda_device", lambda name, t: t.device)
        monkeypatch.setattr(gdn2, "_call", lambda where, device, desc, *a: self.call(where, desc._obj))
        self.status, self.calls = status, []

    def call(self, where, desc):
        self.calls.append(where)
        ctypes.c_int32.from_address(desc.workspace).value = self.status[where]


@pytest.mark.parametrize("fwd,bwd,want", [(0, 0, 0), (8, 0, 8), (0, 8, 8), (5, 5, 5)])
@pytest.mark.parametrize("dtype", [torch.uint8, torch.float32])
def test_backward_keeps_the_status_of_the_states_it_computes_again(monkeypatch, fwd, bwd, want, dtype):
    lib = _Library(monkeypatch, gdn2_gated_scan_fwd=fwd, gdn2_gated_scan_bwd=bwd)
    ws = torch.full((65536,), 77, dtype=dtype)
    gdn2.gated_scan_bwd(_x(*T4), _x(*T4), _x(*T4), _x(*T4), workspace=ws)
    assert lib.calls == ["gdn2_gated_scan_fwd", "gdn2_gated_scan_bwd"]
    assert int(ws.view(torch.uint8)[:4].view(torch.int32)) == want


def test_backward_from_kept_states_reports_its_own_status(monkeypatch):
    _Library(monkeypatch, gdn2_gated_scan_bwd=0)
    ws = torch.full((65536,), 77, dtype=torch.uint8)
    gdn2.gated_scan_bwd(_x(*T4), _x(*T4), _x(*T4), _x(*T4), workspace=ws, chunk_states=_x(1, 2, 64))
    assert int(ws[:4].view(torch.int32)) == 0
