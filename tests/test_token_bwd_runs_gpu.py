"""gdn2_token_prologue_bwd over long runs.  A warp walks one run of tokens, eight a stage, with the rows' powers read 32
rows ahead and a stage without masks wherever the run is inside one sequence; here the runs are more than 64 tokens, so
every form of the kernel refills its powers twice at least and takes that stage most of the time.  Every row is held to the bound that
tests/token_bwd_reference.py derives, from rows whose scales (and so their 8-bit powers) change from row to row, with
sequence borders at every place of a stage.

The tap gradients add up 16 K tokens.  Errors of different tokens are independent, so they add up as the terms do, and
the relative error of the sums stays that of a row: 1e-5 (rel-L2, per head), the bar of the shorter sums too.
"""
import ctypes
import random

import pytest

from tests.token_bwd_reference import C, prologue_gradients

pytestmark = pytest.mark.gpu

H, T = 16, 16384 + 37


@pytest.fixture(scope="module")
def gdn2(cuda_device):
    import gated_delta_rule_129_b200 as mod
    mod.load_library()
    return mod


def _run_length(gdn2, dk, dv, W, io):
    """Tokens of a warp's run at least, from the room for the blocks' partial sums (four warps a block)."""
    d = gdn2.make_desc(1, T, H, dk, dv, gdn2.GDN2_IO_BF16 if io == "bf16" else gdn2.GDN2_IO_F32)
    size = gdn2.load_library().gdn2_token_prologue_bwd_workspace_size(ctypes.byref(d), W)
    return T / (4 * size / (4 * H * W * (2 * dk + dv)))


def _borders(seed):
    """Sequences of 1 to 9 tokens, around a stage and a run, and long ones, in a random order."""
    r = random.Random(seed)
    lens = [1, 1, 1, 2, 2, 3, 4, 5, 6, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 110, 111, 112, 250, 333, 700, 1000, 0, 0]
    lens += [1500, 2100, 3001]
    r.shuffle(lens)
    lens.append(T - sum(lens))
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def _check(gdn2, dk, dv, W, io, packed, cu):
    import torch
    assert _run_length(gdn2, dk, dv, W, io) > 64
    dt = torch.float32 if io == "f32" else torch.bfloat16
    g = torch.Generator(device="cuda")
    g.manual_seed(W + dk + 2 * dv)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    dims = dict(q=dk, k=dk, v=dv)
    scale = torch.exp2(torch.randint(-14, 1, (1, T, H, 1), generator=g, device="cuda").float())
    x = {c: (n(1, T, H, d) * scale).to(dt) for c, d in dims.items()}
    taps, dy = {c: 0.5 * n(H * d, W) for c, d in dims.items()}, {c: n(1, T, H, d) for c, d in dims.items()}
    kept = {c: gdn2.act_pack(a) for c, a in x.items()} if packed else x
    if packed:
        x = {c: p.codes.double() * torch.exp2(p.exps.double() - 127) for c, p in kept.items()}
    got = gdn2.token_prologue_bwd(*kept.values(), *taps.values(), *dy.values(),
                                  None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda"), dtype=dt)
    for c, d in dims.items():
        dx, dtap, bound, _ = prologue_gradients(x[c][0], taps[c], dy[c][0], [0, T] if cu is None else cu, c != "v")
        err = (got[c + "_raw"][0].double() - dx).norm(dim=-1)
        if io == "bf16":
            err -= 2.0 ** -8 * dx.norm(dim=-1)
        assert (err / bound).max().item() <= C, c
        off = (got["conv_" + c].double() - dtap).reshape(H, d * W).norm(dim=1) / dtap.reshape(H, d * W).norm(dim=1)
        assert off.max().item() <= 1e-5, c


@pytest.mark.parametrize("form", ["f32", "bf16", "f32 packed", "bf16 packed"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("W", range(1, 9))
def test_long_runs_with_borders(gdn2, W, d, form):
    _check(gdn2, d, d, W, form.split()[0], "packed" in form, _borders(10 * W + d))


@pytest.mark.parametrize("form", ["f32", "bf16 packed"])
@pytest.mark.parametrize("dk,dv,W", [(64, 128, 4), (128, 64, 5)])
def test_long_runs_of_two_widths(gdn2, dk, dv, W, form):
    _check(gdn2, dk, dv, W, form.split()[0], "packed" in form, _borders(dk))


@pytest.mark.parametrize("form", ["bf16", "f32 packed"])
def test_long_runs_of_one_sequence(gdn2, form):
    _check(gdn2, 128, 128, 4, form.split()[0], "packed" in form, None)
