"""gdn2_token_prologue_bwd on rows of very large values: up to a row norm of 1e18 (where the sum of squares still fits
fp32) the q and k gradients hold the fp32 bar row by row, beside ordinary rows and on their own.  The bar is derived in
tests/token_bwd_reference.py; a gradient stored in bf16 is half a step, 2^-8, farther off."""
import pytest

from tests.token_bwd_reference import C, prologue_gradients

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gdn2(cuda_device):
    import gated_delta_rule_129_b200 as mod
    mod.load_library()
    return mod


@pytest.mark.parametrize("dy_scale", [1.0, 1e-6])
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("d,W", [(128, 4), (64, 4), (128, 1), (64, 7)])
@pytest.mark.parametrize("scale", [1e12, 1e13, 1e14, 1e15, 1e16, 1e17])
@pytest.mark.parametrize("every", [1, 9])
def test_large_rows(gdn2, d, W, scale, every, io, dy_scale):
    import torch
    dt = torch.float32 if io == "f32" else torch.bfloat16
    g = torch.Generator(device="cuda")
    g.manual_seed(int(scale) % 1000 + d + W + every)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    T, H, cu = 60, 2, [0, 23, 24, 60]
    rows = torch.where(torch.arange(T, device="cuda") % every == 0, scale, 1.0).reshape(1, T, 1, 1)
    x = {c: (n(1, T, H, d) * rows).to(dt) for c in "qk"}
    x["v"] = n(1, T, H, d).to(dt)
    taps, dy = {c: 0.5 * n(H * d, W) for c in "qkv"}, {c: dy_scale * n(1, T, H, d) for c in "qkv"}
    got = gdn2.token_prologue_bwd(*x.values(), *taps.values(), *dy.values(),
                                  torch.tensor(cu, dtype=torch.int32, device="cuda"))
    for c in "qkv":
        dx, dtap, bound, tap_bound = prologue_gradients(x[c][0], taps[c], dy[c][0], cu, c != "v")
        err = (got[c + "_raw"][0].double() - dx).norm(dim=-1)
        half = 2.0 ** -8 * dx.norm(dim=-1) if io == "bf16" else 0.0
        worst = ((err - half) / bound).max().item()
        assert worst <= C, (c, worst)
        # sums over 60 tokens: 60 * 2^-24 more
        off = (got["conv_" + c].double() - dtap).reshape(H, d, W).norm(dim=1)
        assert bool((off <= (C + 60 * 2.0 ** -24) * tap_bound).all()), c


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("scale", [1e-20, 1e-3, 1e6, 1e12, 1e15, 1e18])
def test_epilogue_large_and_small_rows(gdn2, scale, d, io):
    """The RMS norm's backward: do within C of r |dn| (row sums of two times, the root, six roundings: as the prologue's
    rows), at every scale whose sum of squares fits fp32 and down to rows that the eps outweighs."""
    import torch
    dt = torch.float32 if io == "f32" else torch.bfloat16
    g = torch.Generator(device="cuda")
    g.manual_seed(d)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    rows = torch.where(torch.arange(40, device="cuda") % 3 == 0, scale, 1.0).reshape(1, 40, 1, 1)
    o, gate, dout = (n(1, 40, 3, d) * rows).to(dt), n(1, 40, 3, d).to(dt), n(1, 40, 3, d).to(dt)
    wt = torch.rand(d, generator=g, device="cuda") + 0.5
    got = gdn2.token_epilogue_bwd(o, gate, wt, dout)
    x, sig = o.double(), torch.sigmoid(gate.double())
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6)
    y, dn = x * r, dout.double() * wt.double() * sig
    half = 2.0 ** -8 if io == "bf16" else 0.0
    for name, ref, scale_of in (("o", r * (dn - y * (y * dn).mean(-1, keepdim=True)), r[..., 0] * dn.norm(dim=-1)),
                                ("gate", dn * y * (1 - sig), (dn * y).norm(dim=-1))):
        off = (got[name].double() - ref).norm(dim=-1) - half * ref.norm(dim=-1)
        assert (off / scale_of).max().item() <= C, name
