"""gdn2_token_epilogue_bwd at every opening of the gate, element by element against 64 bits: the gate's gradient
dout n weight sig(g) (1 - sig(g)) keeps its relative accuracy where sig(g) is 1 to all of fp32's digits.

The bar, 1e-5 of an element: exp(-g)'s argument is rounded (|g| 2^-24: 4.8e-6 at 80), the exponential and the reciprocal
(on both factors) are within 2^-22 (7e-7), n's row sum and root within 1e-6, six products within 2^-24 each (4e-7):
7e-6 in all.  Factors below 2^-126 count as zero, so elements get that much, times dout n weight, on top; gradients stored in
bf16 half a step, 2^-8."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gdn2(cuda_device):
    import gated_delta_rule_129_b200 as mod
    mod.load_library()
    return mod


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("packed", [False, True])
def test_gate_gradient_of_open_and_shut_gates(gdn2, d, io, packed):
    import torch
    dt = torch.float32 if io == "f32" else torch.bfloat16
    g = torch.Generator(device="cuda")
    g.manual_seed(d)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    T, H = 162, 3
    gate = (torch.arange(-80, 82, device="cuda").float().reshape(1, T, 1, 1).clamp(max=80) + 0.3 * n(1, T, H, d).clamp(-1, 1)).to(dt)
    o, dout, wt = n(1, T, H, d).to(dt), n(1, T, H, d).to(dt), torch.rand(d, generator=g, device="cuda") + 0.5
    kept = gdn2.act_pack(gate) if packed else gate
    if packed:
        gate = gdn2.act_unpack(kept, torch.float32)
    got = gdn2.token_epilogue_bwd(o, kept, wt, dout)["gate"].double()
    x, gt = o.double(), gate.double()
    scale = dout.double() * x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * wt.double()
    ref = scale * torch.sigmoid(gt) * torch.sigmoid(-gt)
    bar = 1e-5 * ref.abs() + 2.0 ** -126 * (1 + scale.abs())
    if io == "bf16":
        bar += 2.0 ** -8 * ref.abs()
    off = (got - ref).abs()
    assert bool((off <= bar).all()), (off / ref.abs()).amax((0, 2, 3)).tolist()


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), 200.0, -200.0, 3e38, -3e38])
def test_gates_past_the_exponential(gdn2, value):
    """A gate that is wholly open or shut has no gradient; a NaN stays one, in its element alone."""
    import torch
    torch.manual_seed(1)
    o, dout, wt = torch.randn(1, 9, 2, 64, device="cuda"), torch.randn(1, 9, 2, 64, device="cuda"), torch.ones(64, device="cuda")
    gate = torch.randn_like(o)
    gate[0, 4, 1] = value
    gate[0, 7, 0, 5] = float("nan")
    r = gdn2.token_epilogue_bwd(o, gate, wt, dout)
    assert not bool(r["gate"][0, 4, 1].any()) and bool(torch.isfinite(r["o"][0, 4, 1]).all())
    bad = torch.isnan(r["gate"])
    assert bool(bad[0, 7, 0, 5]) and int(bad[0, :7].sum()) == 0 and int(bad[0, 8].sum()) == 0 and int(bad[0, 7, 1].sum()) == 0
