"""8-bit checkpoints of rows of around and past 2^31 values, and past 2^32: the first and last blocks against the oracle,
and nothing but zeros between.  Both directions are exact, so everything is compared for equality."""
import numpy as np
import pytest

from oracle import act_pack as ap

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gdn2(cuda_device):
    import gated_delta_rule_129_b200 as mod
    mod.load_library()
    return mod


@pytest.mark.parametrize("D", [2 ** 31 - 1, 2 ** 31 + 128, 2 ** 32 + 128])
def test_long_rows(gdn2, D):
    import torch
    head = np.random.default_rng(1).standard_normal(256).astype(np.float32)
    tail = (D - 1) % 128 + 1 + 128                       # the last block and the one before it
    end = np.random.default_rng(2).standard_normal(tail).astype(np.float32) * 16
    bf = lambda a: torch.from_numpy(a).cuda().bfloat16()  # noqa: E731
    x = torch.zeros(D, dtype=torch.bfloat16, device="cuda")
    x[:256], x[-tail:] = bf(head), bf(end)
    p = gdn2.act_pack(x)
    for part, exps, codes in ((x[:256], p.exps[:2], p.codes[:256]), (x[-tail:], p.exps[-2:], p.codes[-tail:])):
        rc, re = ap.pack(part.float().cpu().numpy()[None])
        np.testing.assert_array_equal(codes.cpu().numpy(), rc[0])
        np.testing.assert_array_equal(exps.cpu().numpy(), re[0])
    assert not bool(p.codes[256:-tail].any()) and bool((p.exps[2:-2] == 1).all())
    y = gdn2.act_unpack(p, out=x)
    for part, exps, codes in ((y[:256], p.exps[:2], p.codes[:256]), (y[-tail:], p.exps[-2:], p.codes[-tail:])):
        np.testing.assert_array_equal(part.double().cpu().numpy(), ap.unpack(codes.cpu().numpy()[None], exps.cpu().numpy()[None])[0])
    assert not bool(y[256:-tail].any())
