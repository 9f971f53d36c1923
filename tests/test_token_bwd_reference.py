"""The vectorised fp64 reference of the prologue's gradients (tests/token_bwd_reference.py) against the oracle's loops."""
import numpy as np
import pytest
import torch

from oracle import token_path_backward as tb
from tests.token_bwd_reference import prologue_gradients


@pytest.mark.parametrize("lens", [[13], [3, 0, 1, 6, 2, 0]])
@pytest.mark.parametrize("W", [1, 2, 4, 8])
def test_reference_matches_oracle(W, lens):
    rng = np.random.default_rng(W)
    T, H, d = sum(lens), 2, 5
    cu = np.concatenate([[0], np.cumsum(lens)])
    x = {c: rng.standard_normal((1, T, H, d)) for c in "qkv"}
    w = {c: rng.standard_normal((H * d, W)) for c in "qkv"}
    dy = {c: rng.standard_normal((1, T, H, d)) for c in "qkv"}
    ref = tb.prologue_bwd(*x.values(), *w.values(), *dy.values(), cu)
    for c in "qkv":
        dx, dt, bound, tap_bound = prologue_gradients(*(torch.from_numpy(a) for a in (x[c][0], w[c], dy[c][0])), cu, c != "v")
        np.testing.assert_allclose(dx.numpy(), ref[c + "_raw"][0], rtol=1e-10, atol=1e-12)
        np.testing.assert_allclose(dt.numpy(), ref["conv_" + c], rtol=1e-10, atol=1e-12)
        assert np.all(np.linalg.norm(ref[c + "_raw"][0], axis=-1) <= 1.1 * bound.numpy() * (1 + 1e-12))
        assert np.all(np.linalg.norm(ref["conv_" + c].reshape(H, d, W), axis=1) <= 1.1 * tap_bound.numpy() * (1 + 1e-12))
