"""token_path_bwd, the whole layer backwards, against chained fp64 oracles in the forms that a layer has: heads of 64 and
128, key and value heads of different width, bf16 rows, kept as they were or in 8 bits.

fp32 I/O: the operator's fp32 bar, 1e-4, as in the shorter test.  bf16 I/O: the oracles round where the library stores
bf16 (q, k, v, the operator's output and its gradient), and what is left is the operator's own bf16 error, whose bar is
2e-2 of its output o in rel-L2.  The epilogue divides o by its row's norm, which can double a relative error; its
gradients with respect to o, gate and weight are of first order in it, and what chunk_bwd and the prologue make of dO is
linear in it: twice 2e-2, half a step (2^-8) of each of the three bf16 stores on the way (q, k, v; o and dO; the result)
added: 5.5e-2."""
import numpy as np
import pytest

import oracle
import oracle.backward as ob
from oracle import act_pack as ap
from oracle import token_path as tp
from oracle import token_path_backward as tb
from tests.helpers import rel_l2
from workloads import make_inputs, round_bf16

pytestmark = pytest.mark.gpu

BAR = {"f32": 1e-4, "bf16": 2 * 2e-2 + 4 * 2.0 ** -8}


@pytest.fixture(scope="module")
def gdn2(cuda_device):
    import gated_delta_rule_129_b200 as mod
    mod.load_library()
    return mod


def _value(x):
    return ap.unpack(*ap.pack(x.reshape(-1, x.shape[-1]))).reshape(x.shape)


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("dk,dv,lens", [(128, 128, [75, 0, 1, 64]), (64, 128, [100, 33]), (128, 64, None), (64, 64, None)])
def test_layer_backward_matches_chained_oracles(gdn2, dk, dv, lens, io, packed):
    import torch
    B, T = (1, sum(lens)) if lens else (2, 70)
    H, N = 2, len(lens) if lens else 2
    dt = torch.float32 if io == "f32" else torch.bfloat16
    st = (lambda a: round_bf16(np.asarray(a, np.float32))) if io == "bf16" else (lambda a: np.asarray(a, np.float32))
    g = make_inputs(B, T, H, dk, dv, io="f32", seed=dk + dv, decay="mild", h0_std=0.05, lengths=lens)
    rng = np.random.default_rng(dk + 2 * dv)
    r = lambda *s: rng.standard_normal(s).astype(np.float32)  # noqa: E731
    x = {c: st(r(B, T, H, d)) for c, d in (("q", dk), ("k", dk), ("v", dv), ("gate", dv))}
    taps = {c: 0.5 * r(H * d, 4) for c, d in (("q", dk), ("k", dk), ("v", dv))}
    wt, dout, dhT = rng.uniform(0.5, 1.5, dv).astype(np.float32), st(r(B, T, H, dv)), r(N, H, dk, dv)
    dev = lambda a, t=torch.float32: torch.from_numpy(np.ascontiguousarray(a)).to("cuda", t)  # noqa: E731
    cu = None if lens is None else dev(g.cu_seqlens, torch.int32)
    kept = {c: gdn2.act_pack(dev(a, dt)) if packed else dev(a, dt) for c, a in x.items()}
    val = {c: _value(a) if packed else a.astype(np.float64) for c, a in x.items()}
    got = gdn2.token_path_bwd(kept["q"], kept["k"], kept["v"], dev(g.log_alpha), dev(g.b), dev(g.w), kept["gate"],
                              *(dev(taps[c]) for c in "qkv"), dev(wt), dev(dout, dt), g.scale, dev(g.h0), dev(dhT), cu)
    q, k, v = (st(a) for a in tp.prologue(val["q"], val["k"], val["v"], taps["q"], taps["k"], taps["v"], g.cu_seqlens))
    o, _ = oracle.recurrent(q, k, v, g.log_alpha, g.b, g.w, g.scale, h0=g.h0, cu_seqlens=g.cu_seqlens)
    o = st(o) if io == "bf16" else o
    e = tb.epilogue_bwd(o, val["gate"], wt, dout)
    c = ob.backward(q, k, v, g.log_alpha, g.b, g.w, g.scale, st(e["o"]), dhT=dhT, h0=g.h0, cu_seqlens=g.cu_seqlens)
    p = tb.prologue_bwd(val["q"], val["k"], val["v"], taps["q"], taps["k"], taps["v"], c["q"], c["k"], c["v"], g.cu_seqlens)
    ref = dict(p, gate=e["gate"], norm_weight=e["norm_weight"], log_alpha=c["log_alpha"], b=c["b"], w=c["w"], h0=c["h0"])
    assert set(got) == set(ref)
    off = {n: rel_l2(got[n].float().cpu().numpy(), ref[n]) for n in ref}
    assert max(off.values()) <= BAR[io], off
    for n in ("q_raw", "k_raw", "v_raw", "gate"):
        assert got[n].dtype == dt and got[n].shape == ref[n].shape
