"""The training calls' `stream` argument, with the other arguments by keyword and in any order: the results are those of
the call on the current stream."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gdn2(cuda_device):
    import gated_delta_rule_129_b200 as mod
    mod.load_library()
    return mod


def _leaves(r):
    if isinstance(r, dict):
        return list(r.values())
    return list(r) if isinstance(r, tuple) else [r]


def test_keyword_calls_on_a_stream(gdn2):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    shape = (1, 200, 2, 64)
    x, la, w, dO, wt = n(*shape), -n(*shape).abs(), n(*shape), n(*shape), n(64)
    t = [0.5 * n(128, 4) for _ in range(3)]
    p, state = gdn2.act_pack(x), n(3, 2, 64)
    cu = torch.tensor([0, 70, 200], dtype=torch.int32, device="cuda")
    gates = dict(log_alpha=la, b=torch.sigmoid(n(*shape)), w=torch.sigmoid(w))
    calls = [
        lambda **k: gdn2.act_pack(out=None, x=x, **k),
        lambda **k: gdn2.act_unpack(dtype=torch.float32, packed=p, **k),
        lambda **k: gdn2.act_unpack([p.codes, p.exps], **k),
        lambda **k: gdn2.token_prologue_bwd(cu_seqlens=cu, dtype=torch.float32, q_raw=p, k_raw=p, v_raw=p, conv_q=t[0],
                                            conv_k=t[1], conv_v=t[2], dq=dO, dk=w, dv=la, **k),
        lambda **k: gdn2.token_epilogue_bwd(norm_weight=wt, dout=dO, gate=p, o=x, **k),
        lambda **k: gdn2.gated_scan_fwd(h0=None, cu_seqlens=cu, v=x, log_alpha=la, w=w, **k),
        lambda **k: gdn2.gated_scan_bwd(cu_seqlens=None, dO=dO, v=x, log_alpha=la, w=w, **k),
        lambda **k: gdn2.gated_scan_step(v=x[0, :3].contiguous(), log_alpha=la[0, :3].contiguous(), w=w[0, :3].contiguous(),
                                         state=state.clone(), **k),
        lambda **k: gdn2.token_path_bwd(scale=None, h0=None, cu_seqlens=cu, q_raw=x, k_raw=p, v_raw=dO, gate=p, conv_q=t[0],
                                        conv_k=t[1], conv_v=t[2], norm_weight=wt, dout=dO, **gates, **k),
    ]
    for i, call in enumerate(calls):
        want = _leaves(call())
        torch.cuda.synchronize()
        stream = torch.cuda.Stream()
        got = _leaves(call(stream=stream))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            # chunk_bwd's dlog_alpha adds in no fixed order: the whole path's gradients to fp32's bar
            same = torch.equal(a, b) if i < len(calls) - 1 else bool((a - b).norm() <= 1e-4 * b.norm())
            assert same, i
