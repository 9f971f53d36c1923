"""The gated scan's bounded waits, made to run out on purpose (no fault, no hang): in tests/csrc/scan_probe.cu half of a
cluster's blocks never receive a map.  The launch completes after one limit, not one a step; the status word reads
GDN2_ERR_DEVICE_TIMEOUT; the context stays usable.  With every map sent, a limit of one second changes no bit."""
import ctypes
import os
import subprocess
import time

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = os.path.join(ROOT, "tests", "csrc", "scan_probe.cu")
LIB = os.path.join(ROOT, "tests", "csrc", "libscanprobe.so")
CSRC = os.path.join(ROOT, "gated_delta_rule_129_b200", "csrc")

GDN2_ERR_DEVICE_TIMEOUT = 8
LIMIT_MS = 20


def build_probe():
    deps = [SRC] + [os.path.join(CSRC, f) for f in ("gated_scan.cuh", "common.cuh", "tc.cuh")]
    if os.path.exists(LIB) and all(os.path.getmtime(d) <= os.path.getmtime(LIB) for d in deps):
        return LIB
    tmp = LIB + f".tmp{os.getpid()}"
    subprocess.run(["nvcc", "-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-std=c++17", "--expt-relaxed-constexpr",
                    "-shared", "-Xcompiler", "-fPIC", "-I", CSRC, SRC, "-o", tmp], check=True)
    os.replace(tmp, LIB)
    return LIB


def test_probe_library_compiles():
    """Cross-compiles for sm_100a without a GPU."""
    assert os.path.exists(build_probe())


@pytest.fixture(scope="module")
def probe(cuda_device):
    lib = ctypes.CDLL(build_probe())
    vp, i = ctypes.c_void_p, ctypes.c_int
    lib.scan_probe.argtypes = [i, i, i, i, ctypes.c_ulonglong, i, i] + [vp] * 13
    return lib


@pytest.fixture(scope="module")
def gdn2(cuda_device):
    import gated_delta_rule_129_b200 as mod
    mod.load_library()
    return mod


def _inputs(T, D, io):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(T + D)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    shape = (1, T, D // 64, 64)
    return n(*shape).to(io), -n(*shape).abs(), n(*shape), n(*shape).to(io)


def _run(probe, gdn2, backward, lone, cl, limit_ns, v, la, w, dO, states=None):
    """(outputs, status) of a probe's launch; without `states` of the forward's outputs."""
    import torch
    T, D = v.shape[1], v.shape[2] * 64
    P = lambda t: None if t is None else ctypes.c_void_p(t.data_ptr())  # noqa: E731
    f32 = lambda *s: torch.zeros(s, device="cuda")  # noqa: E731
    out, hT = torch.zeros_like(v), f32(1, D // 64, 64)
    st = gdn2.gated_scan_chunk_states(v).zero_() if states is None else states
    grads = [torch.zeros_like(la) for _ in range(3)] + [torch.zeros_like(hT)]
    status = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    rc = probe.scan_probe(int(backward), int(v.dtype == torch.float32), int(lone), cl, limit_ns, T, D, P(v), P(la), P(w), P(dO),
                          P(out), P(hT), P(st), *map(P, grads), P(status),
                          ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert rc == 0
    torch.cuda.synchronize()
    return ((grads if backward else [out, hT, st]), int(status))


@pytest.mark.gpu
@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_waits_run_out_once_and_not_once_a_step(probe, gdn2, io, backward):
    import torch
    dt = torch.float32 if io == "f32" else torch.bfloat16
    cl = 2 if io == "f32" and not backward else 4
    x = _inputs(64 * 1000, 256, dt)                       # 250 or 500 steps
    states = gdn2.gated_scan_chunk_states(x[0])
    gdn2.gated_scan_fwd(*x[:3], chunk_states=states)
    _run(probe, gdn2, backward, False, cl, 10 ** 9, *x, states=states if backward else None)   # loads the kernel
    t0 = time.perf_counter()
    _, status = _run(probe, gdn2, backward, True, cl, LIMIT_MS * 10 ** 6, *x, states=states if backward else None)
    taken = time.perf_counter() - t0
    assert status == GDN2_ERR_DEVICE_TIMEOUT
    assert LIMIT_MS / 1e3 <= taken < 1.0                  # 250 limits would be five seconds
    # the context is usable, and the next call right
    o, _ = gdn2.gated_scan_fwd(*x[:3])
    o2, _ = gdn2.gated_scan_fwd(*x[:3])
    assert torch.equal(o, o2) and bool(torch.isfinite(o).all())


@pytest.mark.gpu
@pytest.mark.parametrize("cl", [2, 4, 8])
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_with_every_map_the_walk_is_the_librarys(probe, gdn2, io, cl):
    import torch
    dt = torch.float32 if io == "f32" else torch.bfloat16
    x = _inputs(64 * 70 + 5, 128, dt)
    states = gdn2.gated_scan_chunk_states(x[0])
    o, hT = gdn2.gated_scan_fwd(*x[:3], chunk_states=states)
    if io == "bf16" or cl <= 4:
        got, status = _run(probe, gdn2, False, False, cl, 10 ** 9, *x)
        assert status == 0 and torch.equal(got[0], o) and torch.equal(got[1], hT) and torch.equal(got[2], states)
    g = gdn2.gated_scan_bwd(*x, chunk_states=states)
    got, status = _run(probe, gdn2, True, False, cl, 10 ** 9, *x, states=states)
    assert status == 0
    for a, n in zip(got, ("v", "log_alpha", "w", "h0")):
        assert torch.equal(a, g[n]), n


@pytest.mark.gpu
def test_status_of_a_backward_call_that_computes_the_states_again(gdn2):
    """Its workspace's first word: 0, or the malformed cu_seqlens that both launches see; captured and replayed too."""
    import torch
    v, la, w, dO = _inputs(300, 128, torch.bfloat16)
    ws = torch.empty(1 << 16, dtype=torch.uint8, device="cuda")
    word = ws[:4].view(torch.int32)
    for cu, want in (([0, 100, 300], 0), ([0, 100, 299], 5), ([0, 200, 100, 300], 5), (None, 0)):
        t = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
        gdn2.gated_scan_bwd(v, la, w, dO, cu_seqlens=t, workspace=ws)
        assert int(word) == want, cu
    ref = gdn2.gated_scan_bwd(v, la, w, dO)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g = gdn2.gated_scan_bwd(v, la, w, dO, workspace=ws)
    word.fill_(99)
    graph.replay()
    torch.cuda.synchronize()
    assert int(word) == 0 and all(torch.equal(g[k], ref[k]) for k in ref)
