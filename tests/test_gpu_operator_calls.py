"""Calls of the encoder operators that the documentation allows and that are easily got wrong: elements more
than 2^31 from a tensor's start, a process whose first call is captured, and threads that call at once.

Where an element lies does not enter its arithmetic, nor does what else runs, so the results are those of the
plain call bit for bit.
"""
import os
import subprocess
import sys
import threading

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..")
FAR = (1 << 30) + 64  # elements between tokens: the third starts past 2^31


@pytest.fixture(scope="module")
def jl():
    from encoder_decision_model_b200 import _lib
    from encoder_decision_model_b200.build import build
    build()
    return _lib


def _far(x):
    """x [3, heads, n] with FAR elements between its tokens."""
    t, h, n = x.shape
    assert t == 3
    base = torch.empty(2 * FAR + h * n, dtype=x.dtype, device="cuda")
    y = base.as_strided((t, h, n), (FAR, n, 1))
    y.copy_(x)
    return y


@pytest.mark.parametrize("head_dim,dims", [(64, 64), (10, 6)])
@pytest.mark.parametrize("norm", [False, True])
def test_rotary_far_offsets(jl, head_dim, dims, norm):
    g = torch.Generator().manual_seed(head_dim + norm)
    q = torch.randn(3, 2, head_dim, generator=g).bfloat16().cuda()
    cu = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    rc = jl.rotary_config(dims, 1e4)
    call = jl.jd_qk_norm_rotary if norm else jl.jd_rotary
    want, far = torch.zeros_like(q), _far(q)
    out = _far(torch.zeros_like(q))
    st = torch.cuda.current_stream()
    call(q, None, want, None, rc, cu_seqlens=cu, stream=st)
    call(far, None, out, None, rc, cu_seqlens=cu, stream=st)
    call(far, None, far, None, rc, cu_seqlens=cu, stream=st)
    torch.cuda.synchronize()
    assert not torch.equal(want, q) and torch.equal(out, want) and torch.equal(far, want)


@pytest.mark.parametrize("qk,v", [("bfloat16", "float16"), ("bfloat16", "bfloat16"), ("float32", "float32")])
def test_diff_attention_far_offsets(jl, qk, v):
    g = torch.Generator().manual_seed(3)
    q, k = (torch.randn(3, 4, 64, generator=g).to(getattr(torch, qk)).cuda() for _ in range(2))
    val = torch.randn(3, 2, 128, generator=g).to(getattr(torch, v)).cuda()
    lam = [(0.1 * torch.randn(64, generator=g)).cuda() for _ in range(4)]
    cu = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    want, out = torch.zeros(3, 2, 128, dtype=q.dtype, device="cuda"), _far(torch.zeros(3, 2, 128, dtype=q.dtype, device="cuda"))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    st = torch.cuda.current_stream()
    jl.jd_diff_attention(q, k, val, want, cu, *lam, 0.6, status=status, stream=st)
    jl.jd_diff_attention(_far(q), _far(k), _far(val), out, cu, *lam, 0.6, status=status, stream=st)
    torch.cuda.synchronize()
    assert int(status) == 0 and want.abs().sum() > 0 and torch.equal(out, want)


FIRST = """
import sys, torch
sys.path.insert(0, sys.argv[1])
from encoder_decision_model_b200 import _lib as jl
g = torch.Generator().manual_seed(1)
q, k = (torch.randn(150, 6, 64, generator=g).bfloat16().cuda() for _ in range(2))
v = torch.randn(150, 3, 128, generator=g).half().cuda()
lam = [(0.1 * torch.randn(64, generator=g)).cuda() for _ in range(4)]
cu = torch.tensor([0, 37, 150], dtype=torch.int32, device="cuda")
rc = jl.rotary_config(64, 1e4)
def run(outs, st):
    a, b, o = outs
    jl.jd_qk_norm_rotary(q, k, a, b, rc, cu_seqlens=cu, stream=st)
    jl.jd_rotary(a, b, a, b, rc, cu_seqlens=cu, stream=st)
    jl.jd_diff_attention(a, b, v, o, cu, *lam, 0.6, stream=st)
new = lambda: [torch.zeros_like(q), torch.zeros_like(k), torch.zeros(150, 3, 128, dtype=q.dtype, device="cuda")]
got, want, graph = new(), new(), torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(graph):
    run(got, torch.cuda.current_stream())
graph.replay()
torch.cuda.synchronize()
run(want, torch.cuda.current_stream())
torch.cuda.synchronize()
assert want[2].abs().sum() > 0 and all(torch.equal(a, b) for a, b in zip(got, want))
print("same")
"""


def test_first_call_of_a_process_is_captured(jl):
    r = subprocess.run([sys.executable, "-c", FIRST, ROOT], capture_output=True, text=True, timeout=240)
    assert r.returncode == 0 and r.stdout.strip() == "same", r.stderr[-2000:]


def test_threads_at_once(jl):
    g = torch.Generator().manual_seed(2)
    q, k = (torch.randn(300, 6, 64, generator=g).bfloat16().cuda() for _ in range(2))
    v = torch.randn(300, 3, 128, generator=g).half().cuda()
    lam = [(0.1 * torch.randn(64, generator=g)).cuda() for _ in range(4)]
    cu = torch.tensor([0, 129, 300], dtype=torch.int32, device="cuda")
    rc = jl.rotary_config(64, 1e4)
    n = 4
    a, b = [[torch.zeros_like(q) for _ in range(n + 1)] for _ in range(2)]
    o = [torch.zeros(300, 3, 128, dtype=q.dtype, device="cuda") for _ in range(n + 1)]
    streams, faults = [torch.cuda.Stream() for _ in range(n + 1)], []
    torch.cuda.synchronize()

    def work(i, times):
        try:
            for _ in range(times):
                jl.jd_rotary(q, k, a[i], b[i], rc, cu_seqlens=cu, stream=streams[i])
                jl.jd_diff_attention(a[i], b[i], v, o[i], cu, *lam, 0.6, stream=streams[i])
                with pytest.raises(jl.JDError, match="kv_heads|heads"):  # each thread has its own message
                    jl.jd_diff_attention(a[i], b[i], v[:, :2], o[i], cu, *lam, 0.6, stream=streams[i])
        except BaseException as e:  # noqa: BLE001
            faults.append(e)

    work(n, 1)
    threads = [threading.Thread(target=work, args=(i, 25)) for i in range(n)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not faults, faults
    assert o[n].abs().sum() > 0 and all(torch.equal(x, o[n]) for x in o[:n])
