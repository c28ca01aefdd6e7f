"""A status word that already holds an expired wait changes nothing about later calls, and keeps what it holds."""
import pytest

from test_gpu_diff_attention import _cu, _make, _run

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def jl():
    from encoder_decision_model_b200 import _lib
    from encoder_decision_model_b200.build import build
    build()
    return _lib


@pytest.mark.parametrize("qk,v", [("bf16", "f16"), ("bf16", "bf16"), ("f16", "f16"), ("f32", "f32")])
@pytest.mark.parametrize("held", [1, 0x7fffffff])
def test_bits_held_before(jl, qk, v, held):
    lens = [1500, 40, 700, 129] * 6
    x = _make(sum(lens), 3, 3, qk, v, 21)
    x = {n: (t.cuda() if torch.is_tensor(t) else [a.cuda() for a in t]) for n, t in x.items()}
    cu = torch.as_tensor(_cu(lens), dtype=torch.int32, device="cuda")
    want = _run(jl, x, cu)
    for _ in range(3):
        out, status = torch.full_like(want, 7.0), torch.full((1,), held, dtype=torch.int32, device="cuda")
        jl.jd_diff_attention(x["q"], x["k"], x["v"], out, cu, *x["lam"], 0.6, norm_gain=x["gain"], status=status,
                             stream=torch.cuda.current_stream())
        torch.cuda.synchronize()
        assert int(status) == held and torch.equal(out, want)
