"""The rounding of the probabilities in the 16-bit differential attention, where it would show most: two nearly equal
maps and lambda near 1, so that the difference is small beside the products it is taken of and the norm makes
what they lost large.

Tolerance, element by element, as derived in test_gpu_diff_attention.py, with the probabilities a pair of 16-bit numbers
in every type: e_p = 2^-22 in FP16 (two halves of 2^-11) and 2^-25 absolute on each key, 2^-16 in BF16 (two of 2^-8).  A
single FP16 number (2^-11) does not stay within it.
"""
import numpy as np
import pytest

import operator_refs as ref
from test_gpu_diff_attention import _cu, _run

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = [("bfloat16", "float16"), ("bfloat16", "bfloat16"), ("float16", "float16"), ("float16", "bfloat16")]


@pytest.fixture(scope="module")
def jl():
    from encoder_decision_model_b200 import _lib
    from encoder_decision_model_b200.build import build
    build()
    return _lib


@pytest.mark.parametrize("qk,v", TYPES)
@pytest.mark.parametrize("lambda_init", [0.6, 0.8, 0.95])
@pytest.mark.parametrize("lens,window", [([2, 3, 5, 8, 1, 2, 17], -1), ([64, 200, 33], -1), ([700], -1), ([300], 20)])
def test_alike_maps(jl, qk, v, lambda_init, lens, window):
    cu, heads = _cu(lens), 2
    T = int(cu[-1])
    g = torch.Generator().manual_seed(T + int(100 * lambda_init))
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731

    def maps():
        x = 1.2 * r(T, heads, 1, 64)
        return torch.cat([x, x + 0.03 * r(T, heads, 1, 64)], 2).reshape(T, 2 * heads, 64).to(getattr(torch, qk))

    x = dict(q=maps(), k=maps(), v=r(T, heads, 128).to(getattr(torch, v)), lam=[torch.zeros(64)] * 4,
             gain=1 + 0.1 * r(128))
    n64 = lambda t: t.double().cpu().numpy()  # noqa: E731
    q, k, gain = n64(x["q"]), n64(x["k"]), n64(x["gain"])
    # the four dot products are 0: lambda is lambda_init, in FP32
    lam = float(np.float32(lambda_init))
    want, (_, rms, A) = ref.diff_attention(q, k, n64(x["v"]), cu, lam, lam, gain, 1e-5, window)
    got = n64(_run(jl, x, cu, lambda_init=lambda_init, window=window))
    n = max(lens) if window < 0 else 2 * window + 1
    e_s = 64 * 2.0 ** -24 * np.abs(q).max() * np.abs(k).sum(-1).max() * 0.125 / 64 + 2.0 ** -18 + 2.0 ** -22
    e_p = 2.0 ** -16 if v == "bfloat16" else 2.0 ** -22
    dD = (2 * e_s + e_p + (n + 4) * 2.0 ** -24) * A
    if v == "float16":
        dD = dD + n * 2.0 ** -25 * (1 + lam) * np.abs(n64(x["v"])).max()
    factor = np.abs((1 - lam) * gain)
    tol = factor * dD / rms + np.abs(want) * np.sqrt((dD * dD).mean(-1, keepdims=True)) / rms
    tol = tol + 8 * 2.0 ** -24 * np.abs(want) + torch.finfo(x["q"].dtype).eps / 2 * np.abs(want)
    tol = tol + 2.0 ** -25 * (qk == "float16")
    worst = float((np.abs(got - want) / tol).max())
    assert worst <= 1.0, worst
