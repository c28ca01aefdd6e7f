"""Arguments that the calls' 32-bit fields do not hold: refused with the library's own error, not wrapped around into a
value that is allowed (no device needed)."""
import pytest

from encoder_decision_model_b200 import _lib as jl
from encoder_decision_model_b200.build import build

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def built():
    build()


def _refused(call):
    with pytest.raises(jl.JDError) as e:
        call()
    assert e.value.code == jl.JD_ERR_INVALID_ARG


@pytest.mark.parametrize("change", [dict(dims=(1 << 32) + 64), dict(dims=1 << 31), dict(original_length=(1 << 32) + 1),
                                    dict(original_length=-(1 << 31) - 1)])
def test_rotary_config(change):
    _refused(lambda: jl.rotary_config(**{**dict(dims=64, theta=1e4), **change}))


@pytest.mark.parametrize("change", [dict(window=1 << 31), dict(window=-(1 << 40)), dict(window=1.5), dict(lambda_init=None)])
def test_diff_attention(change):
    x = [torch.zeros(10, n, d, dtype=torch.bfloat16) for n, d in ((6, 64), (6, 64), (3, 128), (3, 128))]
    cu = torch.tensor([0, 10], dtype=torch.int32)
    kw = {**dict(lambda_init=0.6), **change}
    _refused(lambda: jl.jd_diff_attention(*x, cu, *[torch.zeros(64)] * 4, **kw))


def test_more_tokens_than_a_field_holds():
    q = torch.zeros(1, 1, 64).expand((1 << 31) + 8, 1, 64)
    cu = torch.tensor([0, 10], dtype=torch.int32)
    rc = jl.rotary_config(64, 1e4)
    _refused(lambda: jl.jd_rotary(q, None, q, None, rc, cu_seqlens=cu))
    _refused(lambda: jl.jd_qk_norm_rotary(q, None, q, None, rc, cu_seqlens=cu))
    v, o = (torch.zeros(1, 1, 128).expand((1 << 31) + 8, 1, 128) for _ in range(2))
    q2 = torch.zeros(1, 1, 64).expand((1 << 31) + 8, 2, 64)
    _refused(lambda: jl.jd_diff_attention(q2, q2, v, o, cu, *[torch.zeros(64)] * 4, 0.6))
