"""Differential attention on batches of many rows: whatever the number of rows, every row's result is written and is its
own.  Against the float64 definition at the tolerances of test_gpu_diff_attention.py, whose outputs hold 7 before the
call, so that a token that is not written shows."""
import random

import numpy as np
import pytest

import gpu_helpers as gh
from test_gpu_diff_attention import TYPES, _check, _cu, _make, _run
from workloads import Row, variant_tensors, write_weights

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def jl():
    from encoder_decision_model_b200 import _lib
    from encoder_decision_model_b200.build import build
    build()
    return _lib


@pytest.mark.parametrize("qk,v", TYPES)
@pytest.mark.parametrize("n", [31, 32, 33, 63, 64, 94])
@pytest.mark.parametrize("heads,window", [(1, -1), (3, -1), (3, 16)])
def test_many_short_rows(jl, qk, v, n, heads, window):
    rng = random.Random(n)
    cu = _cu([rng.randint(1, 70) for _ in range(n)])
    x = _make(int(cu[-1]) + 2, heads, heads, qk, v, n)
    _check(_run(jl, x, cu, window=window), x, cu, window=window)


@pytest.mark.parametrize("qk,v", TYPES)
def test_one_token_each(jl, qk, v):
    cu = _cu([1] * 32)
    x = _make(32, 2, 1, qk, v, 12)
    _check(_run(jl, x, cu), x, cu)


# more work than CTAs: a CTA's search comes to the last rows from where its last item was
@pytest.mark.parametrize("qk,v", TYPES)
@pytest.mark.parametrize("n,length,heads", [(32, 300, 1), (63, 300, 1), (63, 130, 3), (125, 200, 2)])
def test_search_goes_on(jl, qk, v, n, length, heads):
    cu = _cu([length] * n)
    x = _make(int(cu[-1]), heads, 1, qk, v, n)
    _check(_run(jl, x, cu, window=40), x, cu, window=40)


# batches whose last tiles a search that stopped 32 rows before the end did not find
@pytest.mark.parametrize("seed", [250, 398, 718, 842, 993])
def test_ragged_batches(jl, seed):
    rng = random.Random(seed)
    n, top, heads, low = rng.randint(1, 400), rng.choice([1, 70, 128, 300, 1000]), rng.randint(1, 6), rng.choice([0, 1, 64])
    cu = _cu([rng.randint(min(low, top), top) for _ in range(n)])
    x = _make(int(cu[-1]), heads, 1, "bf16", "f16", seed)
    _check(_run(jl, x, cu, window=8), x, cu, window=8)


def test_model_of_32_short_rows(jl, tmp_path):
    """The model's differential layers on 32 rows: the same bits as in smaller batches, also behind another batch."""
    path = tmp_path / "diff.jdw"
    write_weights(path, extra=variant_tensors(5, diff=(0, 1, 2, 12, 21)))
    rng = np.random.Generator(np.random.PCG64(8))
    ids = lambda n: rng.integers(10, 256000, n).astype(np.int32)  # noqa: E731
    rows = [Row(state=ids(rng.integers(8, 30)), question=ids(8), options=[ids(3) for _ in range(2 + i % 3)], qtype=0)
            for i in range(32)]
    opts = dict(max_length=8192, head_budget=512, strict=True)
    m = jl.Model(path, 4096, 64, 256)
    _, other = gh.device_run(m, rows[::-1], opts)
    hb, got = gh.device_run(m, rows, opts)
    small = []
    for at in range(0, 32, 8):
        small.append(gh.device_run(m, rows[at:at + 8], opts)[1]["logits"])
    m.close()
    np.testing.assert_array_equal(got["logits"], np.concatenate(small))
    ends = np.cumsum([len(r.options) for r in rows[::-1]])[:-1]
    np.testing.assert_array_equal(np.concatenate(np.split(other["logits"], ends)[::-1]), got["logits"])
