"""The oracle's encoder variants (head norms, rotations, differential attention) pinned on the CPU: closed
forms and special cases, and the definitions of tests/operator_refs.py, written apart."""
import math

import numpy as np
import pytest

import operator_refs as ref
from oracle import model as om
from workloads import variant_tensors, weight_specs

RNG = np.random.default_rng(3)


def test_plain_record_is_the_plain_rotation():
    x = RNG.standard_normal((40, 6, 64))
    np.testing.assert_allclose(om.rope_as(x, [0, 64, 160000.0, 0, 1, 0, 0, 0]), om.rope(x, 160000.0), atol=1e-12)


def test_interleaved_pairs_and_pass_through():
    x = RNG.standard_normal((5, 1, 8))
    y = om.rope_as(x, [1, 4, 100.0, 0, 1, 0, 0, 0])
    np.testing.assert_array_equal(y[..., 4:], x[..., 4:])
    a = 3 * 100.0 ** (-0.5)  # position 3, second pair
    np.testing.assert_allclose(y[3, 0, 2], x[3, 0, 2] * math.cos(a) - x[3, 0, 3] * math.sin(a))
    np.testing.assert_allclose(y[3, 0, 3], x[3, 0, 3] * math.cos(a) + x[3, 0, 2] * math.sin(a))


def test_linear_scaling_is_position_over_factor():
    x = RNG.standard_normal((9, 2, 64))
    y = om.rope_as(x, [0, 64, 10000.0, 1, 4.0, 0, 0, 0])
    np.testing.assert_allclose(y[8], om.rope(x[[8] * 3], 10000.0)[2], atol=1e-12)  # position 8 / 4 = 2


def test_ntk_keeps_the_fastest_pair_and_stretches_the_slowest():
    _, w, _ = om.rotation([0, 64, 10000.0, 2, 4.0, 0, 0, 0])
    _, plain, _ = om.rotation([0, 64, 10000.0, 0, 1.0, 0, 0, 0])
    assert w[0] == plain[0] == 1.0
    np.testing.assert_allclose(w[-1], plain[-1] / 4.0, rtol=1e-12)


def test_yarn_ends():
    _, w, amp = om.rotation([0, 64, 10000.0, 3, 8.0, 4096, 32.0, 1.0])
    _, plain, _ = om.rotation([0, 64, 10000.0, 0, 1.0, 0, 0, 0])
    np.testing.assert_allclose(w[:5], plain[:5])         # turn more than 32 times over 4096: kept
    np.testing.assert_allclose(w[-5:], plain[-5:] / 8)   # less than once: stretched
    assert amp == pytest.approx(0.1 * math.log(8) + 1)


@pytest.mark.parametrize("rec", [[0, 64, 1e4, 0, 1, 0, 0, 0], [1, 32, 1.6e5, 2, 2.0, 0, 0, 0], [0, 20, 1e4, 1, 3.0, 0, 0, 0],
                                 [1, 50, 1e4, 3, 7.5, 1024, 32.0, 1.0]])
def test_rotation_against_the_operators_definition(rec):
    names = {0: "none", 1: "linear", 2: "ntk", 3: "yarn"}
    x = RNG.standard_normal((300, 3, 64))
    kw = dict(original_length=rec[5], beta_fast=rec[6], beta_slow=rec[7]) if rec[3] == 3 else {}
    w, amp = ref.frequencies(rec[1], rec[2], names[rec[3]], rec[4], **kw)
    want = ref.rotate(x, np.arange(300), w, amp, "interleaved" if rec[0] else "half")
    np.testing.assert_allclose(om.rope_as(x, rec), want, atol=1e-10)


def _lambdas(l):
    t = variant_tensors(1, diff=[l])
    return {k: v.astype(np.float64) for k, v in t.items()}


@pytest.mark.parametrize("window", [None, 5])
def test_differential_attention_against_the_operators_definition(window):
    q, k, v = (RNG.standard_normal((37, 6, 64)) for _ in range(3))
    W, l = _lambdas(4), 4
    got = om.diff_attention(q, k, v, W, "enc.4.", l, window, 1e-5)
    start = 0.8 - 0.6 * math.exp(-0.3 * l)
    lam = ref.diff_lambda(*[W[f"enc.4.lambda_{n}"] for n in ("q1", "k1", "q2", "k2")], start)
    want, _ = ref.diff_attention(q, k, v.reshape(37, 3, 128), [0, 37], lam, start, W["enc.4.diff_norm.g"], 1e-5,
                                 -1 if window is None else window)
    np.testing.assert_allclose(got, want, atol=1e-12)


def test_equal_maps_cancel_up_to_lambda():
    """With equal queries and keys in both maps the difference is (1 - lambda) of one map's output, which the norm
    takes away: the result does not depend on lambda."""
    q1, k1 = RNG.standard_normal((20, 3, 64)), RNG.standard_normal((20, 3, 64))
    q, k = np.repeat(q1, 2, axis=1), np.repeat(k1, 2, axis=1)
    v = RNG.standard_normal((20, 6, 64))
    W = _lambdas(0)
    got = om.diff_attention(q, k, v, W, "enc.0.", 0, None, 0.0)
    one = om.attention(q1, k1, v.reshape(20, 3, 128)[..., :64], None)
    d = got[..., :64] / W["enc.0.diff_norm.g"][:64]
    ratio = d / one
    np.testing.assert_allclose(ratio, np.broadcast_to(ratio[..., :1], ratio.shape), rtol=1e-9)


def test_variant_tensors_have_names_of_their_own():
    plain = {n for n, _, _ in weight_specs()}
    t = variant_tensors(0, norms=range(22), diff=range(22), rotary=[[0] * 8] * 2)
    assert len(t) == 22 * 2 + 22 * 5 + 1 and not plain & set(t)
    assert all(v.dtype == np.float32 for v in t.values())
