"""Differential attention on the GPU against the float64 definition.

Tolerance, element by element.  A probability is off, relatively, by
  - its score: 64 products summed in FP32, 64 * 2^-24 sum |q k| scale, and the exponent's argument, rounded at
    |x| <= 64 (2^-18 ln 2), and 2^-22 of the exponential; the same again in the sum that divides it: with the
    unit-scale inputs here sum |q k| scale <= 64 * 4.5^2 / 8 for every key that matters, so below 2^-11.4 in
    the worst case for FP32 operands and no more for 16-bit ones (their products are exact); measured over
    the inputs themselves rather than bounded, e_s below;
  - its rounding for the second product, e_p: 2^-11 in FP16 beside a BF16 result, 2^-16 as a pair of BF16,
    2^-21 as a pair of FP16, nothing in FP32; FP16 further loses up to 2^-25 absolute on each of n keys, of
    a sum of at least 1.
With A = sum p0 |v| + |lambda| sum p1 |v|, D is off by at most dD = (2 e_s + e_p) A + n 2^-25 (1 + |lambda|) max |v|
plus FP32 sums over n keys, n * 2^-24 A.  The norm divides by rms(D), itself off by at most rms(dD), and the
result is rounded once: eps / 2.
"""
import numpy as np
import pytest

import operator_refs as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"f32": "float32", "f16": "float16", "bf16": "bfloat16"}
TYPES = [("bf16", "bf16"), ("bf16", "f16"), ("f16", "f16"), ("f16", "bf16"), ("f32", "f32")]


@pytest.fixture(scope="module")
def jl():
    from encoder_decision_model_b200 import _lib
    from encoder_decision_model_b200.build import build
    build()
    return _lib


def _make(T, heads, kv, qk, v, seed, std=1.2):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s, f=1.0: torch.randn(*s, generator=g) * f  # noqa: E731
    d, dv = getattr(torch, DT[qk]), getattr(torch, DT[v])
    return dict(q=r(T, 2 * heads, 64, f=std).to(d), k=r(T, 2 * kv, 64, f=std).to(d), v=r(T, kv, 128).to(dv),
                lam=[r(64, f=0.1) for _ in range(4)], gain=1 + 0.1 * r(128))


def _run(jl, x, cu, lambda_init=0.6, norm=True, window=-1, out=None, stream=None, status=None, scale=0.0, eps=1e-5):
    c = {n: (x[n] if x[n].is_cuda else x[n].cuda()) for n in ("q", "k", "v")}
    T, heads = c["q"].shape[0], c["q"].shape[1] // 2
    if out is None:
        out = torch.full((T, heads, 128), 7.0, dtype=c["q"].dtype, device="cuda")
    cud = cu if torch.is_tensor(cu) else torch.as_tensor(np.asarray(cu), dtype=torch.int32, device="cuda")
    lam = [a.cuda() for a in x["lam"]]
    st = torch.zeros(1, dtype=torch.int32, device="cuda") if status is None else status
    jl.jd_diff_attention(c["q"], c["k"], c["v"], out, cud, *lam, lambda_init, norm_gain=x["gain"].cuda() if norm else None,
                         norm_eps=eps, window=window, scale=scale, status=st,
                         stream=stream or torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert int(st) == 0
    return out


def _check(got, x, cu, lambda_init=0.6, norm=True, window=-1, scale=0.125, eps=1e-5):
    n64 = lambda t: t.double().cpu().numpy()  # noqa: E731
    q, k, v = n64(x["q"]), n64(x["k"]), n64(x["v"])
    lam = ref.diff_lambda(*[n64(a) for a in x["lam"]], lambda_init)
    gain = n64(x["gain"]) if norm else None
    want, (D, rms, A) = ref.diff_attention(q, k, v, cu, lam, lambda_init, gain, eps, window, scale)
    n = max(b - a for a, b in zip(cu[:-1], cu[1:]))
    qk, vt = x["q"].dtype, x["v"].dtype
    e_s = 64 * 2.0 ** -24 * np.abs(q).max() * np.abs(k).sum(-1).max() * scale / 64 + 2.0 ** -18 + 2.0 ** -22
    if vt == torch.float32:
        e_p = 0.0
    elif vt == torch.bfloat16:
        e_p = 2.0 ** -16
    else:
        e_p = 2.0 ** -11 if qk == torch.bfloat16 else 2.0 ** -21
    dD = (2 * e_s + e_p + n * 2.0 ** -24) * A
    if vt == torch.float16:
        dD = dD + n * 2.0 ** -25 * (1 + abs(lam)) * np.abs(v).max()
    dD = dD + 4 * 2.0 ** -24 * A  # lambda itself and the difference
    tol = dD
    if norm:
        g = np.abs((1 - lambda_init) * gain)
        tol = g * dD / rms + np.abs(want) * np.sqrt((dD * dD).mean(-1, keepdims=True)) / rms + 8 * 2.0 ** -24 * np.abs(want)
    tol = tol + torch.finfo(qk).eps / 2 * np.abs(want) + 2.0 ** -25 * (qk == torch.float16)
    on = np.zeros(len(q), bool)
    for a, b in zip(cu[:-1], cu[1:]):
        on[a:b] = True
    err = np.abs(n64(got) - want)[on]
    worst = float((err / tol[on]).max()) if err.size else 0.0
    assert worst <= 1.0, worst
    assert (got.cpu()[~torch.from_numpy(on)] == 7).all()


ROWS = {
    "one token": [1],
    "short": [1, 2, 3, 15, 16, 17],
    "empty rows": [0, 5, 0, 0, 130, 0],
    "tile edges": [127, 128, 129, 255, 256, 257],
    "ragged": [300, 64, 513, 1, 77],
}


def _cu(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)


@pytest.mark.parametrize("qk,v", TYPES)
@pytest.mark.parametrize("rows", list(ROWS))
@pytest.mark.parametrize("window", [-1, 0, 1, 64, 200])
def test_rows_types_windows(jl, qk, v, rows, window):
    cu = _cu(ROWS[rows])
    x = _make(int(cu[-1]) + 3, 3, 3, qk, v, 1)  # three tokens behind the last row
    _check(_run(jl, x, cu, window=window), x, cu, window=window)


@pytest.mark.parametrize("qk,v", TYPES)
@pytest.mark.parametrize("heads,kv", [(1, 1), (4, 2), (6, 1), (5, 5)])
@pytest.mark.parametrize("norm", [True, False])
def test_heads_and_norm(jl, qk, v, heads, kv, norm):
    cu = _cu([200, 31])
    x = _make(231, heads, kv, qk, v, 2)
    _check(_run(jl, x, cu, norm=norm, lambda_init=0.2), x, cu, norm=norm, lambda_init=0.2)


@pytest.mark.parametrize("qk,v", TYPES)
def test_many_rows(jl, qk, v):
    cu = _cu([(53 * i) % 97 for i in range(1100)])  # over 1024 rows: the search for a row takes three steps
    x = _make(int(cu[-1]), 1, 1, qk, v, 3)
    _check(_run(jl, x, cu), x, cu)


@pytest.mark.parametrize("qk,v", TYPES)
def test_long_row(jl, qk, v):
    cu = _cu([2100, 900])
    x = _make(3000, 2, 1, qk, v, 4)
    _check(_run(jl, x, cu), x, cu)
    _check(_run(jl, x, cu, window=700), x, cu, window=700)


@pytest.mark.parametrize("qk,v", TYPES)
def test_steep_scores(jl, qk, v):
    """Scores in the hundreds, growing along the row: the running maximum moves in every tile."""
    T = 640
    x = _make(T, 1, 1, qk, v, 5)
    x["k"] = (x["k"].float() * torch.linspace(0.2, 3.0, T)[:, None, None]).to(x["k"].dtype)
    x["q"] = (x["q"].float() * 1.5).to(x["q"].dtype)
    _check(_run(jl, x, _cu([T])), x, _cu([T]))


@pytest.mark.parametrize("qk,v", TYPES)
@pytest.mark.parametrize("window", [-1, 20])
def test_other_rows_do_not_enter(jl, qk, v, window):
    """NaN, infinities and the type's extremes in a row's neighbours and behind the last row leave it alone."""
    lens = [40, 100, 37, 130, 9]
    cu = _cu(lens)
    x = _make(int(cu[-1]) + 200, 2, 2, qk, v, 6)
    clean = _run(jl, x, cu, window=window)
    bad = {n: (t.clone() if torch.is_tensor(t) else t) for n, t in x.items()}
    for n in ("q", "k", "v"):
        t, big = bad[n], torch.finfo(bad[n].dtype).max
        for r, val in ((0, float("nan")), (2, float("inf")), (4, -big)):
            t[cu[r]:cu[r + 1]] = val
        t[cu[-1]:] = float("nan")
    got = _run(jl, bad, cu, window=window)
    for r in (1, 3):
        assert torch.equal(got[cu[r]:cu[r + 1]], clean[cu[r]:cu[r + 1]])
    assert (got[cu[-1]:] == 7).all()


@pytest.mark.parametrize("qk,v", [("bf16", "f16"), ("f32", "f32")])
def test_layouts(jl, qk, v):
    cu = _cu([150, 61])
    T = 211
    x = _make(T, 3, 3, qk, v, 7)
    want = _run(jl, x, cu)
    y = dict(x)
    # heads outermost; q and k side by side in one row; values of a wider buffer; an output of another order
    y["q"] = x["q"].permute(1, 0, 2).contiguous().cuda().permute(1, 0, 2)
    both = torch.cat([x["k"], x["q"]], 1).cuda()
    y["k"] = both[:, :6]
    wide = torch.zeros(T, 9, 128, dtype=x["v"].dtype, device="cuda")
    wide[:, 2:8:2] = x["v"].cuda()
    y["v"] = wide[:, 2:8:2]
    out = torch.full((3, T, 128), 7.0, dtype=x["q"].dtype, device="cuda").permute(1, 0, 2)
    assert torch.equal(_run(jl, y, cu, out=out), want)


def test_scale_and_large_window(jl):
    cu = _cu([90])
    x = _make(90, 1, 1, "bf16", "f16", 8)
    _check(_run(jl, x, cu, scale=0.02), x, cu, scale=0.02)
    assert torch.equal(_run(jl, x, cu, window=2 ** 31 - 1), _run(jl, x, cu))


def test_result_does_not_depend_on_the_batch(jl):
    lens = [77, 300, 5, 260]
    cu = _cu(lens)
    for qk, v in TYPES:
        x = _make(int(cu[-1]), 3, 3, qk, v, 9)
        whole = _run(jl, x, cu)
        for a, b in zip(cu[:-1], cu[1:]):
            one = {n: (x[n][a:b] if n in ("q", "k", "v") else x[n]) for n in x}
            assert torch.equal(_run(jl, one, _cu([b - a])), whole[a:b])


def test_capture_and_streams(jl):
    x = _make(700, 3, 3, "bf16", "f16", 10)
    x = {n: (t.cuda() if torch.is_tensor(t) else [a.cuda() for a in t]) for n, t in x.items()}
    cu = torch.tensor([0, 400, 700], dtype=torch.int32, device="cuda")
    want = _run(jl, x, cu)
    streams, outs = [torch.cuda.Stream() for _ in range(3)], [torch.zeros_like(want) for _ in range(3)]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    call = lambda o, s: jl.jd_diff_attention(x["q"], x["k"], x["v"], o, cu, *x["lam"], 0.6, norm_gain=x["gain"],  # noqa: E731
                                             status=st, stream=s)
    for _ in range(5):
        for s, o in zip(streams, outs):
            call(o, s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    g, out = torch.cuda.CUDAGraph(), torch.zeros_like(want)
    with torch.cuda.graph(g):
        call(out, torch.cuda.current_stream())
    x["q"].mul_(0.5)
    cu.copy_(torch.tensor([0, 133, 690], dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[:690], _run(jl, x, cu)[:690]) and (out[690:] == 0).all() and int(st) == 0


def test_nothing_to_do(jl):
    e = torch.empty(0, 6, 64, device="cuda", dtype=torch.bfloat16)
    v = torch.empty(0, 3, 128, device="cuda", dtype=torch.bfloat16)
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    lam = [torch.zeros(64, device="cuda")] * 4
    jl.jd_diff_attention(e, e, v, v.clone(), cu, *lam, 0.5)
    x = _make(5, 1, 1, "bf16", "f16", 11)
    assert (_run(jl, x, [0, 0, 0]) == 7).all()
