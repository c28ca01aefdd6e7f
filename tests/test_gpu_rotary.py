"""Rotary positions and head norms on the GPU against the float64 definition.

Tolerance, element by element.  The result is rounded once: eps/2 of it.  Before that the arithmetic is
FP32: sine and cosine are off by at most 2^-22 (the fraction of a turn is rounded to 2^-26, an angle of
2 pi 2^-26, and sincospif adds 2 ulp), so a rotated element is off by at most 2^-22 (|a| + |b|) plus two
roundings, within 3 * 2^-22 max|y| of its head y.  A norm adds its sum of squares (13 roundings in the
deepest chain of 256 elements), a root, a division, two products: 20 * 2^-24 of |y|; a layer norm's mean
is off by 13 * 2^-24 mean|x|, which the division by the deviation d carries into every element:
13 * 2^-24 mean|x| / d.
"""
import numpy as np
import pytest

import operator_refs as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"f32": "float32", "f16": "float16", "bf16": "bfloat16"}


@pytest.fixture(scope="module")
def jl():
    from encoder_decision_model_b200 import _lib
    from encoder_decision_model_b200.build import build
    build()
    return _lib


def _inputs(T, H, d, dtype, seed, std=1.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, H, d, generator=g) * std + 0.1).to(getattr(torch, DT[dtype]))


def _check(got, x, pos, rot, dtype, kind=None, gain=None, eps=1e-5):
    """got, x: [T, H, d] CPU tensors; rows of pos < 0 are not looked at."""
    w, amp = ref.frequencies(rot["dims"], rot["theta"], **{k: v for k, v in rot.items()
                                                          if k not in ("dims", "theta", "layout")})
    on = pos >= 0
    x64 = x.double().numpy()[on]
    y = x64 if kind is None else ref.norm(x64, kind, eps, None if gain is None else gain.double().numpy())
    z = ref.rotate(y, pos[on], w, amp, rot["layout"])
    big = np.abs(y).max(-1, keepdims=True) * amp
    tol = torch.finfo(x.dtype).eps / 2 * np.abs(z) + 3 * 2.0 ** -22 * big
    if kind:
        tol = tol + 20 * 2.0 ** -24 * big
    if kind == "layer":
        dev = np.sqrt(((x64 - x64.mean(-1, keepdims=True)) ** 2).mean(-1, keepdims=True) + eps)
        g = 1.0 if gain is None else np.abs(gain.double().numpy()).max()
        tol = tol + 2 * 13 * 2.0 ** -24 * g * np.abs(x64).mean(-1, keepdims=True) / dev
    if dtype == "f16":
        tol = tol + 2.0 ** -25  # half a step of the subnormal range
    err = np.abs(got.double().numpy()[on] - z)
    assert (err <= tol).all(), float((err / tol).max())


def _run(jl, q, k, cu, rot, kind=None, gains=(None, None), pos=None, q_out=None, k_out=None, stream=None, eps=1e-5):
    rc = jl.rotary_config(**rot)
    up = lambda a: None if a is None else torch.as_tensor(np.asarray(a), dtype=torch.int32, device="cuda")  # noqa: E731
    kw = dict(cu_seqlens=up(cu), positions=up(pos), stream=stream or torch.cuda.current_stream())
    if q_out is None:
        q_out = torch.full_like(q, 7.0, memory_format=torch.contiguous_format)
    if k_out is None and k is not None:
        k_out = torch.full_like(k, 7.0, memory_format=torch.contiguous_format)
    if kind is None:
        jl.jd_rotary(q, k, q_out, k_out, rc, **kw)
    else:
        g = [None if x is None else x.cuda() for x in gains]
        jl.jd_qk_norm_rotary(q, k, q_out, k_out, rc, norm=kind, eps=eps, q_gain=g[0], k_gain=g[1], **kw)
    torch.cuda.synchronize()
    return q_out, k_out


ROWS = {
    "one token": [1],
    "ragged with empty rows": [0, 3, 0, 0, 129, 1, 64, 0],
    "many": [(37 * i) % 53 for i in range(200)],
    "long": [8192],
}


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("head_dim,dims,layout", [
    (64, 64, "half"), (64, 32, "half"), (64, 64, "interleaved"), (64, 6, "interleaved"), (64, 20, "half"),
    (80, 80, "half"), (96, 48, "half"), (128, 128, "interleaved"), (256, 256, "half"), (256, 250, "half"),
    (8, 8, "half"), (2, 2, "interleaved"), (20, 10, "half"), (33, 32, "half"), (7, 4, "interleaved"),
])
@pytest.mark.parametrize("kind", [None, "rms", "layer"])
def test_shapes_and_layouts(jl, dtype, head_dim, dims, layout, kind):
    lens = ROWS["ragged with empty rows"]
    cu = np.concatenate([[0], np.cumsum(lens)])
    T = int(cu[-1]) + 5  # five tokens behind the last row
    q, k = _inputs(T, 5, head_dim, dtype, 1), _inputs(T, 2, head_dim, dtype, 2)
    rot = dict(dims=dims, theta=10000.0, layout=layout)
    gains = (torch.linspace(0.5, 1.5, head_dim), torch.linspace(1.5, -0.5, head_dim)) if kind else (None, None)
    qo, ko = _run(jl, q.cuda(), k.cuda(), cu, rot, kind, gains)
    pos = ref.row_positions(cu, T)
    _check(qo.cpu(), q, pos, rot, dtype, kind, gains[0])
    _check(ko.cpu(), k, pos, rot, dtype, kind, gains[1])
    assert (qo[int(cu[-1]):] == 7).all() and (ko[int(cu[-1]):] == 7).all()


@pytest.mark.parametrize("rows", list(ROWS))
@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "yarn"])
def test_rows_and_scalings(jl, rows, scaling):
    cu = np.concatenate([[0], np.cumsum(ROWS[rows])])
    T = int(cu[-1])
    rot = dict(dims=64, theta=160000.0, layout="half", scaling=scaling, factor=4.0, original_length=2048)
    q, k = _inputs(T, 6, 64, "f32", 3), _inputs(T, 6, 64, "f32", 4)
    qo, ko = _run(jl, q.cuda(), k.cuda(), cu, rot)
    pos = ref.row_positions(cu, T)
    _check(qo.cpu(), q, pos, rot, "f32")
    _check(ko.cpu(), k, pos, rot, "f32")


def test_far_positions(jl):
    pos = np.array([0, 1, 8191, 100003, 10 ** 6 + 1, 2 ** 24 + 1, 2 ** 31 - 1, 5])
    for dims, scaling in ((64, "none"), (2, "ntk"), (10, "yarn")):
        rot = dict(dims=dims, theta=10000.0, layout="half", scaling=scaling, factor=2.0)
        q = _inputs(len(pos), 3, 64, "f32", 5)
        qo, _ = _run(jl, q.cuda(), None, None, rot, pos=pos)
        _check(qo.cpu(), q, pos, rot, "f32")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", [None, "rms"])
def test_strides_alignment_and_in_place(jl, dtype, kind):
    cu, T = np.array([0, 70, 131]), 131
    rot = dict(dims=32, theta=10000.0, layout="half")
    base = _inputs(T, 18, 64, dtype, 6)
    want, wk = _run(jl, base[:, :6].contiguous().cuda(), base[:, 6:12].contiguous().cuda(), cu, rot, kind)
    # q | k | v in one row
    packed = base.cuda()
    got, gk = _run(jl, packed[:, :6], packed[:, 6:12], cu, rot, kind)
    assert torch.equal(got, want) and torch.equal(gk, wk)
    # heads outermost, and outputs of another order
    turned = base.permute(1, 0, 2).contiguous().cuda().permute(1, 0, 2)
    out = torch.empty(6, T, 64, dtype=base.dtype, device="cuda").permute(1, 0, 2)
    got, _ = _run(jl, turned[:, :6], turned[:, 6:12], cu, rot, kind, q_out=out)
    assert torch.equal(got, want)
    # one element past a 16-byte boundary, an odd token stride
    odd = torch.zeros(T, 18 * 64 + 1, dtype=base.dtype, device="cuda")
    odd[:, 1:] = base.flatten(1).cuda()
    odd = odd[:, 1:].unflatten(1, (18, 64))
    oq, ok = _run(jl, odd[:, :6], odd[:, 6:12], cu, rot, kind)
    # (another kernel, which sums a head's squares in another order: the tolerance against the definition)
    pos = ref.row_positions(cu, T)
    _check(oq.cpu(), base[:, :6], pos, rot, dtype, kind)
    _check(ok.cpu(), base[:, 6:12], pos, rot, dtype, kind)
    # in place, the values beside them untouched
    for x, a, b in ((packed, want, wk), (odd, oq, ok)):
        v = x[:, 12:].clone()
        _run(jl, x[:, :6], x[:, 6:12], cu, rot, kind, q_out=x[:, :6], k_out=x[:, 6:12])
        assert torch.equal(x[:, :6], a) and torch.equal(x[:, 6:12], b) and torch.equal(x[:, 12:], v)
    # one row of heads for every token (stride 0)
    one = base[:1, :6].cuda().expand(T, 6, 64)
    got, _ = _run(jl, one, None, cu, rot, kind)
    full, _ = _run(jl, one.contiguous(), None, cu, rot, kind)
    assert torch.equal(got, full)


def test_infinities_and_nan_stay_where_they_are(jl):
    rot = dict(dims=32, theta=10000.0, layout="half")
    for odd_dims in (32, 20):
        rot["dims"] = odd_dims
        q = _inputs(9, 4, 64, "f32", 7)
        q[3, 1, 40], q[3, 1, 41], q[5, 2, 3] = float("inf"), float("nan"), float("nan")
        got = _run(jl, q.cuda(), None, [0, 9], rot)[0].cpu()
        bad = ~torch.isfinite(got)
        want = torch.zeros_like(bad)
        want[3, 1, 40:42] = True
        want[5, 2, 3] = want[5, 2, 3 + odd_dims // 2] = True
        assert torch.equal(bad, want) and got[3, 1, 40] == float("inf")


def test_norm_of_zeros_and_of_large_values(jl):
    q = torch.zeros(4, 2, 64)
    q[1] = 3e4
    q[2] = 1e-30
    rot = dict(dims=64, theta=10000.0, layout="half")
    got, _ = _run(jl, q.cuda(), None, None, rot, "rms", pos=np.zeros(4))
    assert (got[0] == 0).all() and torch.allclose(got[1], torch.ones(2, 64, device="cuda"), atol=1e-6)
    got, _ = _run(jl, q.cuda(), None, None, rot, "layer", pos=np.zeros(4), eps=0.0)
    assert torch.isnan(got[0]).all()  # 0 / 0 where the definition has it


def test_no_tokens_and_capture(jl):
    rc = jl.rotary_config(64, 10000.0)
    e = torch.empty(0, 6, 64, device="cuda")
    jl.jd_rotary(e, e, e, e, rc)
    q, k = _inputs(50, 6, 64, "bf16", 8).cuda(), _inputs(50, 6, 64, "bf16", 9).cuda()
    cu = torch.tensor([0, 20, 50], dtype=torch.int32, device="cuda")
    qo, ko = torch.zeros_like(q), torch.zeros_like(k)
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        jl.jd_qk_norm_rotary(q, k, qo, ko, rc, cu_seqlens=cu, stream=torch.cuda.current_stream())
    q2 = _inputs(50, 6, 64, "bf16", 10).cuda()
    q.copy_(q2)
    cu.copy_(torch.tensor([0, 33, 50], dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    want, _ = _run(jl, q2, k, [0, 33, 50], dict(dims=64, theta=10000.0), "rms")
    assert torch.equal(qo, want)


def test_two_streams_at_once(jl):
    q, k = _inputs(5000, 6, 64, "bf16", 11).cuda(), _inputs(5000, 6, 64, "bf16", 12).cuda()
    rot = dict(dims=64, theta=10000.0, layout="half")
    want, wk = _run(jl, q, k, [0, 5000], rot)
    torch.cuda.synchronize()
    cu = torch.tensor([0, 5000], dtype=torch.int32, device="cuda")
    rc, streams = jl.rotary_config(**rot), [torch.cuda.Stream() for _ in range(2)]
    outs = [(torch.zeros_like(q), torch.zeros_like(k)) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, o in zip(streams, outs):
            jl.jd_rotary(q, k, *o, rc, cu_seqlens=cu, stream=s)
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o[0], want) and torch.equal(o[1], wk)
