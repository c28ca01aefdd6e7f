"""What the operator calls refuse, and the binding's records of their arguments (no device needed)."""
import ctypes as C
import os
import re
import subprocess

import pytest

from encoder_decision_model_b200 import _lib as jl
from encoder_decision_model_b200.build import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def L():
    build()
    return jl.lib()


def _heads(n, d=64, base=0x10000):
    return jl.jd_heads(base, n * d, d, n)


def _rotary(**kw):
    a = jl.jd_rotary_args(jl.rotary_config(64, 10000.0), jl.JD_BF16, 64, 100, 2, None, 0x900000, _heads(6),
                          _heads(6, base=0x200000), _heads(6, base=0x400000), _heads(6, base=0x600000))
    for name, v in kw.items():
        obj = a
        *path, last = name.split("__")
        for p in path:
            obj = getattr(obj, p)
        setattr(obj, last, v)
    return a


@pytest.mark.parametrize("change,word", [
    (dict(dtype=3), "dtype"), (dict(head_dim=1), "head_dim"), (dict(head_dim=257), "head_dim"),
    (dict(n_tokens=-1), "negative"), (dict(n_rows=-1), "negative"), (dict(n_rows=0), "cu_seqlens"),
    (dict(n_tokens=(1 << 30) + 1), "too many"),
    (dict(cu_seqlens=None), "cu_seqlens"), (dict(q__n_heads=0), "heads"), (dict(k__n_heads=-1), "heads"),
    (dict(q_out__n_heads=5), "n_heads"), (dict(k_out__n_heads=7), "n_heads"),
    (dict(q__data=None), "NULL"), (dict(k_out__data=None), "NULL"),
    (dict(rotary__layout=2), "layout"), (dict(rotary__dims=0), "dims"), (dict(rotary__dims=63), "dims"),
    (dict(rotary__dims=66), "dims"), (dict(rotary__theta=0.0), "theta"), (dict(rotary__theta=float("nan")), "theta"),
    (dict(rotary__theta=float("inf")), "theta"), (dict(rotary__scaling=4), "scaling"),
    (dict(rotary__scaling=1, rotary__factor=0.0), "factor"),
    (dict(rotary__scaling=2, rotary__factor=float("inf")), "factor"),
    (dict(rotary__scaling=3, rotary__original_length=0), "yarn"),
    (dict(rotary__scaling=3, rotary__beta_fast=1.0), "yarn"), (dict(rotary__scaling=3, rotary__theta=1.0), "yarn"),
    (dict(q__token_stride=-1), "strides"), (dict(q_out__token_stride=0), "overlap"),
    (dict(q_out__head_stride=63), "overlap"), (dict(q_out__token_stride=383), "overlap"),
    (dict(k_out__token_stride=1 << 60), "strides"),
    (dict(q_out__data=0x10000, q_out__token_stride=768), "other strides"),
    (dict(q_out__data=0x600000), "other output"), (dict(k_out__data=0x10000), "other input"),
])
def test_rotary_refuses(L, change, word):
    norm = jl.jd_head_norm(0, 1e-5, None, None)
    a = _rotary(**change)
    for code in (L.jd_rotary(C.byref(a), None), L.jd_qk_norm_rotary(C.byref(a), C.byref(norm), None)):
        assert code == jl.JD_ERR_INVALID_ARG
        assert word in L.jd_last_error().decode()


def test_rotary_null_arguments_and_norms(L):
    a = _rotary()
    assert L.jd_rotary(None, None) == jl.JD_ERR_INVALID_ARG
    assert L.jd_qk_norm_rotary(C.byref(a), None, None) == jl.JD_ERR_INVALID_ARG
    for kind, eps in ((2, 1e-5), (-1, 1e-5), (0, -1.0), (1, float("nan"))):
        n = jl.jd_head_norm(kind, eps, None, None)
        assert L.jd_qk_norm_rotary(C.byref(a), C.byref(n), None) == jl.JD_ERR_INVALID_ARG
        assert "norm" in L.jd_last_error().decode()


def test_nothing_to_do_needs_no_device(L):
    a = _rotary(n_tokens=0, q__data=None, k__data=None, q_out__data=None, k_out__data=None, cu_seqlens=None)
    assert L.jd_rotary(C.byref(a), None) == jl.JD_OK


def test_host_memory_or_no_device_is_an_error(L):
    buf = (C.c_float * 4096)()
    p = C.addressof(buf)
    h = [jl.jd_heads(p + 4096 * i, 64, 64, 1) for i in range(4)]
    a = jl.jd_rotary_args(jl.rotary_config(64, 10000.0), jl.JD_F32, 64, 4, 1, None, p, *h)
    assert L.jd_rotary(C.byref(a), None) in (jl.JD_ERR_CUDA, jl.JD_ERR_INVALID_ARG)
    assert list(buf) == [0.0] * 4096


def test_binding_refuses(L):
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 2, 64)
    rc = jl.rotary_config(64, 1e4)
    cu = torch.zeros(2, dtype=torch.int32)
    for args, kw in [((x[0], None, x, None), {}), ((x, None, x[:3], None), {}), ((x, x[:, :, :32], x, x), {}),
                     ((x, x.half(), x, x), {}), ((x, x, x, None), {}), ((x.transpose(1, 2), None, x, None), {}),
                     ((x.long(), None, x.long(), None), {}), ((x, None, x, None), dict(cu_seqlens=cu.long())),
                     ((x, None, x, None), dict(cu_seqlens=cu, positions=cu))]:
        with pytest.raises(jl.JDError) as e:
            jl.jd_rotary(*args, rc, **{"cu_seqlens": cu, **kw})
        assert e.value.code == jl.JD_ERR_INVALID_ARG
    for kw in (dict(norm="group"), dict(q_gain=torch.ones(63)), dict(k_gain=torch.ones(64).half())):
        with pytest.raises(jl.JDError):
            jl.jd_qk_norm_rotary(x, None, x, None, rc, cu_seqlens=cu, **kw)
    for kw in (dict(layout="third"), dict(scaling="other")):
        with pytest.raises(jl.JDError):
            jl.rotary_config(64, 1e4, **kw)


def test_argument_records_have_the_headers_layout(tmp_path):
    """sizeof and offsetof of every operator struct, as a C compiler sees the header, against the binding's."""
    structs = [n for n in ("jd_heads", "jd_rotary_config", "jd_rotary_args", "jd_head_norm", "jd_diff_attention_args")
               if hasattr(jl, n)]
    lines, want = [], []
    for n in structs:
        ct = getattr(jl, n)
        lines.append(f'printf("%zu\\n", sizeof({n}));')
        want.append(C.sizeof(ct))
        for f, _ in ct._fields_:
            lines.append(f'printf("%zu\\n", offsetof({n}, {f}));')
            want.append(getattr(ct, f).offset)
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include "julia_decide.h"\nint main(void) {\n' + "\n".join(lines) + "\nreturn 0; }\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)],
                   check=True)
    got = [int(x) for x in re.findall(r"\d+", subprocess.run([str(exe)], capture_output=True, text=True).stdout)]
    assert got == want
    # the bytes that the binding packs are those structures
    assert jl._ROTARY_ARGS.size == C.sizeof(jl.jd_rotary_args) and jl._HEAD_NORM.size == C.sizeof(jl.jd_head_norm)
    torch = pytest.importorskip("torch")
    x = torch.zeros(5, 7, 16)
    y, cu, pos = torch.zeros(5, 3, 16), torch.zeros(3, dtype=torch.int32), torch.zeros(5, dtype=torch.int32)
    rc = jl.rotary_config(8, 3.0, "interleaved", "yarn", 2.0, 77, 30.0, 2.0)
    data, d = jl._rotary_args(x, y, x.clone(), y.clone(), rc, cu, pos)
    a = jl.jd_rotary_args.from_buffer_copy(data)
    assert d == 16 and bytes(a.rotary) == bytes(rc)
    assert (a.dtype, a.head_dim, a.n_tokens, a.n_rows, a.positions, a.cu_seqlens) == (
        jl.JD_F32, 16, 5, 2, pos.data_ptr(), cu.data_ptr())
    assert (a.q.data, a.q.token_stride, a.q.head_stride, a.q.n_heads) == (x.data_ptr(), 112, 16, 7)
    assert (a.k.data, a.k.token_stride, a.k.n_heads, a.k_out.n_heads) == (y.data_ptr(), 48, 3, 3)


def _diff(**kw):
    h = [_heads(6, base=0x100000), _heads(6, base=0x200000), _heads(3, 128, base=0x300000),
         _heads(3, 128, base=0x400000)]
    a = jl.jd_diff_attention_args(jl.JD_BF16, jl.JD_F16, 100, 2, 3, -1, 0x900000, *h, 0x910000, 0x910100, 0x910200,
                                  0x910300, 0x910400, 0.5, 1e-5, 0.0, None)
    for name, v in kw.items():
        obj = a
        *path, last = name.split("__")
        for p in path:
            obj = getattr(obj, p)
        setattr(obj, last, v)
    return a


@pytest.mark.parametrize("change,word", [
    (dict(qk_dtype=3), "dtype"), (dict(qk_dtype=-1), "dtype"), (dict(v_dtype=0), "v_dtype"),
    (dict(qk_dtype=0), "v_dtype"), (dict(n_tokens=-1), "negative"), (dict(n_rows=-2), "negative"),
    (dict(kv_heads=0), "heads"), (dict(kv_heads=2), "heads"), (dict(out__n_heads=0), "heads"),
    (dict(q__n_heads=5), "heads"), (dict(k__n_heads=3), "heads"), (dict(v__n_heads=6), "heads"),
    (dict(n_tokens=(1 << 24) + 1), "too many"), (dict(n_rows=1 << 30), "too many"),
    (dict(lambda_init=float("nan")), "lambda_init"), (dict(norm_eps=-1.0), "norm_eps"),
    (dict(scale=float("inf")), "scale"), (dict(scale=-0.125), "scale"), (dict(q__token_stride=0), "strides"), (dict(k__head_stride=0), "strides"),
    (dict(v__token_stride=-8), "strides"), (dict(q__head_stride=1 << 39), "strides"),
    (dict(out__token_stride=0), "overlap"), (dict(out__head_stride=64), "overlap"),
    (dict(q__data=None), "NULL"), (dict(cu_seqlens=None), "NULL"), (dict(lambda_k2=None), "NULL"),
    (dict(q__data=0x100008), "alignment"), (dict(k__token_stride=388), "alignment"),
    (dict(v__head_stride=132), "alignment"), (dict(out__data=0x400002), "alignment"),
    (dict(out__data=0x300000), "input"),
])
def test_diff_attention_refuses(L, change, word):
    a = _diff(**change)
    assert L.jd_diff_attention(C.byref(a), None) == jl.JD_ERR_INVALID_ARG
    assert word in L.jd_last_error().decode()


def test_diff_attention_nothing_to_do_and_null(L):
    assert L.jd_diff_attention(None, None) == jl.JD_ERR_INVALID_ARG
    for kw in (dict(n_tokens=0), dict(n_rows=0)):
        a = _diff(cu_seqlens=None, q__data=None, **kw)
        assert L.jd_diff_attention(C.byref(a), None) == jl.JD_OK


def test_diff_attention_binding_refuses(L):
    torch = pytest.importorskip("torch")
    q, k, v, o = torch.zeros(4, 6, 64), torch.zeros(4, 6, 64), torch.zeros(4, 3, 128), torch.zeros(4, 3, 128)
    cu, lam = torch.zeros(2, dtype=torch.int32), [torch.zeros(64)] * 4
    for args in ((q, k, v[:3], o), (q, k.half(), v, o), (q, k, v, o.half()), (q[:, :, :32], k, v, o),
                 (q, k, v[:, :, :64], o), (q[0], k, v, o)):
        with pytest.raises(jl.JDError):
            jl.jd_diff_attention(*args, cu, *lam, 0.5)
    for kw in (dict(norm_gain=torch.ones(64)), dict(status=torch.zeros(1))):
        with pytest.raises(jl.JDError):
            jl.jd_diff_attention(q, k, v, o, cu, *lam, 0.5, **kw)
    with pytest.raises(jl.JDError):
        jl.jd_diff_attention(q, k, v, o, cu.long(), *lam, 0.5)
    # the bytes packed are the structure
    assert jl._DIFF_ARGS.size == C.sizeof(jl.jd_diff_attention_args)
