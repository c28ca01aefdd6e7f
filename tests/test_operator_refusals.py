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
