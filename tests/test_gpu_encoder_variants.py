"""Models whose weights file carries the encoder layers' optional tensors: head norms, differential
attention, other rotations.  The whole forward pass against the oracle, at the parity tolerances of the plain
model, through every entry point."""
import struct

import numpy as np
import pytest

import gpu_helpers as gh
from workloads import rows_config1, rows_config2, variant_tensors, write_weights

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

OPTS = dict(max_length=8192, head_budget=512, strict=True)
VARIANTS = {
    # steep scores (head norms with gains around 3) through the plain attention, rotations of their own pass
    "norms": dict(norms=range(22), gain=3.0, rotary=[[1, 32, 160000.0, 2, 2.0, 0, 0, 0], [0, 64, 10000.0, 1, 2.0, 0, 0, 0]]),
    # differential attention in global and local layers, some with norms; the global rotation stays in the GEMM
    "diff": dict(norms=(1, 3, 20), diff=(0, 1, 2, 3, 7, 12, 20, 21),
                 rotary=[[0, 64, 160000.0, 3, 4.0, 512, 32.0, 1.0], [0, 40, 10000.0, 0, 1.0, 0, 0, 0]]),
}


@pytest.fixture(scope="module")
def jl():
    from encoder_decision_model_b200 import _lib
    from encoder_decision_model_b200.build import build
    build()
    return _lib


@pytest.fixture(scope="module", params=list(VARIANTS))
def weights(request, tmp_path_factory):
    path = tmp_path_factory.mktemp("weights") / f"{request.param}.jdw"
    write_weights(path, extra=variant_tensors(5, **VARIANTS[request.param]))
    yield path
    path.unlink()


def _rows():
    return rows_config1() + [r for r in rows_config2(8) if len(r.state) > 300][:2]


@pytest.mark.parametrize("precision", ["bf16", "fp32", "fp8"])
def test_forward_matches_oracle(jl, weights, precision):
    rows = _rows()
    prec = {"bf16": jl.JD_PREC_BF16, "fp32": jl.JD_PREC_FP32, "fp8": jl.JD_PREC_FP8}[precision]
    m = jl.Model(weights, 8192, 16, 256, precision=prec)
    hb, res = gh.device_run(m, rows, OPTS, taps=True)
    if (weights.stem, precision) == ("norms", "fp8"):
        # E4M3 operands round by 2^-4 / sqrt(3) = 0.036 in the mean square, input and weight: a query or key is off by
        # 0.05 of its length, a score of deviation 9 by 9 * 0.05 * sqrt(2) = 0.65.  No tolerance says anything about
        # probabilities a factor of two off: only that the outputs are numbers.
        assert np.isfinite(res["logits"]).all() and np.isfinite(res["encoder_out"]).all()
        m.close()
        return
    want = gh.oracle_run(weights, rows, OPTS)
    gh.compare(hb, res, want, bf16=precision != "fp32", label=f"{weights.stem} {precision}", check_taps=False)
    tol = tap_tolerance(weights.stem, precision)
    for i, r in want.items():
        for got, name in ((res["encoder_out"][hb.cu_seqlens[i]:hb.cu_seqlens[i + 1]], "encoder_out"),
                          (res["marker_state"][hb.opt_off[i]:hb.opt_off[i + 1]], "marker_state")):
            rel = np.linalg.norm(got - r[name]) / np.linalg.norm(r[name])
            assert rel <= tol, (weights.stem, precision, i, name, rel)
    m.close()


def tap_tolerance(variant, precision):
    """The plain model's relative tolerance of the taps (1e-4 in FP32, 3e-2 in 16 bits), except where 16-bit
    queries and keys meet steep scores.  With gains around 3 a head's query and key are 24 long, so scores have a
    deviation of 24 * 24 / 8 / 8 = 9.  Queries and keys are rounded to BF16 twice each (out of the projection, out of
    the norm), 2^-9 / sqrt(3) of an element in the mean square: a score is off by sqrt(4) * 2^-9 / sqrt(3) * 9 = 0.020, and
    so, relatively, are the probabilities and each layer's attention output.  An input that is off by e turns scores
    by sqrt(2) * 9 e = 12.7 e: the 0.020 of one layer come back in the later layers' attention as up to 0.26 of what
    they add.  Attention adds under a third of the residual stream's energy: 0.020 + 0.26 / 3 = 0.11 in all.  (The FP32
    mode, with the same amplification of 2^-24, keeps its 1e-4.)"""
    if precision == "fp32":
        return 1e-4
    return 0.11 if variant == "norms" else 3e-2


def test_every_entry_point_agrees(jl, weights):
    rows = _rows()[:4]
    m = jl.Model(weights, 4096, 16, 256)
    hb, want = gh.device_run(m, rows, OPTS)
    launches = m.jd_last_launch_count()
    v = VARIANTS[weights.stem]
    plain = jl.Model(gh_plain(), 4096, 16, 256)
    gh.device_run(plain, rows, OPTS)
    # one more launch for each layer whose rotation has a pass of its own
    own = [l for l in range(22) if l in v["norms"] or (l % 3 and v["rotary"][1][1] != 64) or (l % 3 == 0 and v["rotary"][0][0])]
    assert launches == plain.jd_last_launch_count() + len(own)
    plain.close()
    out = m.jd_decide_host(rows, jl.encode_opts(**OPTS))
    np.testing.assert_array_equal(out["logits"], want["logits"])
    s = jl.Model.shared(m, 2048, 8, 128)
    _, got = gh.device_run(s, rows[:3], OPTS)  # no row's result depends on the rest of its batch
    np.testing.assert_array_equal(got["logits"], want["logits"][:len(got["logits"])])
    s.close()
    m.jd_set_graph_mode(True)
    for _ in range(3):
        _, got = gh.device_run(m, rows, OPTS)
        np.testing.assert_array_equal(got["logits"], want["logits"])
    m.jd_set_graph_mode(False)
    hb, small = gh.device_run(m, rows[:3], OPTS)
    up = [torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in (hb.tokens, hb.cu_seqlens, hb.mask_pos, hb.opt_off, hb.row_type)]
    logits = torch.zeros(hb.n_markers, device="cuda")
    m.jd_forward_noalloc(jl.Model.device_batch(hb.n_rows, hb.n_tokens, hb.n_markers, hb.max_row_len, *up), logits)
    m.jd_noalloc_check_status()
    np.testing.assert_array_equal(logits.cpu().numpy(), small["logits"])
    m.close()


def gh_plain():
    from workloads import weights_path
    return weights_path(0)


def test_incomplete_or_invalid_tensors_are_refused(jl, weights):
    """A norm without its other half, a rotation that does not exist: edited in the file, then put back."""
    name = b"enc.3.k_norm.g"
    with open(weights, "r+b") as fh:
        head = fh.read(1 << 16)
        at = head.index(name)
        fh.seek(at)
        fh.write(b"enc.3.x_norm.g")
    with pytest.raises(jl.JDError) as e:
        jl.Model(weights, 256, 4, 64)
    assert e.value.code == jl.JD_ERR_IO and "k_norm" in str(e.value)
    from workloads import read_weight_index
    with open(weights, "r+b") as fh:
        fh.seek(at)
        fh.write(name)
    _, off = read_weight_index(weights)["enc.rotary"]
    for i, bad in ((0, 2.0), (1, 66.0), (1, 33.0), (2, -1.0), (3, 7.5), (9, float("nan"))):
        with open(weights, "r+b") as fh:
            fh.seek(off + 4 * i)
            old = fh.read(4)
            fh.seek(off + 4 * i)
            fh.write(struct.pack("<f", bad))
        with pytest.raises(jl.JDError) as e:
            jl.Model(weights, 256, 4, 64)
        assert e.value.code == jl.JD_ERR_IO and "enc.rotary" in str(e.value)
        with open(weights, "r+b") as fh:
            fh.seek(off + 4 * i)
            fh.write(old)
