"""The status word of a differential attention call only collects: what a caller left in it must not reach the kernel's
waits, which give up early once a wait of their own CTA has expired.  Read from the source (no device needed: a kernel whose
waits give up works on tiles that have not landed, and is not run)."""
import os
import re

SRC = os.path.join(os.path.dirname(__file__), "..", "encoder_decision_model_b200", "csrc", "diff_attention.cu")


def _kernel():
    text = re.sub(r"//[^\n]*", "", open(SRC).read())
    body = text[text.index("k_diff_attention(const __grid_constant__ CUtensorMap tm_q"):]
    return body[:body.index("k_diff_attention_f32")]


def test_waits_go_by_the_ctas_own_word():
    body = _kernel()
    calls = re.findall(r"\b(?:mbar_)?wait\(((?:[^()]|\((?:[^()]|\([^()]*\))*\))*)\)", body)
    # producer: q, k, v; tail of V; MMA issue: k, P used, q, v, P, O read, next q; softmax: S, O at rest; read-out: sums, two O
    assert len(calls) == 16 and all(c.split(",")[-1].strip() == "status" for c in calls), calls
    assert re.findall(r"unsigned \*status = [^;]*;", body) == ["unsigned *status = tmem_slot + 1;"]


def test_callers_word_is_only_written():
    assert re.findall(r"[^;{}]*p\.status[^;]*;", _kernel()) == [
        "\n    if (threadIdx.x == 0 && p.status && *status) atomicOr(p.status, *status);"]
