"""What a model sets up for kernels that only some weights files call (read from the source: a kernel whose compiled register
count differs from the one it is written for cannot be made here).  The differential attention refuses to be set up then;
a model without such layers must not ask for it."""
import os
import re

SRC = os.path.join(os.path.dirname(__file__), "..", "encoder_decision_model_b200", "csrc", "model.cu")


def test_only_models_with_differential_layers_prepare_its_kernels():
    text = re.sub(r"\s+", " ", re.sub(r"//[^\n]*", "", open(SRC).read()))
    assert text.count("diff_attention_prepare(") == 1
    assert ("const bool diff = std::any_of(std::begin(m->lam), std::end(m->lam), [](const float *p) { return p != nullptr; }); "
            "if (diff) CK(diff_attention_prepare(m->device));") in text
    # and the weights, the shared handle's among them, are known by then
    create = text[text.index('extern "C" jd_status jd_model_create('):text.index('extern "C" void jd_model_destroy')]
    order = [create.index(s) for s in ("load_weights(m, weights_path)", "alloc_workspace(m)", "share_weights(*m, base)")]
    assert order == sorted(order) and create.rindex("alloc_workspace(m)") > order[2]
