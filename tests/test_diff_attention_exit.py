"""How a block of k_diff_attention ends once one of its waits has expired: what it asked for (TMA copies into its shared
memory, products into its TMEM) may still be on its way, so it waits, with a limit in time and in steps, before it gives
either up.  Read from the source: nothing that a caller passes makes a wait expire."""
import os
import re

SRC = os.path.join(os.path.dirname(__file__), "..", "encoder_decision_model_b200", "csrc", "diff_attention.cu")


def test_a_block_waits_for_what_it_asked_for():
    text = re.sub(r"\s+", " ", re.sub(r"//[^\n]*", "", open(SRC).read()))
    end = text[text.rindex("__syncthreads();", 0, text.index("tmem_dealloc(tmem, 512);")):]
    end = end[:end.index("tmem_dealloc(tmem, 512);")]
    assert re.search(r"if \(\*status\) \{ const uint64_t from = globaltimer_ns\(\); "
                     r"for \(int i = 0; i < LINGER_STEPS && globaltimer_ns\(\) - from < LINGER_NS; \+\+i\) __nanosleep\(1000\); \}",
                     end), end
    steps, ns = (int(re.search(rf"{n} = ([\d']+)", text).group(1).replace("'", "")) for n in ("LINGER_STEPS", "LINGER_NS"))
    assert 1_000_000 <= ns <= 100_000_000 and ns // 1000 <= steps <= 1_000_000
