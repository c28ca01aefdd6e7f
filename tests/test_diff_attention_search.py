"""How `k_diff_attention` (csrc/diff_attention.cu) finds its work, restated with the state it carries.

Item w is head w % heads of query tile w // heads; row r's tiles start at number cu[r] // 128 + r.  A CTA takes the
items blockIdx, blockIdx + grid, ...; each of its roles looks for an item's row 32 rows at a time from `lo`, the row of
its last item, and goes on by 31 rows when all 32 start at or before the tile.  Over all CTAs of a launch every tile of
every row and head must be found exactly once.  (The FP32 kernel searches from the first row each time.)
"""
import os
import random
import re

import pytest

SRC = os.path.join(os.path.dirname(__file__), "..", "encoder_decision_model_b200", "csrc", "diff_attention.cu")
TILE = 128


def find_item(cu, starts, b, lo):
    """(row, first query, carried lo) of tile number b."""
    n = len(starts)
    while True:
        below = 0  # the ballot: lane i looks at row lo + i
        while below < 32 and lo + below < n and starts[lo + below] <= b:
            below += 1
        if below == 32:
            lo += 31
            continue
        lo += max(below, 1) - 1
        return lo, cu[lo] + (b - starts[lo]) * TILE, lo


def launch(cu, n_tokens, heads, sms=148):
    """(row, head, first query) of every item that the CTAs of one launch find on."""
    n = len(cu) - 1
    starts = [c // TILE + r for r, c in enumerate(cu[:-1])]
    items = (n_tokens // TILE + n) * heads
    grid = min(items, sms)
    found = []
    for cta in range(grid):
        lo = 0
        for w in range(cta, items, grid):
            b, h = divmod(w, heads)
            row, q0, lo = find_item(cu, starts, b, lo)
            if cu[row] <= q0 < cu[row + 1]:
                found.append((row, h, q0))
    return found


def _check(lens, heads, behind=0, sms=148):
    cu = [0]
    for x in lens:
        cu.append(cu[-1] + x)
    found = launch(cu, cu[-1] + behind, heads, sms)
    want = [(r, h, q) for r in range(len(lens)) for h in range(heads) for q in range(cu[r], cu[r + 1], TILE)]
    assert sorted(found) == want, (lens, heads, behind, sms)


@pytest.mark.parametrize("heads", [1, 2, 3, 6])
def test_every_row_count(heads):
    for n in range(1, 401):
        rng = random.Random(100 * n + heads)
        _check([rng.randint(1, 70) for _ in range(n)], heads)
        top = rng.choice([0, 1, 127, 128, 129, 1000])
        _check([rng.randint(0, top) for _ in range(n)], heads, behind=rng.choice([0, 1, 500]))


def test_same_lengths_and_other_grids():
    for n in (31, 32, 33, 62, 63, 64, 93, 94, 95, 125, 156, 400):
        for length in (1, 68, 100, 128, 300):
            for heads, sms in ((1, 148), (2, 148), (3, 148), (1, 1), (3, 7), (2, 64)):
                _check([length] * n, heads, sms=sms)


def test_random_batches():
    for seed in range(400):
        rng = random.Random(seed)
        n, heads = rng.randint(1, 400), rng.randint(1, 6)
        low, top = rng.choice([0, 1, 64]), rng.choice([70, 128, 300, 1000])
        _check([rng.randint(low, top) if rng.random() < 0.9 else 0 for _ in range(n)], heads, behind=rng.choice([0, 64]))


def test_restates_the_source():
    """The search's lines, with what surrounds them."""
    text = re.sub(r"\s+", " ", re.sub(r"//[^\n]*", "", open(SRC).read()))
    for line in (
        "const int b = w / p.heads; t.h = w - b * p.heads; for (;;) { const int at = lo + lane, v = p.cu[min(at, p.n_rows)]; "
        "const unsigned below = __ballot_sync(0xffffffffu, at < p.n_rows && (v >> 7) + at <= b); "
        "if (below == 0xffffffffu) { lo += 31; continue; } "
        "const int k = 31 - __clz(below | 1u); "
        "t.cs = max(__shfl_sync(0xffffffffu, v, k), 0); t.ce = min(__shfl_sync(0xffffffffu, v, k + 1), p.n_tokens); "
        "lo += k; break; }",
        "t.q0 = t.cs + (b - (t.cs >> 7) - lo) * TQ; t.on = t.q0 >= t.cs && t.q0 < t.ce;",
        "for (t.on = false; w < n_items && !t.on; w += gridDim.x) t = find_item(p, w, lane, lo);",
        "for (int w = blockIdx.x; w < n_items; w += gridDim.x) { const Item t = find_item(p, w, lane, row); if (!t.on) continue;",
        "const int64_t items = ((int64_t)op.n_tokens / TQ + op.n_rows) * op.heads;",
    ):
        assert line in text, line
