"""The drawn cases of perf/operators.py, the kernels against 64 bits: the
error's 2-norm over that of the exact values rounded once to bf16. Prints the
largest ratio of every result (run with -s)."""
import importlib.util
import os
import random

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
spec = importlib.util.spec_from_file_location("block_operators",
                                              os.path.join(ROOT, "perf", "operators.py"))
operators = importlib.util.module_from_spec(spec)
spec.loader.exec_module(operators)

# A norm or a turn rounds once; binary32 sums add 2^-10 of that. An attention
# output carries a second rounding of the same size (of P), a gradient that of
# dS or P and up to half of one through D: sqrt(2) and sqrt(2.5) over many
# elements. 2 leaves room for draws of a few rows and keys.
ONCE, MORE = 1.05, 2.0
LIMIT = {"r": ONCE, "h": ONCE, "dx": ONCE, "dy": ONCE, "dq": MORE, "dk": MORE, "dv": MORE}
DRAWS, GROUPS = 300, 10
largest = {}


def ratio(got, want):
    """Error over one rounding's; a result that is 0 but for the 64-bit form's
    own roundings counts as exact when it is as small."""
    off = float((got.double() - want).norm())
    once = float((want.bfloat16().double() - want).norm())
    return off / (once + 1e-9 * max(1.0, want.numel() ** 0.5))


@pytest.mark.parametrize("group", range(GROUPS))
def test_errors_of_drawn_cases(group, monkeypatch):
    monkeypatch.setattr(operators, "own", True)
    for seed in range(group, DRAWS, GROUPS):
        case = operators.draw(random.Random(seed))
        got, want = operators.run(operators.prepare(case, seed)), operators.exact(case, seed)
        assert set(got) == set(want)
        for n, w in want.items():
            if w is None:
                assert got[n] is None
            elif got[n].dtype == torch.bfloat16:
                limit = MORE if n == "out" and case["op"] == "attention" else LIMIT.get(n, ONCE)
                r = ratio(got[n], w)
                key = case["op"], n
                largest[key] = max(largest.get(key, (0, None)), (r, seed))
                assert r <= limit, (seed, n, r, case)
            else:
                # binary32: results and sums of up to 100,000 rows, 2^-16 of
                # their size; lse the same of its own (scores stay under 10)
                there = torch.isfinite(w)
                assert torch.equal(got[n][~there].double(), w[~there]), (seed, n)
                off = (got[n].double() - w)[there].norm()
                assert float(off) <= 2.0 ** -16 * float(w[there].norm()) + 1e-30, (seed, n, case)
        del got, want
    print({"%s %s" % k: "%.3f (draw %d)" % v for k, v in sorted(largest.items())}, flush=True)
