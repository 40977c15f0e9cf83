"""The drawn cases of perf/more_operators.py, the kernels against 64 bits: the
error's 2-norm over that of the exact values rounded once. Prints the largest
ratio of every bf16 result (run with -s)."""
import importlib.util
import os
import random

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
spec = importlib.util.spec_from_file_location("model_operators",
                                              os.path.join(ROOT, "perf", "more_operators.py"))
operators = importlib.util.module_from_spec(spec)
spec.loader.exec_module(operators)

# A bf16 result is rounded once; binary32 before it adds 2^-10 of that.
ONCE = 1.05
DRAWS, GROUPS = 240, 8
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
        state = operators.prepare(case, seed)
        got, want = operators.run(state), operators.exact(case, seed)
        assert set(got) == set(want)
        moved = 0.0
        if case["op"] == "linear":
            # A token's integer that is one off (see q below) moves its outputs by
            # its weights times both scales, through an activation whose slope
            # stays under 1.13: that much is the integers' difference and not the
            # product's error.
            d = (got["q"].long() - want["q"]).double() @ state["weight"].double().t().contiguous()
            moved = 1.13 * float((d * want["scale"][:, None] * state["weight_scale"]).norm())
        for n, w in want.items():
            g, where = got[n], (seed, n, case)
            if g.dtype == torch.bfloat16:
                r = ratio(g, w)
                key = case["op"], n
                largest[key] = max(largest.get(key, (0, None)), (r, seed))
                assert r <= ONCE, (r, where)
            elif n == "q":
                # The exact form's scale is the quotient by 127, the call's the
                # product: 2^-23 apart at most, which moves a quotient of up to
                # 127 by 1.5e-5, over a middle in 3e-5 of all cases
                off = (g.long() - w).abs()
                assert int(off.max()) <= 1 and int(off.sum()) <= 2 + 1e-4 * off.numel(), where
            elif g.dtype == torch.float8_e4m3fn:
                # binary32's few roundings of a state (2^-21 of its terms, and m's
                # may cancel to a sixteenth of them) against numbers 2^-4 to 2^-3
                # apart that 16 random bits choose from: one in 2^13 at most goes
                # to the other neighbour
                off = g.double() - w
                far = off != 0
                assert bool((off.abs() <= w.abs() / 7 + 2.0 ** -9).all()), where
                assert int(far.sum()) <= 2 + 2.0 ** -13 * g.numel(), where
            else:
                # binary32: results and sums of up to 100,000 rows, 2^-16 of
                # their size
                off = float((g.double() - w).norm())
                assert off <= 2.0 ** -16 * float(w.norm()) + 1e-30 + (moved if n == "out" else 0), where
        del got, want, state
    print({"%s %s" % k: "%.3f (draw %d)" % v for k, v in sorted(largest.items())}, flush=True)
