"""The rule that lays out a scan's work chooses each of its layouts for some call."""

from __future__ import annotations

import random

import scan_layouts as plan
import test_gpu_scan
import test_gpu_scan_layouts as gpu


def calls(n, seed=0):
    g = random.Random(seed)
    spread = lambda a, b: int(a * (b / a) ** g.random())  # noqa: E731
    for _ in range(n):
        size, N, D = g.choice([2, 4]), g.choice([1, 1, spread(2, 200)]), spread(1, 8192)
        longest = spread(1, 300000)
        lens = [longest] + [spread(1, longest + 1) for _ in range(N - 1)]
        yield lens, spread(1, 5000), D, size, g.random() < 0.5


def test_every_layout_is_the_best_of_some_call():
    seen = {}
    for lens, heads, D, size, backward in calls(20000):
        got = plan.layout(lens, heads, D, size, backward)
        seen.setdefault((plan.way_of(D, size), backward), set()).add(got)
    narrow = {c for c in plan.choices() if c[0] == 32}
    for (way, backward), got in seen.items():
        want = narrow if backward or way != plan.TMA else set(plan.choices())
        assert got == want | {"walk"}, (way, backward, got ^ (want | {"walk"}))
    assert len(seen) == 6


def test_wide_cases_are_laid_out_as_they_say():
    for (B, T, D, size), want in gpu.WIDE.items():
        assert plan.way_of(D, size) == plan.TMA
        assert plan.layout([T], B, D, size, False) == want, (B, T, D, size)
    for (lens, H, D), want in gpu.WIDE_PACKED.items():
        for size in (2, 4):
            assert plan.way_of(D, size) == plan.TMA
            assert plan.layout(lens, H or 1, D, size, False) == want, (lens, D, size)
    # more tiles than are on their way at once (3): stages are used again
    for (_, T, _, _), (width, _) in gpu.WIDE.items():
        assert T > 4 * 4096 // width


def test_the_gpu_tests_reach_every_layout():
    def marked(test):   # the shapes of a parametrised test
        return next(m.args[1] for m in test.pytestmark if m.args[0] in ("B,T,D", "T,D"))

    shapes = [(2, T, 36) for T in test_gpu_scan.LENGTHS] + gpu.NARROW
    shapes += [(3, 150, D) for D in test_gpu_scan.WIDTHS]
    shapes += marked(test_gpu_scan.test_shapes_of_few_and_many_sequences)
    shapes += marked(test_gpu_scan.test_many_short_sequences)
    seen = {(plan.way_of(D, size), size, False, want) for (_, _, D, size), want in gpu.WIDE.items()}
    for B, T, D in shapes:
        for size in (2, 4):
            for backward in (False, True):
                seen.add((plan.way_of(D, size), size, backward,
                          plan.layout([T], B, D, size, backward)))
    for way, size in ((plan.TMA, 2), (plan.TMA, 4), (plan.FOUR, 2), (plan.ONE, 2), (plan.ONE, 4)):
        for backward in (False, True):
            for choice in ["walk"] + plan.choices():
                if choice == "walk" or choice[0] == 32 or (way == plan.TMA and not backward):
                    assert (way, size, backward, choice) in seen
