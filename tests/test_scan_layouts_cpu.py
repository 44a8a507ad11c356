"""The rule that lays out a scan's work chooses each of its layouts for some call."""

from __future__ import annotations

import random

import scan_layouts as plan


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
