"""The rotation's table against 60-digit arithmetic: each fraction of a turn is right
to its 64 bits, so that the angle of the farthest position is right to 2^-32 turns."""

import decimal
import math
from decimal import Decimal as X

import pytest

from dynamic_hierarchical_sparse_b200 import api, build, workloads as W

decimal.getcontext().prec = 60
PI = X("3.14159265358979323846264338327950288419716939937510582097494459")
TURN = 2 ** 64


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def _frequencies(rotary, base, sc):
    f = [(-(X(2 * i) / X(rotary)) * X(base).ln()).exp() for i in range(rotary // 2)]
    if sc is None:
        return f
    by = X(sc.factor)
    if sc.kind == "linear":
        return [x / by for x in f]
    if sc.kind == "llama3":
        lo, hi = X(sc.low_freq_factor), X(sc.high_freq_factor)
        keep = [min(max((X(sc.original_len) * x / (2 * PI) - lo) / (hi - lo), X(0)), X(1)) for x in f]
        return [k * x + (1 - k) * x / by for k, x in zip(keep, f)]
    index = lambda turns: rotary * math.log(sc.original_len / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
    low, high = max(math.floor(index(sc.beta_fast)), 0), min(math.ceil(index(sc.beta_slow)), rotary - 1)
    high = X(high) + (X(0.001) if high == low else 0)
    share = [min(max((X(i) - low) / (high - low), X(0)), X(1)) for i in range(len(f))]
    return [s * x / by + (1 - s) * x for s, x in zip(share, f)]


def _off(table, freqs):
    """The largest distance of the table's fractions from the true ones, in units of 2^-64 turns."""
    worst = X(0)
    for got, f in zip(table, freqs):
        d = (X(int(got)) - f / (2 * PI) * TURN) % TURN
        worst = max(worst, min(abs(d), TURN - abs(d)))
    return worst


@pytest.mark.parametrize("scaling", [None, W.RopeScaling("linear", 3.0), W.RopeScaling("llama3", 8.0, 8192.0),
                                     W.RopeScaling("yarn", 16.0, 4096.0), W.RopeScaling("yarn", 7.0, 300.0)],
                         ids=lambda s: "plain" if s is None else s.kind)
@pytest.mark.parametrize("base", [10000.0, 500000.0, 1000003.7])
@pytest.mark.parametrize("rotary", [2, 64, 90, 128, 256])
def test_fractions_of_a_turn(rotary, base, scaling):
    r = api.Rope(rotary, base, scaling=scaling)
    # of 2^-64 turns: half from the rounding; and a frequency of up to 1 (0.16 turns), worked out in a few roundings
    # of 2^-64 of itself, of which the power has as many as the logarithm of its result (f ln(1 / f) is below 0.37)
    assert _off(r.c.turns[:rotary // 2], _frequencies(rotary, base, scaling)) <= 2


def test_given_frequencies():
    freq = [1.0, 0.1, 3.25, -0.7, 100.0, 1e-9, 0.0, 6.283185307179586]
    r = api.Rope(16, inv_freq=freq)
    for got, f in zip(r.c.turns, freq):
        assert _off([got], [X(f)]) <= X(0.5) + X(abs(f)), f


def test_angles_of_far_positions():
    """The angle as the kernel takes it, position times fraction modulo a turn, from the top 32 bits."""
    r, f = api.Rope(128, 500000.0), _frequencies(128, 500000.0, None)
    for p in (1, 131071, 10 ** 7, 2 ** 31 - 1, -2 ** 31):
        for got, x in zip(r.c.turns, f):
            top = (p * int(got) % TURN) >> 32
            d = (X(top) / 2 ** 32 - X(p) * x / (2 * PI)) % 1
            assert min(d, 1 - d) <= X(2) ** -32 + abs(p) * X(2) ** -63
