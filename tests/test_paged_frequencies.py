"""Frequencies scaled by parts: the ramp's middle, and another program's ramp passed in.  No GPU needed."""

import math

import pytest

from speculative_decoding_draft_kv_gb300 import paged as P


@pytest.mark.parametrize("rotary,theta,factor,length,fast,slow", [
    (128, 1e6, 4.0, 4096, 32.0, 1.0), (64, 1e4, 8.0, 2048, 32.0, 1.0), (128, 5e5, 16.0, 8192, 24.0, 2.0)])
def test_the_ramp_is_linear_in_the_number_of_turns(rotary, theta, factor, length, fast, slow):
    got, magnitude = P.rope_frequencies(rotary, theta, "yarn", factor, length, fast, slow)
    assert abs(magnitude - (0.1 * math.log(factor) + 1)) < 1e-15
    between = 0
    for i, f in enumerate(got):
        plain = theta ** (-2 * i / rotary)
        turns = length * plain / (2 * math.pi)
        # what is kept of the plain frequency, beside the slowed one: 0 at slow turns, 1 at fast
        kept = (f - plain / factor) / (plain - plain / factor)
        assert abs(kept - min(1.0, max(0.0, (turns - slow) / (fast - slow)))) < 1e-9
        between += 0.0 < kept < 1.0
    assert between >= 5


def test_a_ramp_over_the_pairs_comes_as_frequencies():
    r, theta, factor, length = 128, 1e6, 4.0, 4096
    plain = [theta ** (-2 * i / r) for i in range(r // 2)]

    def border(turns):                         # the index of the pair that turns so often
        return r * math.log(length / (2 * math.pi * turns)) / (2 * math.log(theta))

    low, high = math.floor(border(32.0)), math.ceil(border(1.0))
    keep = [1 - min(1.0, max(0.0, (i - low) / (high - low))) for i in range(r // 2)]
    mine = [(1 - g) * f / factor + g * f for g, f in zip(keep, plain)]
    other, _ = P.rope_frequencies(r, theta, "yarn", factor, length)
    assert max(abs(a / b - 1) for a, b in zip(mine, other)) > 0.05      # not the same thing
    rope = P.PagedRope(r, inv_freq=mine, magnitude=1.25)
    assert rope.inv_freq == mine and rope.magnitude == 1.25 and rope.args.magnitude == 1.25
    for f, t in zip(mine, rope.args.turns):
        assert abs(t / 2.0 ** 64 - f / (2 * math.pi) % 1) < 1e-15
