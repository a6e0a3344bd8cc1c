"""Frequencies by parts where the original length is large: no pair then turns
as little as beta_slow times, and none may be divided by the whole factor."""
import math

import pytest

import gated_linear_recurrence_history_amd as gs


def by_parts(rot, base, factor, length, fast=32.0, slow=1.0):
    """The rule in 64 bits: between the pairs that turn `fast` and `slow` times
    over `length` tokens, rounded outwards, the share of the divided frequency
    grows evenly."""
    def index(turns):  # length * base^(-2 i / rot) = 2 pi turns
        return rot / 2 * math.log(length / (2 * math.pi * turns), base)
    low, high = max(math.floor(index(fast)), 0), math.ceil(index(slow))
    out = []
    for i in range(rot // 2):
        share = min(max((i - low) / (high - low), 0.0), 1.0)
        f = base ** (-2 * i / rot)
        out.append((1 - share) * f + share * f / factor)
    return out


@pytest.mark.parametrize("rot,base,factor,length", [
    (64, 10000.0, 4.0, 131072),    # the slowest pair turns 2.8 times
    (64, 10000.0, 4.0, 2048),
    (128, 10000.0, 8.0, 1 << 20),
    (32, 10000.0, 2.0, 65536),     # 1.8 times
    (128, 500000.0, 16.0, 8192),
])
def test_frequencies_by_parts_of_any_length(rot, base, factor, length):
    f, _ = gs.rotary_frequencies(rot, base, "parts", factor, length)
    # rounded once to float32 (2^-24), some roundings in 64 bits before it
    for x, want in zip(f.tolist(), by_parts(rot, base, factor, length)):
        assert abs(x - want) <= 2.0 ** -24 * want * (1 + 1e-6)


def test_a_pair_that_turns_often_enough_is_not_divided_whole():
    f, _ = gs.rotary_frequencies(64, 10000.0, "parts", 4.0, 131072)
    slowest = 10000.0 ** (-62 / 64)
    assert 131072 * slowest / (2 * math.pi) > 2.7
    assert float(f[-1]) > slowest / 4 * 1.05
