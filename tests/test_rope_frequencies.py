"""CPU: the scalings by parts of the rotary frequencies, value by value between
their ends, from second formulations: turns in the original context found by
bisection or from wave lengths, in place of the library's logarithm and turns."""

import math

import pytest

import gemm_lora_shrink_amd as glsa


def _pair_of_turns(turns, rot, base, L):
    """The real-valued pair that makes `turns` turns in L positions, by bisection."""
    lo, hi = -10.0 * rot, 10.0 * rot
    for _ in range(200):
        mid = (lo + hi) / 2
        if L * base ** (-2.0 * mid / rot) / (2 * math.pi) > turns:
            lo = mid
        else:
            hi = mid
    return (lo + hi) / 2


@pytest.mark.parametrize("rot,base,s,L,low,high", [(128, 10000.0, 4.0, 4096, 0, 0), (64, 10000.0, 16.0, 4096, 0, 0),
                                                   (128, 500000.0, 8.0, 8192, 2.0, 20.0), (20, 10000.0, 2.0, 512, 0, 0),
                                                   (128, 10000.0, 40.0, 64, 0, 0), (8, 1.5, 4.0, 4096, 0, 0)])
def test_yarn_between_the_ends(rot, base, s, L, low, high):
    scaling = dict(type="yarn", factor=s, original_max_position=L)
    if high:
        scaling.update(low=low, high=high)
    got, magnitude = glsa.rope_frequencies(rot, base, scaling)
    first = max(math.floor(_pair_of_turns(high or 32.0, rot, base, L)), 0)
    last = min(math.ceil(_pair_of_turns(low or 1.0, rot, base, L)), rot - 1)
    between = 0
    for i, f in enumerate(got):
        plain = base ** (-2.0 * i / rot)
        if i <= first:
            kept = 1.0
        elif i >= last:
            kept = 0.0
        else:
            kept = (last - i) / (last - first)
            between += 1
        want = math.exp(math.log(plain)) * (kept + (1.0 - kept) / s)
        assert math.isclose(f, want, rel_tol=1e-12), i
    assert math.isclose(magnitude, 1.0 + math.log(s) / 10.0, rel_tol=1e-14)
    assert between > 0 or last - first <= 1 or last <= 0 or first >= rot // 2


@pytest.mark.parametrize("rot,base,s,L,low,high", [(128, 500000.0, 8.0, 8192, 0, 0), (64, 500000.0, 32.0, 8192, 0, 0),
                                                   (128, 10000.0, 4.0, 2048, 1.5, 9.0)])
def test_llama3_between_the_ends(rot, base, s, L, low, high):
    scaling = dict(type="llama3", factor=s, original_max_position=L)
    if high:
        scaling.update(low=low, high=high)
    got, magnitude = glsa.rope_frequencies(rot, base, scaling)
    low, high, between = low or 1.0, high or 4.0, 0
    for i, f in enumerate(got):
        wave = 2 * math.pi * base ** (2.0 * i / rot)  # positions of a turn
        if wave <= L / high:
            want = 2 * math.pi / wave
        elif wave >= L / low:
            want = 2 * math.pi / (wave * s)
        else:
            m = (L / wave - low) / (high - low)
            want = 2 * math.pi / wave * ((1 - m) / s + m)
            between += 1
        assert math.isclose(f, want, rel_tol=1e-12), i
    assert between >= 3 and magnitude == 1.0
