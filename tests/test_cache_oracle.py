"""CPU: the reference of the quantized cache is pinned to something other than
itself: torch's own e4m3 numbers and rounding, hand-worked blocks, and planted
mistakes that its pins notice."""

import math

import numpy as np
import torch

from oracle import cache_oracle as co


def test_e4m3_numbers_are_torchs():
    want = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    got = co.e4m3_numbers()
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(got[~np.isnan(got)], want[~np.isnan(want)])


def test_nearest_is_torchs_rounding():
    rng = np.random.default_rng(0)
    table = np.sort(co.e4m3_numbers()[:127])
    mids = (table[1:] + table[:-1]) / 2
    x = np.concatenate([table, mids, np.nextafter(mids, 0), np.nextafter(mids, 9e9), rng.normal(0, 100, 2000),
                        rng.normal(0, 0.01, 500)])
    x = np.float32(np.clip(np.concatenate([x, -x]), -448, 448))
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal([co.nearest(float(v), "e4m3") for v in x], want)
    assert [co.nearest(v, "int8") for v in (0.5, 1.5, -2.5, 126.5, 127.5, 1e9, -1e9)] == [0, 2, -2, 126, 127, 127, -127]
    assert co.nearest(1e9, "e4m3") == 448 and math.isnan(co.nearest(math.nan, "e4m3")) and co.nearest(math.nan, "int8") == 0


def test_least_exponent():
    for fmt, most in co.LARGEST.items():
        for e in (-126, -7, 0, 5, co.TOP[fmt]):
            assert co.least_exponent(math.ldexp(most, e), fmt) == e
            assert co.least_exponent(math.ldexp(most, e) * (1 + 2 ** -23), fmt) == min(e + 1, co.TOP[fmt])
        assert co.least_exponent(0.0, fmt) == co.LOW and co.least_exponent(1e300, fmt) == co.TOP[fmt]


def _empty(fmt="int8", pages=2, heads=1, page=4, d=2, blocks=2):
    return dict(k=np.zeros((pages, heads, page, d)), v=np.zeros((pages, heads, page, d)),
                k_exp=np.full((pages, heads, blocks), 9), v_exp=np.full((pages, heads, blocks), 9), fmt=fmt)


def test_store_by_hand():
    c = _empty()
    x = np.array([[[100.0, -3.0]], [[1.0, 0.5]], [[508.0, 2.5]]])
    co.store(c, x[:1], x[:1], [4])          # page 1, row 0: exponent 0
    assert c["k_exp"][1, 0].tolist() == [0, 9] and c["k"][1, 0, 0].tolist() == [100, -3]
    co.store(c, x[2:], x[2:], [5])          # 508 = 127 * 4: exponent 2; the first row is rounded again
    assert c["k_exp"][1, 0].tolist() == [2, 9] and c["k"][1, 0, :2].tolist() == [[25, -1], [127, 1]]
    assert co.values(c, "k")[1, 0, :2].tolist() == [[100, -4], [508, 4]]
    co.store(c, x[1:2], x[1:2], [4])        # a sequence's first token again: the block starts anew
    assert c["v_exp"][1, 0].tolist() == [-6, 9] and c["v"][1, 0, 0].tolist() == [64, 32]
    assert not c["k"][0].any() and c["k_exp"][0].tolist() == [[9, 9]]


def test_keep_by_hand():
    c = _empty(page=4, blocks=2, pages=2)
    c["k"][1, 0] = [[8, 4], [1, 2], [100, 50], [7, 3]]   # page 1 is first: positions 0..3
    c["k_exp"][1, 0] = [0, 2]
    c["k_exp"][0, 0] = [1, 5]
    c["k"][0, 0] = [[6, 2], [9, 9], [0, 0], [0, 0]]       # positions 4..7
    table = np.array([[1, 0]])
    # context 1; nodes 1 (position 2, exponent 2) and 3 (position 4, exponent 1) move to 1 and 2
    co.keep(c, table, [1], np.array([[1, 3]]), [2])
    assert c["k_exp"][1, 0].tolist() == [2, 1]            # the first block grows for the row from the second
    assert c["k"][1, 0, :3].tolist() == [[2, 1], [100, 50], [6, 2]]


def test_pool_by_hand():
    refs, table = np.array([1, 0, 2, 0, 0]), np.array([[2, 0, -1], [2, -1, -1], [-1, -1, -1]])
    assert co.reserve(refs, table, [9, 4, 5], 4) == 0
    assert table.tolist() == [[2, 0, 1], [2, -1, -1], [3, 4, -1]] and refs.tolist() == [1, 1, 2, 1, 1]
    co.release(refs, table, [2, 2], None, 4)
    to = np.full((1, 3), 7)
    assert co.fork(refs, table, to, [0], [0], [6], 4) == ([(0, 3)], 0)
    assert to.tolist() == [[2, 3, -1]] and refs.tolist() == [1, 1, 3, 1, 0]
    co.release(refs, table, [0], [4], 4)
    assert table[0].tolist() == [2, -1, -1] and refs.tolist() == [0, 0, 3, 1, 0]
    both = np.concatenate([table, to])
    assert co.compact(refs, both) == (2, [(2, 0), (3, 1)]) and both.tolist() == [[0, -1, -1], [0, -1, -1], [-1] * 3, [0, 1, -1]]


def test_planted_mistakes_are_seen():
    """Each pin above fails for the mistake that it is there for."""
    x = np.array([[[100.0, -3.0]], [[508.0, 2.5]]])
    good, bad = _empty(), _empty()
    for c, old in ((good, False), (bad, True)):
        co.store(c, x[:1], x[:1], [4])
        if old:
            c["k_exp"][1, 0, 0] = -3   # an exponent that the bytes were not written under
        co.store(c, x[1:], x[1:], [5])
    assert not np.array_equal(good["k"], bad["k"])
    assert co.nearest(2.5, "int8") != round(2.5 + 1e-9)                 # ties away from zero
    assert co.least_exponent(449.0, "e4m3") == 1 and math.ceil(math.log2(449.0 / 512)) == 0  # the type's power for its number
