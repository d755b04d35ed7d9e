"""CPU: the fp64 reference of the attention operators is pinned to properties
and second formulations that are not its own code."""

import math

import numpy as np
import pytest
import torch

from oracle import attention_oracle as ao


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotation_keeps_lengths_and_depends_on_distance_alone(layout):
    rng = np.random.default_rng(0)
    f = 10000.0 ** (-np.arange(8) / 8)
    a = ao.rope_angles(np.arange(64), f)
    table = np.concatenate([np.cos(a), np.sin(a)], 1)
    q, k = rng.normal(size=(1, 1, 24)), rng.normal(size=(1, 1, 24))
    at = lambda x, p: ao.rotate_heads(x, table, [p], layout)[0][0, 0]
    assert math.isclose(np.linalg.norm(at(q, 17)), np.linalg.norm(q), rel_tol=1e-12)
    assert np.array_equal(at(q, 9)[16:], q[0, 0, 16:])  # the rest of the head
    near = [at(q, p + 5) @ at(k, p) for p in (0, 11, 58)]
    assert np.allclose(near, near[0], rtol=1e-11)
    assert not math.isclose(at(q, 6) @ at(k, 0), near[0], rel_tol=1e-3)
    # a complex product, pair by pair
    z = (q[0, 0, :8] + 1j * q[0, 0, 8:16]) if layout == "half" else (q[0, 0, 0:16:2] + 1j * q[0, 0, 1:16:2])
    z = z * np.exp(1j * 17 * f)
    got = at(q, 17)
    got = (got[:8] + 1j * got[8:16]) if layout == "half" else (got[0:16:2] + 1j * got[1:16:2])
    assert np.allclose(got, z, rtol=1e-12)


def test_norm_gives_unit_mean_square():
    x = np.random.default_rng(1).normal(size=(3, 2, 40)) * 7
    assert np.allclose(np.mean(ao.norm_heads(x, None, 0.0) ** 2, -1), 1.0, rtol=1e-12)


def test_ancestors_are_the_closure_of_the_parents():
    rng = np.random.default_rng(2)
    parents = [int(rng.integers(-1, j)) if j else -1 for j in range(30)]
    step = np.eye(30, dtype=int)
    for j, p in enumerate(parents):
        if p >= 0:
            step[j, p] = 1
    assert np.array_equal(ao.ancestors(parents), np.linalg.matrix_power(step, 30) > 0)
    assert np.array_equal(ao.ancestors(list(range(-1, 9))), np.tril(np.ones((10, 10), bool)))


def test_attention_against_a_library_softmax():
    rng = np.random.default_rng(3)
    page, hk, hq, d, ctx, n = 4, 2, 6, 8, 9, 3
    k, v = rng.normal(size=(5, hk, page, d)), rng.normal(size=(5, hk, page, d))
    q = rng.normal(size=(n, hq, d))
    table = np.array([[4, 0, 3, 1]])
    out, lse, _, _ = ao.attend(q, k, v, table, [ctx], [0, n], [np.tril(np.ones((n, n), bool))], 0.3)
    kk, vv = (np.concatenate([c[p] for p in table[0]], 1)[:, :ctx + n] for c in (k, v))
    t = lambda x: torch.from_numpy(np.ascontiguousarray(x))
    bias = torch.zeros(n, ctx + n, dtype=torch.float64)
    bias[:, ctx:].masked_fill_(~torch.ones(n, n).tril().bool(), -math.inf)
    for h in range(hq):
        s = 0.3 * t(q[:, h]) @ t(kk[h // 3]).T + bias
        assert np.allclose(out[:, h], torch.softmax(s, -1) @ t(vv[h // 3]), rtol=1e-12)
        assert np.allclose(lse[:, h], torch.logsumexp(s, -1), rtol=1e-12)


def test_kept_rows_are_those_of_the_path():
    page = 3
    cache = np.arange(6 * page, dtype=float).reshape(6, 1, page, 1)
    table = np.array([[2, 5, 0, 1]])
    want = cache.copy()
    flat = lambda c, p: c[table[0, p // page], 0, p % page, 0]
    ao.keep(cache, table, [2], np.array([[0, 3, 4, 7]]), [4])
    assert [flat(cache, 2 + j) for j in range(4)] == [flat(want, 2 + j) for j in (0, 3, 4, 7)]
    assert [flat(cache, p) for p in (0, 1, 6, 7, 8, 9)] == [flat(want, p) for p in (0, 1, 6, 7, 8, 9)]
