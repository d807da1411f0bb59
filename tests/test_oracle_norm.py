"""Pins of the norm oracle (oracle/norm.py): closed forms and central differences of
the forward against the backward, for every combination of its optional parts."""
import itertools

import numpy as np
import pytest

import oracle


def test_closed_forms():
    r = np.array([[3.0, 4.0], [0.0, 0.0]])
    ro, n, p, q = oracle.norm_fwd(r, None, np.array([1.0, 2.0]), None, None, 1.0, 1e-30)
    assert q is None and np.array_equal(ro, r)
    assert np.allclose(n[0], [3 / np.sqrt(12.5), 8 / np.sqrt(12.5)], rtol=1e-15)
    assert np.array_equal(n[1], [0.0, 0.0])              # a zero row stays zero, whatever eps
    y = np.array([[1.0, -1.0], [2.0, 0.0]])
    ro, n, p, q = oracle.norm_fwd(r, y, None, np.ones(2), np.array([0.5, 2.0]), 4.0, 1e-30)
    assert n is None and p is None
    assert np.allclose(ro[0], [3 + 2.0, 4 - 8.0], rtol=1e-15)
    assert np.allclose(ro[1], [4 * 0.5 * np.sqrt(2.0), 0.0], rtol=1e-15)


@pytest.mark.parametrize("pre,post,gate", itertools.product([True, False], repeat=3))
def test_backward_by_differences(pre, post, gate):
    rng = np.random.default_rng(1)
    m, h, alpha, eps = 3, 7, 0.7, 1e-3
    r, y = rng.standard_normal((m, h)), rng.standard_normal((m, h))
    w = {k: rng.standard_normal(h) + 1 for k in ("pre", "post", "gate")}
    dn, dro = rng.standard_normal((m, h)), rng.standard_normal((m, h))

    def value(r, y, wp, wq, g):
        ro, n, _, _ = oracle.norm_fwd(r, y, wp if pre else None, wq if post else None, g if gate else None, alpha, eps)
        return np.sum(ro * dro) + (np.sum(n * dn) if pre else 0.0)

    args = [r, y, w["pre"], w["post"], w["gate"]]
    ro, n, p, q = oracle.norm_fwd(r, y, w["pre"] if pre else None, w["post"] if post else None,
                                  w["gate"] if gate else None, alpha, eps)
    got = oracle.norm_bwd(dn if pre else None, dro, ro, y, p, q, w["pre"] if pre else None,
                          w["post"] if post else None, w["gate"] if gate else None, alpha)
    for i, used in enumerate((True, True, pre, post, gate)):
        if not used:
            assert got[i] is None
            continue
        diff = np.empty_like(args[i])
        for at in np.ndindex(diff.shape):
            lo, hi = [a.copy() for a in args], [a.copy() for a in args]
            lo[i][at] -= 1e-5
            hi[i][at] += 1e-5
            diff[at] = (value(*hi) - value(*lo)) / 2e-5
        assert np.max(np.abs(diff - got[i])) < 1e-7, i
