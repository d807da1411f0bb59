"""Pins of the dropout oracle (oracle/dropout.py): the generator's published known
answers, the keep rate and its independence, and central differences of the linear."""
import numpy as np
import pytest

from oracle import dropout as od


def test_known_answers():
    # the authors' known answers of the 10-round form: all zeros, all ones
    assert od.philox4x32([0] * 4, [0] * 2, 10) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    f = 0xFFFFFFFF
    assert od.philox4x32([f] * 4, [f] * 2, 10) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]


def test_bits_of_an_element():
    seed, offset = 0x0123456789ABCDEF, 2 ** 64 - 3          # the counter wraps within the range
    for p in (0.25, 0.5):
        k = od.keep(seed, offset, 61, p)
        for e in range(61):
            c = (offset + e // 8) % 2 ** 64
            w = od.philox4x32([c & 0xFFFFFFFF, c >> 32, 0, 0], [seed & 0xFFFFFFFF, seed >> 32], 7)
            assert k[e] == ((w[e % 8 // 2] >> (16 * (e % 2)) & 0xFFFF) >= od.threshold(p))


@pytest.mark.parametrize("p", [0.0, 0.05, 0.5, 0.9])
def test_keep_rate(p):
    n = 1 << 18
    k = od.keep(12345, 7, n, p)
    q = od.threshold(p) / 65536
    assert abs(k.mean() - (1 - q)) <= 5 * np.sqrt(q * (1 - q) / n)
    if 0 < p:
        c = k - k.mean()
        for lag in (1, 2, 7, 8, 64):                        # neighbours do not follow each other
            assert abs(np.mean(c[lag:] * c[:-lag])) <= 5 * q * (1 - q) / np.sqrt(n)
        other = od.keep(12345, 7 + n // 8, n, p)            # the next offset: other decisions
        assert abs(np.mean((other - other.mean()) * c)) <= 5 * q * (1 - q) / np.sqrt(n)


def test_linear_by_differences():
    rng = np.random.default_rng(5)
    m, h, o, r, s, p = 4, 6, 5, 2, 0.7, 0.3
    W, X, L1, L2 = (rng.standard_normal(x) for x in ((h, o), (m, h), (h, r), (r, o)))
    dY, kept = rng.standard_normal((m, o)), od.keep(1, 2, m * h, p).reshape(m, h)
    _, T = od.linear_fwd_dropout(W, X, L1, L2, s, p, kept)
    got = od.linear_bwd_dropout(W, X, T, dY, L1, L2, s, p, kept)
    args = [X, L1, L2]
    for i in range(3):
        for at in np.ndindex(args[i].shape):
            v = []
            for e in (1e-6, -1e-6):
                b = [a.copy() for a in args]
                b[i][at] += e
                v.append(np.sum(od.linear_fwd_dropout(W, *b, s, p, kept)[0] * dY))
            assert abs((v[0] - v[1]) / 2e-6 - got[i][at]) < 1e-7
