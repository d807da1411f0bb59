"""The head's products where a persistent workgroup takes several units: a unit's last
stages copy the next one's first, at numbers of stages that leave the rings in every
position, with splits of unlike length.  Bounds as in test_gpu_loss.py."""
import pytest
import torch

from test_gpu_loss import DEV, compare, problem, run

pytestmark = pytest.mark.gpu

GROUPS = 256  # persistent workgroups


def cdiv(a, b):
    return -(-a // b)


def head_splits(n, h, piece, rows):
    """Splits of dH's sum over the vocabulary: the rule of the launch."""
    tiles, blocks = cdiv(n, 256) * cdiv(h, 256), cdiv(piece, 64)
    best = cost = 0
    for s in range(1, 17):
        if s > 1 and (blocks < 8 * s or s * n > rows):
            break
        c = cdiv(tiles * s, 256) * 10000 // s + 400 * s * tiles // 256
        if s == 1 or c < cost:
            best, cost = s, c
    return best


#        tokens, h, words: h / 64 is 64, 65, 66 (every remainder by the three pairs of slots)
SHAPES = [(2050, 4160, 8001), (2050, 4096, 10241), (2050, 4224, 7700), (2100, 3904, 9000), (4100, 4160, 1700)]


@pytest.mark.parametrize("skip", ["none", "some"])
@pytest.mark.parametrize("M,h,V", SHAPES)
def test_several_units_per_workgroup(M, h, V, skip):
    splits = head_splits(M, h, V, 8192)
    units = dict(logits=cdiv(M, 256) * cdiv(V, 256), dh=cdiv(M, 256) * cdiv(h, 256) * splits,
                 dw=cdiv(V, 256) * cdiv(h, 256))
    print(f"loss units M={M} h={h} V={V} {skip}: {units}, {splits} splits", flush=True)
    if V > 2000:
        assert min(units.values()) > GROUPS and splits > 1
    else:
        assert units["dh"] > GROUPS and splits == 1
    t = [x.to(DEV) for x in problem(M, h, V, skip)]
    got = run(*t)
    compare(got, *t)
    again = run(*t)
    assert all(torch.equal(got[k], again[k]) for k in got)


def test_the_stage_counts_differ():
    """Of the shapes above: dH's splits are of unlike length somewhere, and the products'
    double stages leave every remainder by 3 (pairs of W's slots) and several by 5."""
    blocks = set()
    for M, h, V in SHAPES:
        n, s = cdiv(V, 64), head_splits(M, h, V, 8192)
        blocks |= {n * (k + 1) // s - n * k // s for k in range(s)}
    assert len({b % 5 for b in blocks}) >= 3
    assert {h // 64 % 3 for _, h, _ in SHAPES} == {0, 1, 2}
    assert any(cdiv(V, 64) % head_splits(M, h, V, 8192) for M, h, V in SHAPES)
