"""The norms where a workgroup walks several rows: the next row's prefetch, the sums' LDS
rows taken in turn and the column sums carried over rows, at every number of pieces per
thread, whole and odd widths.  Bounds as in test_gpu_norm.py."""
import pytest
import torch

from test_gpu_norm import BF, F32, check_bwd, check_fwd, dev, problem

import bit_quantized_fine_nf4_amd as nf4

pytestmark = pytest.mark.gpu


def rows_per_workgroup(m, h, most):
    """(rows that the busiest workgroup walks, pieces per thread): the launch rule of the norms."""
    shift = 7 if h % 8 and h > 8 and (h + 14) // 8 <= 2048 else 0
    pieces = (h + shift + 7) // 8
    depth = 1 if pieces <= most else 2 if pieces <= 2 * most else 4
    threads = -(-pieces // (64 * depth)) * 64
    grid = min(m, 256 * ((512 if depth == 4 else 1024) // threads))
    return -(-m // grid), depth


#        rows, width, pieces per thread forward and backward
SHAPES = [(9000, 7, 1, 1), (9000, 40, 1, 1), (9000, 41, 1, 1), (4200, 2048, 1, 1), (600, 4096, 1, 1), (600, 8192, 2, 1),
          (1300, 8200, 4, 2), (600, 16384, 4, 2), (600, 8193, 4, 2), (600, 16381, 4, 2), (1300, 5003, 2, 1)]


@pytest.mark.parametrize("rt", [BF, F32])
@pytest.mark.parametrize("post,gate", [(False, False), (True, True)])
@pytest.mark.parametrize("m,h,df,db", SHAPES)
def test_parity(m, h, df, db, post, gate, rt):
    for most, depth in ((512, df), (1024, db)):
        rows, d = rows_per_workgroup(m, h, most)
        assert rows >= 2 and d == depth
    print(f"norm rows m={m} h={h} post={post} gate={gate} {rt}", flush=True)
    alpha, eps = 0.5, 1e-5
    d = problem(m, h, rt, post, gate)
    w = dict(w_pre=dev(d["w_pre"]), w_post=dev(d["w_post"]), gate=dev(d["gate"]), alpha=alpha)
    check_fwd(d, alpha, eps, nf4.qlora_norm_fwd(dev(d["R"]), dev(d["Y"]), eps=eps, **w))
    R, Y = dev(d["R"]), dev(d["Y"])
    p = torch.rsqrt(R.float().square().mean(1) + eps)
    q = torch.rsqrt(Y.float().square().mean(1) + eps) if post else None
    out = nf4.qlora_norm_bwd(dev(d["dN"]), dev(d["dR_out"]), R, Y, p, q, weight_grads=True, **w)
    check_bwd(d, (p, q), alpha, out, m)
    frozen = nf4.qlora_norm_bwd(dev(d["dN"]), dev(d["dR_out"]), R, Y, p, q, **w)
    assert torch.equal(frozen[0], out[0]) and torch.equal(frozen[1], out[1])


@pytest.mark.parametrize("rt", [BF, F32])
@pytest.mark.parametrize("norms", [True, False])
@pytest.mark.parametrize("m,h", [(600, 8192), (1300, 5003), (600, 16384), (600, 8193), (9000, 41)])
def test_in_place_stream(m, h, norms, rt):
    """Rows prefetched from the buffer that the rows before them are stored into.  Without
    norms no barrier stands between a row's loads and its stores."""
    d = problem(m, h, rt, norms, True, pre=norms)
    w = dict(w_pre=dev(d["w_pre"]), w_post=dev(d["w_post"]), gate=dev(d["gate"]), alpha=0.5)
    Y = dev(d["Y"])
    a = nf4.qlora_norm_fwd(dev(d["R"]), Y, **w)
    R = dev(d["R"])
    b = nf4.qlora_norm_fwd(R, Y, R_out=R, **w)
    assert b[0] is R and all(torch.equal(x, y) for x, y in zip(a, b) if x is not None)
    dN = dev(d["dN"]) if norms else None
    x = nf4.qlora_norm_bwd(dN, dev(d["dR_out"]), a[0], Y, a[2], a[3], weight_grads=True, **w)
    g = dev(d["dR_out"])
    y = nf4.qlora_norm_bwd(dN, g, a[0], Y, a[2], a[3], dR=g, weight_grads=True, **w)
    assert y[0] is g and all(torch.equal(s, t) for s, t in zip(x, y) if s is not None)
