"""GPU parity of the norms with residual update (qlora_norm_fwd, qlora_norm_bwd)
against the float64 oracle (oracle/norm.py).

Bounds, with u = 2^-24 (a float32 rounding) and H the output's own half step (2^-8 of
the value for bf16, u for float32).  Each step of the chain rounds a few times: a sum
over a row takes at most 32 additions per thread, 6 between lanes and 16 between waves,
its root and reciprocal 3 more and halve the sum's error, the products around it at most
5: C = 64 roundings cover every chain.  They act on the magnitudes that enter:
  r     |R| + |alpha gate u|
  N     |r| rstd w, and the row's relative error of rstd: K = ||magnitude of r|| / ||r||
  dR    |dR_out| + rstd (|d| + |x| mean|d x|)
  dY    the same through the second norm, with the magnitude of du in place of du
  sums over M rows: M + C roundings of the sum of magnitudes."""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import bit_quantized_fine_nf4_amd as nf4  # noqa: E402

DEV = "cuda:0"
U = 2.0 ** -24
C = 64
BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F32: U}


def f64(t):
    return None if t is None else t.detach().cpu().to(torch.float64).numpy()


def check(name, got, ref, mag, factor=C):
    g = f64(got)
    bound = HALF[got.dtype] * np.abs(ref) + factor * U * mag
    bad = np.argwhere(~(np.abs(g - ref) <= bound))
    assert bad.size == 0, (name, len(bad), bad[:3], [(g[tuple(b)], ref[tuple(b)]) for b in bad[:3]])


def problem(m, h, rt, post, gate, pre=True, seed=0):
    g = torch.Generator().manual_seed(1000 * seed + 7 * m + h)
    n = lambda *s, std=1.0: torch.randn(*s, generator=g) * std
    d = dict(R=n(m, h, std=2.0).to(rt), Y=n(m, h).to(BF), dN=n(m, h).to(BF), dR_out=n(m, h).to(rt),
             w_pre=1 + n(h, std=0.2) if pre else None, w_post=1 + n(h, std=0.2) if post else None,
             gate=n(h) if gate else None)
    if m > 2:
        d["R"][1] = 0
        d["Y"][1] = 0      # an empty row: rstd is 1 / sqrt(eps) and everything stays finite
        d["Y"][2] = 0
    return d


def dev(t):
    return None if t is None else t.to(DEV)


def check_fwd(d, alpha, eps, got):
    R_out, N, p, q = got
    r, y, wp, wq, g = (f64(d[k]) for k in ("R", "Y", "w_pre", "w_post", "gate"))
    rr, rn, rp, rq = oracle.norm_fwd(r, y, wp, wq, g, alpha, eps)
    mag = np.abs(r)
    if y is not None:
        u = np.abs(y) if wq is None else np.abs(y * rq[:, None] * wq)
        mag = mag + np.abs(alpha * (1.0 if g is None else g)) * u
        check("R_out", R_out, rr, mag)
        if wq is not None:
            check("rstd_post", q, rq, rq)
    if wp is not None:
        h = r.shape[1]
        K = (np.linalg.norm(mag, axis=1) + np.sqrt(h * eps)) / np.sqrt(np.sum(rr ** 2, 1) + h * eps)
        check("rstd_pre", p, rp, rp * (1 + K))
        check("N", N, rn, (mag + np.abs(rr) * (1 + K)[:, None]) * rp[:, None] * np.abs(wp))


def through(mag_g, x, s):
    return s[:, None] * (mag_g + np.abs(x * s[:, None]) * np.mean(mag_g * np.abs(x * s[:, None]), 1, keepdims=True))


def check_bwd(d, stats, alpha, got, M):
    dR, dY, dwp, dwq, dg = got
    v = {k: f64(d[k]) for k in d}
    p, q = f64(stats[0]), f64(stats[1])
    ref = oracle.norm_bwd(v["dN"], v["dR_out"], v["R"], v["Y"], p, q, v["w_pre"], v["w_post"], v["gate"], alpha)
    mag = np.abs(v["dR_out"]) if v["dR_out"] is not None else 0.0
    if v["w_pre"] is not None:
        mag = mag + through(np.abs(v["dN"] * v["w_pre"]), v["R"], p)
    check("dR", dR, ref[0], mag)
    g = np.abs(alpha * (1.0 if v["gate"] is None else v["gate"]))
    if dY is not None:
        mdu = g * mag
        check("dY", dY, ref[1], mdu if v["w_post"] is None else through(mdu * np.abs(v["w_post"]), v["Y"], q), 2 * C)
    if dwp is not None:
        check("dw_pre", dwp, ref[2], np.sum(np.abs(v["dN"] * v["R"] * p[:, None]), 0), M + C)
    if dwq is not None:
        check("dw_post", dwq, ref[3], np.sum(g * mag * np.abs(v["Y"] * q[:, None]), 0), M + 2 * C)
    if dg is not None:
        u = v["Y"] if v["w_post"] is None else v["Y"] * q[:, None] * v["w_post"]
        check("dgate", dg, ref[4], np.sum(np.abs(alpha * mag * u), 0), M + 2 * C)


SHAPES = [(1, 1), (1, 8192), (3, 7), (2, 64), (5, 511), (4, 512), (4, 513), (300, 1000), (3, 2047), (2, 2056),
          (3, 4100), (7, 5003), (1100, 5003), (700, 4099), (3, 8191), (300, 8185), (2, 8193), (3, 16384), (2, 16381), (2500, 40)]


@pytest.mark.parametrize("rt", [BF, F32])
@pytest.mark.parametrize("post,gate", [(False, False), (True, True), (True, False), (False, True)])
@pytest.mark.parametrize("m,h", SHAPES)
def test_parity(m, h, post, gate, rt):
    print(f"norm m={m} h={h} post={post} gate={gate} {rt}", flush=True)
    alpha, eps = 0.5, 1e-5
    d = problem(m, h, rt, post, gate)
    w = dict(w_pre=dev(d["w_pre"]), w_post=dev(d["w_post"]), gate=dev(d["gate"]), alpha=alpha)
    got = nf4.qlora_norm_fwd(dev(d["R"]), dev(d["Y"]), eps=eps, **w)
    check_fwd(d, alpha, eps, got)
    # the backward of the stored stream
    R, Y = dev(d["R"]), dev(d["Y"])
    p = torch.rsqrt(R.float().square().mean(1) + eps)
    q = torch.rsqrt(Y.float().square().mean(1) + eps) if post else None
    out = nf4.qlora_norm_bwd(dev(d["dN"]), dev(d["dR_out"]), R, Y, p, q, weight_grads=True, **w)
    assert (out[3] is not None) == post and (out[4] is not None) == gate
    check_bwd(d, (p, q), alpha, out, m)
    frozen = nf4.qlora_norm_bwd(dev(d["dN"]), dev(d["dR_out"]), R, Y, p, q, **w)
    assert frozen[2] is frozen[3] is frozen[4] is None
    assert torch.equal(frozen[0], out[0]) and torch.equal(frozen[1], out[1])


@pytest.mark.parametrize("rt", [BF, F32])
def test_parts_left_out(rt):
    """No block output (the first norm), no norm after the update (the last block), and a
    backward without a residual gradient."""
    d = problem(6, 72, rt, False, False)
    first = nf4.qlora_norm_fwd(dev(d["R"]), w_pre=dev(d["w_pre"]), eps=1e-5)
    assert torch.equal(first[0].cpu(), d["R"])
    check_fwd(dict(d, Y=None), 1.0, 1e-5, first)
    last = nf4.qlora_norm_fwd(dev(d["R"]), dev(d["Y"]), alpha=0.5)
    assert last[1] is None and last[2] is None
    check_fwd(dict(d, w_pre=None), 0.5, 1e-5, last)
    R = dev(d["R"])
    p = torch.rsqrt(R.float().square().mean(1) + 1e-5)
    out = nf4.qlora_norm_bwd(dev(d["dN"]), None, R, rstd_pre=p, w_pre=dev(d["w_pre"]), block=False, weight_grads=True)
    assert out[1] is None
    check_bwd(dict(d, dR_out=None, Y=None), (p, None), 1.0, out, 6)
    out = nf4.qlora_norm_bwd(None, dev(d["dR_out"]), None, alpha=0.5)
    assert torch.equal(out[0].cpu(), d["dR_out"])
    check_bwd(dict(d, w_pre=None, dN=None), (None, None), 0.5, out, 6)


@pytest.mark.parametrize("rt", [BF, F32])
def test_in_place_stream(rt):
    d = problem(9, 1032, rt, True, True)
    w = dict(w_pre=dev(d["w_pre"]), w_post=dev(d["w_post"]), gate=dev(d["gate"]), alpha=0.5)
    a = nf4.qlora_norm_fwd(dev(d["R"]), dev(d["Y"]), **w)
    R = dev(d["R"])
    b = nf4.qlora_norm_fwd(R, dev(d["Y"]), R_out=R, **w)
    assert b[0] is R and all(torch.equal(x, y) for x, y in zip(a, b))
    x = nf4.qlora_norm_bwd(dev(d["dN"]), dev(d["dR_out"]), a[0], dev(d["Y"]), a[2], a[3], **w)
    g = dev(d["dR_out"])
    y = nf4.qlora_norm_bwd(dev(d["dN"]), g, a[0], dev(d["Y"]), a[2], a[3], dR=g, **w)
    assert y[0] is g and torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])


def test_neighbours_are_left_alone_and_repeats_agree():
    """Rows behind the last one and values behind an odd row's end stay as they were, and
    the sums come out the same every time."""
    m, h = 37, 1003
    d = problem(m, h, BF, True, True)
    w = dict(w_pre=dev(d["w_pre"]), w_post=dev(d["w_post"]), gate=dev(d["gate"]), alpha=0.5)
    guard = lambda n, t: torch.full((n + 64,), 7.0, dtype=t, device=DEV)
    big = {k: guard(m * h, BF) for k in ("R_out", "N", "dR", "dY")}
    view = {k: t[: m * h].view(m, h) for k, t in big.items()}
    sums = {k: guard(h, F32) for k in ("dw_pre", "dw_post", "dgate")}
    sv = {k: t[:h] for k, t in sums.items()}
    _, _, p, q = nf4.qlora_norm_fwd(dev(d["R"]), dev(d["Y"]), R_out=view["R_out"], N=view["N"], **w)
    first = None
    for _ in range(3):
        out = nf4.qlora_norm_bwd(dev(d["dN"]), dev(d["dR_out"]), view["R_out"], dev(d["Y"]), p, q, dR=view["dR"],
                                 dY=view["dY"], **sv, **w)
        now = [t.clone() for t in out]
        first = first or now
        assert all(torch.equal(a, b) for a, b in zip(first, now))
    for t, n in [(t, m * h) for t in big.values()] + [(t, h) for t in sums.values()]:
        assert torch.all(t[n:] == 7.0)


def test_captured_step():
    """Forward and backward in one captured graph, replayed on new inputs between eager
    calls, on a stream that is not the default one."""
    m, h = 65, 520
    d = problem(m, h, BF, True, True)
    w = dict(w_pre=dev(d["w_pre"]), w_post=dev(d["w_post"]), gate=dev(d["gate"]), alpha=0.5)
    R, Y, dN, dRo = (dev(d[k]) for k in ("R", "Y", "dN", "dR_out"))

    def step():
        ro, n, p, q = nf4.qlora_norm_fwd(R, Y, **w)
        return (ro, n) + nf4.qlora_norm_bwd(dN, dRo, ro, Y, p, q, weight_grads=True, **w)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for k in range(3):
        e = problem(m, h, BF, True, True, seed=k + 1)
        for t, s in ((R, "R"), (Y, "Y"), (dN, "dN"), (dRo, "dR_out")):
            t.copy_(e[s])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, step()))
