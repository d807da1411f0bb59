"""GPU parity of the counter-based dropout (qlora_dropout) and of the linear with dropout
on its adapter's input (qlora_linear_fwd_dropout, qlora_linear_bwd_dropout) against the
oracle (oracle/dropout.py, float64).

Decisions are compared exactly.  Values of qlora_dropout: the scale and the product are
one float32 rounding each, then the output's half step.
The linear, with u = 2^-24, H = 2^-8 (half a bf16 step) and s' the scaled s; a matrix-core
sum of n products has 2 n u of its magnitudes (the 2: its rounding is not specified as
to-nearest; + 64 for joined partial sums):
  T    H |T| + 2 (h + 64) u |X||L1|
  Y    H |Y| + 2 (h + r + 64) u (|X||W| + s'|T||L2|) + 2 H s'|T||L2|     (T's bf16 copy)
  dX   H |dX| + 2 (o + r + 64) u (...) + 2 H s' keep |U||L1|             (U's bf16 copy)
  dL1  s' |keep X| (eU + 2^-25 |U|) + 2 (M + 64) u s' |keep X||U| with eU = 2 (o + 64) u |dY||L2|
  dL2  2 (M + 64) u s' |T||dY|
W is the bf16 dequantization.  With at most 16 tokens the kernels use bf16 levels instead
and the backward bf16 scaled dY: 2 H and 3 H of |X||W| and |dY||W| more."""
import numpy as np
import pytest
import torch

import oracle
import workloads as wl
from oracle import dropout as od
from parity import oracle_weight

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import bit_quantized_fine_nf4_amd as nf4  # noqa: E402

DEV = "cuda:0"
U, H = 2.0 ** -24, 2.0 ** -8
BF = torch.bfloat16


def state(seed, offset):
    wrap = lambda v: v - 2 ** 64 if v >= 2 ** 63 else v
    return torch.tensor([wrap(seed), wrap(offset)], dtype=torch.int64, device=DEV)


STATES = [(1, 0), (0xFEDCBA9876543210, 2 ** 32 - 2), (77, 2 ** 64 - 3)]   # counters pass 2^32 and wrap


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("p", [0.0, 0.05, 0.5, 65535 / 65536])
@pytest.mark.parametrize("n", [1, 7, 8, 9, 2047, 2049, 1 << 20, (1 << 23) + 5])
def test_elementwise(n, p, dtype):
    seed, offset = STATES[n % 3]
    print(f"dropout n={n} p={p} {dtype}", flush=True)
    g = torch.Generator().manual_seed(n)
    x = torch.randn(n, generator=g).to(dtype)
    x[n // 2] = float("nan")
    x[0] = float("inf")
    kept = torch.from_numpy(od.keep(seed, offset, n, p))
    rng = state(seed, offset)
    y = nf4.qlora_dropout(x.to(DEV), p, rng)
    z = x.to(DEV)
    assert nf4.qlora_dropout(z, p, rng, out=z) is z      # in place
    y, z = y.cpu(), z.cpu()
    same = (y == z) | (y.isnan() & z.isnan())
    assert same.all() and torch.all(y[~kept] == 0)
    ref = torch.where(kept, x.double() * od.scale(p), 0.0)
    fine = ref.isfinite()
    assert torch.equal(y.isnan(), ref.isnan()) and torch.equal(y.isinf(), ref.isinf())
    half = H if dtype == BF else U
    assert torch.all((y.double() - ref).abs()[fine] <= (half + 2 * U) * ref.abs()[fine])


def test_backward_and_next_offset():
    x = torch.ones(4096, dtype=torch.float32, device=DEV)
    rng = state(5, 100)
    a, b = nf4.qlora_dropout(x, 0.5, rng), nf4.qlora_dropout(2 * x, 0.5, rng)
    assert torch.equal(2 * a, b)                          # the gradient sees the same mask
    rng[1] += 4096 // 8
    c = nf4.qlora_dropout(x, 0.5, rng)
    assert not torch.equal(a, c)
    kept = od.keep(5, 100, 8192, 0.5)
    assert np.array_equal(torch.cat([a, c]).cpu().numpy() > 0, kept)


def bf16_weight(w, codebook="nf4"):
    """The bf16 dequantization, h x o."""
    if codebook == "nf4":
        wh = oracle_weight(w)
    else:
        o, h = w.shape
        p, a = oracle.codebooks.quantize(w.numpy().ravel(), codebook)
        q, s2, mean = oracle.double_quant(a)
        wh = oracle.codebooks.dequantize(p, q, s2, mean, h * o, codebook).reshape(o, h)
    return torch.from_numpy(np.ascontiguousarray(wh, dtype=np.float32)).to(BF).double().numpy().T


def check(name, got, ref, bound):
    g = got.detach().cpu().double().numpy()
    bad = np.argwhere(~(np.abs(g - ref) <= bound))
    assert bad.size == 0, (name, len(bad), bad[:3].tolist(), [(g[tuple(b)], ref[tuple(b)]) for b in bad[:3]])


def run_case(M, h, o, r, p, s=2.0, codebook="nf4", seed=3, offset=2 ** 32 - 5):
    w, l1, l2, x, dy = wl.small_linear(h, o, r, M, seed=M + r, lora_std=0.05)
    Wq = nf4.quantize_weight(w.to(DEV), codebook=nf4.CODEBOOKS[codebook])
    rng = state(seed, offset)
    d = [t.to(DEV) for t in (x, l1, l2)]
    Y, T = nf4.qlora_linear_fwd_dropout(Wq, *d, s, p, rng)
    dX, dL1, dL2 = nf4.qlora_linear_bwd_dropout(Wq, d[0], T, dy.to(DEV), d[1], d[2], s, p, rng)
    W = bf16_weight(w, codebook)
    X, A, B, dY = (t.double().numpy() for t in (x, l1, l2, dy))
    kept = od.keep(seed, offset, M * h, p).reshape(M, h)
    t64 = T.cpu().double().numpy()
    rY, rT = od.linear_fwd_dropout(W, X, A, B, s, p, kept)
    rdX, rdA, rdB = od.linear_bwd_dropout(W, X, t64, dY, A, B, s, p, kept)
    q, kx, a = s * od.scale(p), np.where(kept, X, 0.0), np.abs
    few = M <= 16
    check("T", T, rT, H * a(rT) + 2 * (h + 64) * U * (a(kx) @ a(A)))
    lora = q * (a(kx) @ a(A)) @ a(B)
    base = a(X) @ a(W)
    check("Y", Y, rY, H * a(rY) + 2 * (h + r + 64) * U * (base + lora) + 2 * H * q * (a(rT) @ a(B)) + few * 2 * H * base)
    mU, rU = a(dY) @ a(B).T, dY @ B.T
    base = a(dY) @ a(W).T
    lora = np.where(kept, q * mU @ a(A).T, 0.0)
    check("dX", dX, rdX, H * a(rdX) + 2 * (o + r + 64) * U * (base + lora) +
          2 * H * np.where(kept, q * a(rU) @ a(A).T, 0.0) + few * 3 * H * base)
    eU = 2 * (o + 64) * U * mU
    check("dL1", dL1, rdA, q * a(kx).T @ (eU + 2.0 ** -25 * a(rU)) + 2 * (M + 64) * U * q * (a(kx).T @ a(rU)))
    check("dL2", dL2, rdB, 2 * (M + 64) * U * q * (a(t64).T @ a(dY)))
    # a float32 result: far below what one bf16 U would leave (2^-9)
    assert np.linalg.norm(dL1.cpu().double().numpy() - rdA) <= 2e-6 * np.linalg.norm(rdA)
    return Wq, d, rng, Y, T, dX


CASES = [(1, 64, 64, 1), (2, 192, 128, 8), (9, 128, 640, 5), (16, 1024, 320, 64), (17, 64, 192, 16), (40, 320, 64, 17),
         (64, 128, 128, 100), (65, 576, 256, 128), (129, 192, 448, 33), (300, 256, 192, 7), (700, 512, 384, 64),
         (2100, 128, 64, 16), (200, 20480, 64, 8), (300, 30848, 64, 5), (257, 30848, 192, 70), (520, 15424, 448, 16)]


@pytest.mark.parametrize("p", [0.05, 0.5])
@pytest.mark.parametrize("M,h,o,r", CASES)
def test_linear(M, h, o, r, p):
    print(f"dropout linear M={M} h={h} o={o} r={r} p={p}", flush=True)
    run_case(M, h, o, r, p)


@pytest.mark.parametrize("codebook", ["int4", "fp4"])
def test_linear_codebooks(codebook):
    run_case(33, 128, 192, 16, 0.1, codebook=codebook)
    run_case(5, 128, 192, 16, 0.1, codebook=codebook)


@pytest.mark.parametrize("M,h,o,r", [(5, 128, 192, 16), (70, 128, 256, 24), (300, 30848, 64, 8)])
def test_no_dropout_is_the_plain_linear(M, h, o, r):
    Wq, d, rng, Y, T, _ = run_case(M, h, o, r, 0.0)
    pY, pT = nf4.qlora_linear_fwd(Wq, *d, 2.0)
    assert torch.equal(Y, pY) and torch.equal(T, pT)
    frozen = nf4.qlora_linear_fwd_dropout(Wq, d[0], None, None, 2.0, 0.5, rng)
    assert torch.equal(frozen[0], nf4.qlora_linear_fwd(Wq, d[0], None, None, 2.0)[0]) and frozen[1] is None
    dY = torch.randn(M, o, device=DEV).to(BF)
    a = nf4.qlora_linear_bwd_dropout(Wq, d[0], None, dY, None, None, 2.0, 0.5, rng)
    assert torch.equal(a[0], nf4.qlora_linear_bwd(Wq, None, None, dY, None, None, 2.0)[0]) and a[1] is a[2] is None


def test_dropped_values_reach_nothing():
    """NaN in elements that the adapter drops changes neither T nor dL1."""
    M, h, o, r, p = 20, 128, 64, 8, 0.5
    w, l1, l2, x, dy = wl.small_linear(h, o, r, M, seed=1)
    Wq, rng = nf4.quantize_weight(w.to(DEV)), state(9, 9)
    kept = torch.from_numpy(od.keep(9, 9, M * h, p).reshape(M, h))
    bad = torch.where(kept, x, torch.tensor(float("nan"), dtype=BF))
    l1, l2, dy = l1.to(DEV), l2.to(DEV), dy.to(DEV)
    res = []
    for v in (x, bad):
        _, T = nf4.qlora_linear_fwd_dropout(Wq, v.to(DEV), l1, l2, 1.0, p, rng)
        res.append((T, nf4.qlora_linear_bwd_dropout(Wq, v.to(DEV), T, dy, l1, l2, 1.0, p, rng)[1]))
    assert torch.equal(res[0][0], res[1][0]) and torch.equal(res[0][1], res[1][1])


def test_captured_step_with_an_advancing_state():
    """A graph that advances its own offset makes other decisions at each replay, the same
    as eager calls at those offsets."""
    M, h, o, r, p = 130, 256, 128, 16, 0.25
    w, l1, l2, x, dy = wl.small_linear(h, o, r, M, seed=8)
    Wq = nf4.quantize_weight(w.to(DEV))
    x, l1, l2, dy = (t.to(DEV) for t in (x, l1, l2, dy))
    rng = state(4, 1000)

    def step():
        Y, T = nf4.qlora_linear_fwd_dropout(Wq, x, l1, l2, 2.0, p, rng)
        return (Y, T) + nf4.qlora_linear_bwd_dropout(Wq, x, T, dy, l1, l2, 2.0, p, rng)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
        rng[1:].add_(M * h // 8)
    seen = []
    for k in range(3):
        at = state(4, 1000 + k * (M * h // 8))
        graph.replay()
        torch.cuda.synchronize()
        Y, T = nf4.qlora_linear_fwd_dropout(Wq, x, l1, l2, 2.0, p, at)
        eager = (Y, T) + nf4.qlora_linear_bwd_dropout(Wq, x, T, dy, l1, l2, 2.0, p, at)
        assert all(torch.equal(a, b) for a, b in zip(held, eager)), k
        seen.append(T.clone())
    assert not torch.equal(seen[0], seen[1])


def test_neighbours_are_left_alone():
    M, h, o, r, p = 37, 192, 128, 5, 0.3
    w, l1, l2, x, dy = wl.small_linear(h, o, r, M, seed=2)
    Wq, rng = nf4.quantize_weight(w.to(DEV)), state(1, 1)
    x, l1, l2, dy = (t.to(DEV) for t in (x, l1, l2, dy))
    ws = torch.full((nf4.workspace_size(nf4.QLORA_OP_LINEAR_DROPOUT, M, h, o, r) + 256,), 255, dtype=torch.uint8,
                    device=DEV)
    big = {k: torch.full((n + 64,), 7.0, dtype=t, device=DEV) for k, n, t in
           (("Y", M * o, BF), ("T", M * r, BF), ("dX", M * h, BF), ("dL1", h * r, torch.float32),
            ("dL2", r * o, torch.float32))}
    v = {k: big[k][:-64].view(*s) for k, s in
         (("Y", (M, o)), ("T", (M, r)), ("dX", (M, h)), ("dL1", (h, r)), ("dL2", (r, o)))}
    nf4.qlora_linear_fwd_dropout(Wq, x, l1, l2, 1.0, p, rng, Y=v["Y"], T=v["T"], workspace=ws[:-256])
    nf4.qlora_linear_bwd_dropout(Wq, x, v["T"], dy, l1, l2, 1.0, p, rng, dX=v["dX"], dL1=v["dL1"], dL2=v["dL2"],
                                 workspace=ws[:-256])
    assert torch.all(ws[-256:] == 255) and all(torch.all(t[-64:] == 7.0) for t in big.values())
