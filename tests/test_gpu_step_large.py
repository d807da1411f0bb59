"""The training step's operators on tensors of more than 2^31 values, where element offsets
pass 32 bits: values in places around the borders and at the end, against float64, with the
bounds of the operators' own tests.  Gradients that sum over rows get their terms from the
sampled rows alone (the others' factors are 0)."""
import numpy as np
import pytest
import torch

import oracle
import test_gpu_loss as tl
import test_gpu_norm as tn
from oracle import dropout as od
from test_gpu_dropout import BF, DEV, H, U, bf16_weight, check, state

import bit_quantized_fine_nf4_amd as nf4

pytestmark = pytest.mark.gpu
F32 = torch.float32


@pytest.fixture(autouse=True)
def room():
    yield
    torch.cuda.empty_cache()


def randn(*shape, seed=0, std=1.0, dtype=BF):
    t = torch.empty(shape, dtype=dtype, device=DEV)
    return t.normal_(0.0, std, generator=torch.Generator(device=DEV).manual_seed(seed))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_dropout(dtype):
    n, p = (1 << 31) + 77, 0.3
    print(f"dropout of {n} values", flush=True)
    x = randn(n, dtype=dtype)
    offset = 2 ** 32 - 2 ** 27          # the counter's low half wraps on the way
    y = nf4.qlora_dropout(x, p, state(77, offset))
    for at in (0, (1 << 30) - 64, (1 << 31) - 4096, n - n % 8 - 4096):
        k = min(n - at, 8192)
        kept = torch.from_numpy(od.keep(77, offset + at // 8, k, p)).to(DEV)
        ref = torch.where(kept, x[at:at + k].double() * od.scale(p), 0.0)
        half = H if dtype == BF else U
        assert torch.all((y[at:at + k].double() - ref).abs() <= (half + 2 * U) * ref.abs())


@pytest.mark.parametrize("m,h", [(131200, 16384), (131100, 16383)])
def test_norm(m, h):
    print(f"norm {m} x {h}", flush=True)
    rows = torch.tensor([0, 1, 65535, 65536, 131071, 131072, m - 2, m - 1], device=DEV)
    R, Y = randn(m, h, seed=1, std=2.0), randn(m, h, seed=2)
    w = dict(w_pre=1 + randn(h, seed=3, std=0.2, dtype=F32), w_post=1 + randn(h, seed=4, std=0.2, dtype=F32),
             gate=randn(h, seed=5, dtype=F32))
    got = nf4.qlora_norm_fwd(R, Y, eps=1e-5, alpha=0.5, **w)
    d = dict(R=R[rows], Y=Y[rows], **w)
    tn.check_fwd(d, 0.5, 1e-5, [t[rows] for t in got])
    p, q = got[2], got[3]
    del got
    dN, dR = torch.zeros_like(R), torch.zeros_like(R)
    dN[rows], dR[rows] = randn(len(rows), h, seed=6), randn(len(rows), h, seed=7)
    out = nf4.qlora_norm_bwd(dN, dR, R, Y, p, q, alpha=0.5, weight_grads=True, **w)
    d.update(dN=dN[rows], dR_out=dR[rows])
    tn.check_bwd(d, (p[rows], q[rows]), 0.5, [out[0][rows], out[1][rows], *out[2:]], m)
    assert not out[0][2:65535].any() and not out[1][65537:131071].any()


@pytest.mark.parametrize("r", [8, 24])
def test_linear_with_dropout(r):
    M, h, o, p, s = 1 << 18, 8256, 64, 0.25, 2.0
    print(f"dropout linear {M} x {h} -> {o}, r {r}", flush=True)
    rows = [0, 7, 1 << 17, (1 << 31) // h, (1 << 31) // h + 1, M - 17, M - 1]
    at = torch.tensor(rows, device=DEV)
    w = torch.randn(o, h, generator=torch.Generator().manual_seed(1)) * 0.02
    Wq = nf4.quantize_weight(w.to(DEV))
    l1, l2 = randn(h, r, seed=2, std=0.05), randn(r, o, seed=3, std=0.05)
    X = torch.zeros(M, h, dtype=BF, device=DEV)
    X[at] = randn(len(rows), h, seed=4)
    dY = randn(M, o, seed=5)
    seed, offset = 5, 2 ** 32 - 1000
    rng = state(seed, offset)
    Y, T = nf4.qlora_linear_fwd_dropout(Wq, X, l1, l2, s, p, rng)
    dX, dL1, dL2 = nf4.qlora_linear_bwd_dropout(Wq, X, T, dY, l1, l2, s, p, rng)
    W = bf16_weight(w)
    A, B = (t.cpu().double().numpy() for t in (l1, l2))
    x, y, t, dy, dx = (v[at].cpu().double().numpy() for v in (X, Y, T, dY, dX))
    kept = np.stack([od.keep(seed, offset + m * h // 8, h, p) for m in rows])
    q, kx, a = s * od.scale(p), np.where(kept, x, 0.0), np.abs
    rY, rT = od.linear_fwd_dropout(W, x, A, B, s, p, kept)
    check("T", T[at], rT, H * a(rT) + 2 * (h + 64) * U * (a(kx) @ a(A)))
    mag = a(x) @ a(W) + q * (a(kx) @ a(A)) @ a(B)
    check("Y", Y[at], rY, H * a(rY) + 2 * (h + r + 64) * U * mag + 2 * H * q * (a(rT) @ a(B)))
    rdX, rdA, rdB = od.linear_bwd_dropout(W, x, t, dy, A, B, s, p, kept)   # X, and so T, is 0 elsewhere
    mU, rU = a(dy) @ a(B).T, dy @ B.T
    mag = a(dy) @ a(W).T + np.where(kept, q * mU @ a(A).T, 0.0)
    check("dX", dX[at], rdX, H * a(rdX) + 2 * (o + r + 64) * U * mag + 2 * H * np.where(kept, q * a(rU) @ a(A).T, 0.0))
    check("dL1", dL1, rdA, q * a(kx).T @ (2 * (o + 64) * U * mU + 2.0 ** -25 * a(rU)) +
          2 * (M + 64) * U * q * (a(kx).T @ a(rU)))
    check("dL2", dL2, rdB, 2 * (M + 64) * U * q * (a(t).T @ a(dy)))
    assert not T[8:1 << 17].any()


def test_loss_of_many_hidden_values():
    M, h, V = 1 << 18, 8256, 300
    print(f"loss {M} x {h} x {V}", flush=True)
    at = torch.tensor([0, 1, 131071, 260100, 260112, M - 2, M - 1], device=DEV)
    Hs, W = randn(M, h, seed=1), randn(V, h, seed=2, std=0.02)
    labels = torch.randint(0, V, (M,), device=DEV, generator=torch.Generator(device=DEV).manual_seed(3))
    dl = torch.zeros(M, device=DEV)
    dl[at] = randn(len(at), seed=4, dtype=F32)
    loss, lse = nf4.qlora_loss_fwd(Hs, W, labels)
    dH, dW = nf4.qlora_loss_bwd(Hs, W, labels, lse, dl, train_head=True)
    _, ref = tl.reference(Hs[at], W, labels[at], dl[at])
    for k, got in (("loss", loss[at]), ("lse", lse[at]), ("dH", dH[at]), ("dW", dW)):
        tl.check(k, got, *ref[k])
    assert not dH[2:131071].any()


@pytest.mark.parametrize("M", [20, 40, 200])
def test_loss_of_a_large_head(M):
    h, V = 8256, 1 << 18
    print(f"loss {M} x {h} x {V}", flush=True)
    Hs, W = randn(M, h, seed=1), randn(V, h, seed=2, std=0.02)
    labels = torch.randint(0, V, (M,), device=DEV, generator=torch.Generator(device=DEV).manual_seed(3))
    labels[0], labels[1], labels[2] = V - 1, 260111, 0
    dl = randn(M, seed=4, dtype=F32)
    loss, lse = nf4.qlora_loss_fwd(Hs, W, labels)
    dH, dW = nf4.qlora_loss_bwd(Hs, W, labels, lse, dl, train_head=True)
    # the reference of test_gpu_loss.py over pieces of the vocabulary
    x, dl64, row = Hs.double(), dl.double(), torch.arange(M, device=DEV)
    z, mag = (torch.cat([f(x) @ f(w.double()).t() for w in W.split(1 << 14)], 1) for f in (lambda t: t, torch.abs))
    ez = 2 * h * U * mag
    ref = torch.logsumexp(z, 1)
    el = ez.amax(1) + (256 + 4 * (z.amax(1) - z.amin(1))) * U + 2 * U * ref.abs()
    tl.check("lse", lse, ref, el)
    tl.check("loss", loss, ref - z[row, labels], el + ez[row, labels] + U * (ref - z[row, labels]).abs())
    P = torch.exp(z - ref[:, None])
    eG = P * (ez + el[:, None] + (4 + 2 * (z - ref[:, None]).abs()) * U) * dl64.abs()[:, None]
    P[row, labels] -= 1
    G = P * dl64[:, None]
    eG += (2.0 ** -8 + 6 * U) * G.abs() + tl.TINY * (dl64.abs()[:, None] + 2 * dl64.abs().max())
    rH, eH = torch.zeros_like(x), torch.zeros_like(x)
    for k, w in enumerate(W.split(1 << 14)):
        c = slice(k << 14, (k << 14) + len(w))
        w = w.double()
        rH += G[:, c] @ w
        eH += (eG[:, c] + 2 * (V + 32) * U * G[:, c].abs()) @ w.abs()
    tl.check("dH", dH, rH, eH + 2.0 ** -8 * rH.abs())
    for c in (slice(0, 300), slice(260000, 260300), slice(V - 300, V)):
        rW = G[:, c].t() @ x
        tl.check("dW", dW[c], rW, eG[:, c].t() @ x.abs() + 2 * (M + 32) * U * (G[:, c].abs().t() @ x.abs()) + 2.0 ** -8 * rW.abs())
