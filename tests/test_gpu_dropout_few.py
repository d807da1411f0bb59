"""The linear with dropout on its adapter's input at 16 tokens and fewer, against float64
with the format's weight: the bf16 dequantization that calls of more tokens multiply by.

Bounds as in test_gpu_dropout.py, and nothing more for few tokens: with u = 2^-24 and H =
2^-8 (half a bf16 step) each product of two bf16 values is exact in float32, a sum of n has
2 n u of its magnitudes, and the result is rounded once (H), as are s'T and s'U (2 H with
T's own rounding)."""
import numpy as np
import pytest
import torch

import workloads as wl
from oracle import dropout as od
from test_gpu_dropout import BF, DEV, H, U, bf16_weight, check, state

import bit_quantized_fine_nf4_amd as nf4

pytestmark = pytest.mark.gpu


def run_case(M, h, o, r, p, codebook="nf4", s=2.0, seed=11, offset=7):
    w, l1, l2, x, dy = wl.small_linear(h, o, r, M, seed=M + r, lora_std=0.05)
    Wq = nf4.quantize_weight(w.to(DEV), codebook=nf4.CODEBOOKS[codebook])
    rng = state(seed, offset)
    x_, l1_, l2_, dy_ = (t.to(DEV) for t in (x, l1, l2, dy))
    Y, T = nf4.qlora_linear_fwd_dropout(Wq, x_, l1_, l2_, s, p, rng)
    dX = nf4.qlora_linear_bwd_dropout(Wq, x_, T, dy_, l1_, l2_, s, p, rng)[0]
    W = bf16_weight(w, codebook)
    X, A, B, dY = (t.double().numpy() for t in (x, l1, l2, dy))
    kept = od.keep(seed, offset, M * h, p).reshape(M, h)
    q, kx, a = s * od.scale(p), np.where(kept, X, 0.0), np.abs
    rY, rT = od.linear_fwd_dropout(W, X, A, B, s, p, kept)
    rdX = od.linear_bwd_dropout(W, X, T.cpu().double().numpy(), dY, A, B, s, p, kept)[0]
    mag = a(X) @ a(W) + q * (a(kx) @ a(A)) @ a(B)
    check("Y", Y, rY, H * a(rY) + 2 * (h + r + 64) * U * mag + 2 * H * q * (a(rT) @ a(B)))
    mag = a(dY) @ a(W).T + np.where(kept, q * (a(dY) @ a(B).T) @ a(A).T, 0.0)
    check("dX", dX, rdX, H * a(rdX) + 2 * (o + r + 64) * U * mag +
          2 * H * np.where(kept, q * a(dY @ B.T) @ a(A).T, 0.0))


CASES = [(1, 64, 64, 1), (1, 192, 1088, 16), (1, 16448, 64, 4), (2, 192, 128, 8), (3, 576, 1088, 128), (4, 320, 192, 5),
         (5, 4096, 512, 16), (8, 1024, 4096, 8), (9, 128, 640, 5), (16, 1024, 320, 64), (16, 64, 20480, 33)]


@pytest.mark.parametrize("p", [1 / 65536, 0.05, 0.5])
@pytest.mark.parametrize("M,h,o,r", CASES)
def test_few_tokens_multiply_the_formats_weight(M, h, o, r, p):
    print(f"dropout linear, few tokens: M={M} h={h} o={o} r={r} p={p}", flush=True)
    run_case(M, h, o, r, p)


@pytest.mark.parametrize("codebook", ["int4", "fp4"])
@pytest.mark.parametrize("M", [1, 3, 13])
def test_codebooks(codebook, M):
    run_case(M, 448, 192, 16, 0.1, codebook=codebook)


def test_captured_and_replayed():
    """One captured step of few tokens, replayed on new inputs and states between eager calls."""
    M, h, o, r, p = 6, 320, 192, 8, 0.3
    w, l1, l2, x, dy = wl.small_linear(h, o, r, M, seed=4)
    Wq = nf4.quantize_weight(w.to(DEV))
    x, l1, l2, dy = (t.to(DEV) for t in (x, l1, l2, dy))
    rng = state(3, 5)

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
    for k in range(3):
        x.copy_(torch.randn(M, h, generator=torch.Generator().manual_seed(k)).to(BF))
        rng[1] += 1000
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, step())), k
