"""The adapter gradients of odd token counts at odd ranks: T then has an odd number of
elements, which ends in half a dword.

dL2 = s T^T dY on the T that the forward returned: bf16 products are exact, the float32
sum of M of them is off by at most 2 (M + 64) 2^-24 of its magnitudes (2: the matrix
cores' rounding is not specified as to-nearest; 64: joined partial sums)."""
import numpy as np
import pytest
import torch

import workloads as wl

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import bit_quantized_fine_nf4_amd as nf4  # noqa: E402

DEV = "cuda:0"


@pytest.mark.parametrize("M,h,o,r", [(129, 192, 448, 33), (17, 64, 64, 17), (1, 64, 128, 19), (3, 128, 64, 127),
                                     (65, 128, 128, 101), (2049, 64, 64, 21), (128, 64, 64, 33), (33, 64, 64, 9)])
def test_last_token_counts(M, h, o, r):
    print(f"odd T M={M} h={h} o={o} r={r}", flush=True)
    w, l1, l2, x, dy = wl.small_linear(h, o, r, M, seed=M, lora_std=0.05)
    W = nf4.quantize_weight(w.to(DEV))
    x, l1, l2, dy = (t.to(DEV) for t in (x, l1, l2, dy))
    _, T = nf4.qlora_linear_fwd(W, x, l1, l2, 0.5)
    _, _, dL2 = nf4.qlora_linear_bwd(W, x, T, dy, l1, l2, 0.5)
    t, d, got = (v.cpu().double().numpy() for v in (T, dy, dL2))
    assert np.all(np.abs(got - 0.5 * t.T @ d) <= 0.5 * 2 * (M + 64) * 2.0 ** -24 * (np.abs(t).T @ np.abs(d)))
