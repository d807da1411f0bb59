"""GPU parity of attention under caps that the scores do not come near: the error of a capped
score goes by the score, not by the cap (bounds: attention_bounds.py, and for one new token
those of test_gpu_cache.py with 16 u |z| in the place of its cap's term)."""
import pytest
import torch

import oracle
from attention_bounds import BF, DEV, R, U, check, problem, reference, run

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import bit_quantized_fine_nf4_amd as nf4  # noqa: E402

CAPS = [2.0, 30.0, 1e3, 1e5, 1e7, 1e18]


@pytest.mark.parametrize("cap", CAPS)
@pytest.mark.parametrize("M,hq,hk,d", [(200, 4, 2, 64), (330, 3, 3, 128), (90, 2, 1, 40)])
def test_caps(M, hq, hk, d, cap):
    p = problem(M, hq, hk, d, oracle.spans([0, 40, M], M))
    # (a query of 256 keys or fewer has D from its own sum)
    own = (p["spans"][:, 1] - p["spans"][:, 0] <= 256) if M <= 256 else False
    check(run(nf4, p, cap=cap), reference(p, d ** -0.5, cap, own=own))


@pytest.mark.parametrize("cap", CAPS)
def test_caps_of_one_new_token(cap):
    B, hq, hk, d, page, width = 5, 6, 2, 64, 16, 30
    g = torch.Generator().manual_seed(3)
    k, v = (torch.randn(B * width, hk, page, d, generator=g).to(BF).to(DEV) for _ in range(2))
    table = torch.randperm(B * width, generator=g).view(B, width).to(torch.int32).to(DEV)
    lens = torch.tensor([1, 30, 129, 300, 480], dtype=torch.int32, device=DEV)
    q = (torch.randn(B, hq, d, generator=g) * 4).to(BF).to(DEV)
    got = nf4.qlora_decode_attn(q, k, v, table, lens, cap=cap).double()
    for b, n in enumerate(lens.tolist()):
        j = torch.arange(n, device=DEV)
        at = table[b].long()[j // page]
        for h in range(hq):
            kk, vv = (x[at, h // (hq // hk), j % page].double() for x in (k, v))
            x = d ** -0.5 * (kk @ q[b, h].double())
            z = cap * torch.tanh(x / cap)
            ez = 2 * d * U * d ** -0.5 * (kk.abs() @ q[b, h].double().abs()) + 16 * U * z.abs()
            ez = ez + 8 * U * (z.abs() + z.abs().max())
            w = torch.softmax(z, 0)
            o = w @ vv
            bound = (w * (ez + R + (2 * n + 80) * U)) @ vv.abs() + o.abs() * (ez.max() + (n + 80) * U + R)
            off = (got[b, h] - o).abs()
            assert bool((off <= bound * (1 + 2.0 ** -5) + n * 2.0 ** -120).all()), (b, h, float(off.max()))
