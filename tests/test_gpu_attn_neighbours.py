"""What a token's gradients depend on: its own document, and not what is packed beside it."""
import pytest
import torch

import oracle
from attention_bounds import DEV, check, problem, reference, run

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import bit_quantized_fine_nf4_amd as nf4  # noqa: E402


@pytest.mark.parametrize("n", [20, 100, 170])
@pytest.mark.parametrize("d", [64, 128])
def test_queries_gradient_beside_a_long_document(n, d):
    """A short document alone and with one behind it whose tokens see hundreds of keys: the
    queries' tiles and the keys of each are the same, and so is dQ."""
    M, hq, hk = 900, 4, 2
    spans = oracle.spans([0, n, M], M, causal=False)
    p = problem(M, hq, hk, d, spans)
    short = {k: x[:n].contiguous() for k, x in p.items()}
    alone, beside = run(nf4, short), run(nf4, p)
    assert torch.equal(alone["O"], beside["O"][:n]) and torch.equal(alone["lse"], beside["lse"][:, :n])
    assert torch.equal(alone["dQ"], beside["dQ"][:n])


def test_few_keys_beside_many():
    """Queries of few keys (32, whose dS nearly cancel) in the same workgroups as queries of many:
    D of each by its own span (bounds: attention_bounds.py)."""
    M, hq, hk, d = 700, 2, 2, 64
    lo = torch.arange(M) // 64 * 64
    spans = torch.stack([lo, lo + 32], 1)
    many = torch.arange(M) % 64 >= 40
    spans[many] = torch.tensor([0, M])
    p = problem(M, hq, hk, d, spans.clamp(max=M))
    check(run(nf4, p), reference(p, d ** -0.5, own=(~many).to(DEV)))


@pytest.mark.parametrize("cap", [0.0, 30.0])
def test_steep_negative_bias(cap):
    """A bias that favours far keys leaves weight to a few of many keys as well: the oldest ones."""
    M, hq, hk, d = 700, 4, 2, 64
    p = problem(M, hq, hk, d, oracle.spans([0, M], M))
    slopes = -torch.tensor([0.0625, 0.25, 0.5, 1.0], device=DEV)
    check(run(nf4, p, cap=cap, slopes=slopes), reference(p, 0.125, cap, slopes, own=True))
