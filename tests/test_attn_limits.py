"""Scales and caps whose factors would overflow are turned away, on the CPU: with a cap of 2^-128
the factor 2 scale log2(e) / cap is infinite, and a score of zero times it is NaN; a cap of 2^127.9
times log2(e) is infinite."""
import ctypes

import pytest

nf4 = pytest.importorskip("bit_quantized_fine_nf4_amd")
lib = nf4.lib

A = [ctypes.c_void_p(0x100000 + 0x10000 * i) for i in range(16)]   # distinct, aligned, never dereferenced


def call(name, scale, cap, M=0):
    """M = 0 is invalid whatever the scale: sizes are looked at before limits."""
    if name == "fwd":
        return lib.qlora_attn_fwd(A[0], 128, A[1], 128, A[2], 128, A[3], None, scale, cap, M, 1, 1, 128, A[4], A[5], None)
    if name == "bwd":
        return lib.qlora_attn_bwd(A[6], A[0], 128, A[1], 128, A[2], 128, A[4], A[5], A[3], None, scale, cap, M, 1, 1,
                                  128, A[7], A[8], A[9], A[10], 1 << 40, None)
    return lib.qlora_decode_attn(A[0], A[1], A[2], 4, 16, A[3], 1, A[4], None, scale, cap, 0, M, 1, 1, 128, A[5], None,
                                 0, None)


@pytest.mark.parametrize("name", ["fwd", "bwd", "decode"])
@pytest.mark.parametrize("scale,cap", [(2.0 ** -61, 0.0), (2.0 ** 61, 0.0), (0.1, 2.0 ** -61), (0.1, 2.0 ** -128),
                                       (0.1, 2.0 ** -149), (0.1, 2.0 ** 61), (0.1, 2.0 ** 127 * 1.9)])
def test_refused(name, scale, cap):
    assert call(name, scale, cap, M=1) == nf4.QLORA_ERR_UNSUPPORTED
    assert call(name, scale, cap) == nf4.QLORA_ERR_INVALID_VALUE


@pytest.mark.gpu
@pytest.mark.parametrize("scale,cap", [(2.0 ** -60, 2.0 ** 60), (2.0 ** -60, 2.0 ** -60), (2.0 ** 60, 2.0 ** -60), (1.0, 0.0)])
def test_zero_scores_at_the_limits(scale, cap):
    """Scores of zero weigh all keys alike at every scale and cap that is taken."""
    import torch

    M, d = 40, 64
    q = torch.zeros(M, 1, d, dtype=torch.bfloat16, device="cuda:0")
    k = torch.randn(M, 1, d, generator=torch.Generator().manual_seed(1)).to(q)
    spans = torch.tensor([[0, M]] * M, dtype=torch.int32, device="cuda:0")
    O, lse = nf4.qlora_attn_fwd(q, k, k, spans, scale=scale, cap=cap)
    want = k.double().mean(0)
    # weights exp(0) = 1 are exact; the sum's roundings and O's own
    assert bool(((O.double() - want).abs() <= 2.0 ** -8 * want.abs() + 64 * 2.0 ** -24 * k.double().abs().mean(0)).all())
    assert torch.allclose(lse, torch.full_like(lse, 3.6888794541139363), rtol=2.0 ** -20)
