"""Attention of one new token for thousands of sequences (bound: test_gpu_cache.py)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import bit_quantized_fine_nf4_amd as nf4  # noqa: E402

DEV = "cuda:0"
BF = torch.bfloat16
U, R = 2.0 ** -24, 2.0 ** -8


def batch(B, hq, hk, d, page, width, most, seed=0):
    """Sequences that share a cache of a few pages (each may be in many tables)."""
    g = torch.Generator(device=DEV).manual_seed(seed + B)
    k, v = (torch.randn(64, hk, page, d, generator=g, device=DEV).to(BF) for _ in range(2))
    table = torch.randint(0, 64, (B, width), generator=g, device=DEV, dtype=torch.int32)
    lens = torch.randint(0, most + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
    lens[lens % 5 == 0] = 1
    q = torch.randn(B, hq, d, generator=g, device=DEV).to(BF)
    return q, k, v, table, lens


@pytest.mark.parametrize("B,hq,hk,d,page,width,most", [(5000, 4, 2, 32, 16, 20, 320), (9000, 1, 1, 64, 64, 8, 500),
                                                       (2500, 34, 2, 16, 8, 30, 240)])
def test_thousands_of_sequences(B, hq, hk, d, page, width, most):
    q, k, v, table, lens = batch(B, hq, hk, d, page, width, most)
    got = nf4.qlora_decode_attn(q, k, v, table, lens).double()
    n = width * page
    group, scale = hq // hk, d ** -0.5
    for b0 in range(0, B, 500):
        t, m = table[b0:b0 + 500].long(), lens[b0:b0 + 500].long()
        kk, vv = (x[t].double().transpose(1, 2).reshape(len(m), hk, n, d) for x in (k, v))
        qq = q[b0:b0 + 500].double().view(len(m), hk, group, d)
        seen = (torch.arange(n, device=DEV) < m[:, None])[:, None, None]
        z = scale * (qq @ kk.transpose(2, 3).contiguous())
        ez = 2 * d * U * scale * (qq.abs() @ kk.abs().transpose(2, 3).contiguous())
        z = z.masked_fill(~seen, -torch.inf)
        far = torch.where(seen, z.abs(), 0.0)
        ez = torch.where(seen, ez + 8 * U * (far + far.amax(-1, keepdim=True)), 0.0)
        w = torch.nan_to_num(torch.softmax(z, -1))          # (a sequence of none: zero)
        o = w @ vv
        bound = (w * (ez + R + (2 * n + 80) * U)) @ vv.abs() + o.abs() * (ez.amax(-1, keepdim=True) + (n + 80) * U + R)
        off = (got[b0:b0 + 500].view_as(o) - o).abs()
        assert bool((off <= bound * (1 + 2.0 ** -5) + n * 2.0 ** -120).all()), (b0, float(off.max()))


def test_time_goes_by_the_sequences():
    """The join of a row does not look through all sequences: with eight times as many (one token
    each, so that the lengths are what is read) a call takes well under the 64 times that it
    would; 24 leaves room for what does not grow."""
    def time(B):
        q, k, v, table, lens = batch(B, 16, 1, 32, 16, 9, 1)
        ws = torch.empty(nf4.workspace_size(nf4.QLORA_OP_DECODE_ATTN, B, 16, 9 * 16, 1), dtype=torch.uint8, device=DEV)
        O = torch.empty_like(q)
        best = float("inf")
        for _ in range(6):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            nf4.qlora_decode_attn(q, k, v, table, lens, O=O, workspace=ws)
            b.record()
            b.synchronize()
            best = min(best, a.elapsed_time(b))
        return best

    small, large = time(8192), time(65536)
    print(f"8192 sequences {1e3 * small:.0f} us, 65536 {1e3 * large:.0f} us", flush=True)
    assert large < 24 * small
