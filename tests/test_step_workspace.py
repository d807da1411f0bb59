"""Workspaces of the cross entropy hold what few tokens need, and the kernels stay inside."""
import pytest
import torch

nf4 = pytest.importorskip("bit_quantized_fine_nf4_amd")


def rup(x, m):
    return -(-x // m) * m


@pytest.mark.parametrize("M", [1, 16, 32, 33, 100, 128])
@pytest.mark.parametrize("h,V", [(64, 1 << 20), (4096, 32000), (8192, 128256)])
def test_few_tokens_need_little(M, h, V):
    """Backward: G of whole 32- or 128-token tiles, dH's partial sums (at most 512 workgroups'
    of 256 values a token, or 8192 rows for more tokens), a copy of the rows, and lists."""
    G = 2 * rup(M, 32 if M <= 32 else 128) * rup(V, 256)
    sums = 4 * (M * (512 * 256 + rup(h, 256)) if M <= 64 else min(16 * M, 8192) * h)
    assert nf4.workspace_size(nf4.QLORA_OP_LOSS_BWD, M, h, V) <= G + sums + 2 * rup(M, 32) * h + 32 * M + 4096
    stats = 8 * rup(-(-V // 128), 2) * M
    copy = 0 if M <= 32 else 2 * rup(M, 32) * h
    assert nf4.workspace_size(nf4.QLORA_OP_LOSS_FWD, M, h, V) <= stats + copy + 16 * M + 4096


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 31, 32, 33, 64, 65, 127, 128, 129, 200, 256, 257])
@pytest.mark.parametrize("h,V", [(64, 300), (192, 1000), (256, 70001)])
def test_kernels_stay_inside(M, h, V):
    dev = "cuda:0"
    print(f"loss workspace M={M} h={h} V={V}", flush=True)
    g = torch.Generator(device=dev).manual_seed(M)
    H = torch.randn(M, h, generator=g, device=dev).to(torch.bfloat16)
    W = (torch.randn(V, h, generator=g, device=dev) * 0.2).to(torch.bfloat16)
    labels = torch.randint(-V // 8, V, (M,), generator=g, device=dev)
    dl = torch.ones(M, device=dev)
    out = {}
    for fill in (0, 255):          # whatever it held before: the same results, and nothing behind it
        ws = {}
        for op in (nf4.QLORA_OP_LOSS_FWD, nf4.QLORA_OP_LOSS_BWD):
            n = nf4.workspace_size(op, M, h, V)
            room = 2 * 512 * rup(V, 256)   # a whole larger tile of G more
            ws[op] = torch.full((n + room,), fill, dtype=torch.uint8, device=dev), n
        f, fn = ws[nf4.QLORA_OP_LOSS_FWD]
        b, bn = ws[nf4.QLORA_OP_LOSS_BWD]
        loss, lse = nf4.qlora_loss_fwd(H, W, labels, workspace=f[:fn])
        dH, dW = nf4.qlora_loss_bwd(H, W, labels, lse, dl, train_head=True, workspace=b[:bn])
        out[fill] = (loss, lse, dH, dW)
        assert torch.all(f[fn:] == fill) and torch.all(b[bn:] == fill)
    assert all(torch.equal(x, y) for x, y in zip(out[0], out[255]))
