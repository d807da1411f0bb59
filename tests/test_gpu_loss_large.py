"""Cross entropy at the edge of the documented sizes, where one launch of 128 x 128 tiles
would hold 2^32 threads: 131072 tokens, 2^21 words, 64 values.  Loss and lse of sampled
tokens against float64.  Bounds as in test_gpu_loss.py, and for the join of the tiles'
statistics, of which a lane takes 257 (there at most 8): two products, a sum and an
exponential's half step each, 4 * 257 u more."""
import pytest
import torch

from test_gpu_loss import BF, DEV, U, check, reference

import bit_quantized_fine_nf4_amd as nf4

pytestmark = pytest.mark.gpu


def test_more_workgroups_than_one_launch_holds():
    M, h, V = 1 << 17, 64, (1 << 21) + 33
    assert (M // 128) * -(-V // 128) >= 1 << 24
    g = torch.Generator(device=DEV).manual_seed(5)
    H = torch.randn(M, h, generator=g, device=DEV).to(BF)
    W = (torch.randn(V, h, generator=g, device=DEV) * 0.2).to(BF)
    labels = torch.randint(0, V, (M,), generator=g, device=DEV)
    labels[::7] = -100
    at = torch.tensor([1, 2, 63, 128, 6001, M // 2, M - 300, M - 2, M - 1], device=DEV)
    labels[at] = torch.tensor([0, V - 1, V - 34, 1 << 20, 127, 128, 2097024, 2096895, 5], device=DEV)
    print(f"loss M={M} h={h} V={V}", flush=True)
    loss, lse = nf4.qlora_loss_fwd(H, W, labels)
    live, ref = reference(H[at], W, labels[at], torch.ones(len(at), device=DEV))
    assert len(live) == len(at)
    for name, got in (("lse", lse), ("loss", loss)):
        value, bound = ref[name]
        check(name, got[at], value, bound + 4 * 257 * U)
    dead = labels < 0
    assert torch.all(loss[dead] == 0) and torch.all(lse[dead] == 0)
    assert torch.isfinite(loss).all() and torch.all(lse[~dead] > 10)    # log(V) is 14.6
