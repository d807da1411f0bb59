"""Cross entropy where whole stretches of the vocabulary are masked with -inf: a head whose
last column is a bias (0, or -inf for the masked words) and hidden states whose last value
is 1.  A masked word's logit is -inf and its probability 0, also where every word of a tile
is masked.  Bounds as in test_gpu_loss.py, over the other words."""
import pytest
import torch

from test_gpu_loss import BF, DEV, check, problem, reference

import bit_quantized_fine_nf4_amd as nf4

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("masked", [[(0, 128)], [(128, 512)], [(0, 40), (96, 160), (600, 901)], [(0, 900)]])
@pytest.mark.parametrize("M", [1, 7, 32, 33, 128, 200, 600])
@pytest.mark.parametrize("V", [901, 14001])
def test_masked_words(M, V, masked):
    h = 192
    H, W, labels, dl = problem(M, h, V, "none")
    H[:, -1], W[:, -1] = 1.0, 0.0
    word = torch.zeros(V, dtype=torch.bool)
    for a, b in masked:
        word[a:min(b, V)] = True
    word[V - 1] = False
    left = (~word).nonzero()[:, 0]
    labels = left[labels % len(left)]
    place = torch.cumsum(~word, 0) - 1         # of a word among those that are left
    W[word, -1] = float("-inf")
    print(f"masked words M={M} V={V} {masked}", flush=True)
    H, W, labels, dl = (x.to(DEV) for x in (H, W, labels, dl))
    loss, lse = nf4.qlora_loss_fwd(H, W, labels)
    _, ref = reference(H, W[left.to(DEV)], place.to(DEV)[labels], dl)
    check("lse", lse, *ref["lse"])
    check("loss", loss, *ref["loss"])
    dH, _ = nf4.qlora_loss_bwd(H, W, labels, lse, dl)
    # (the bias's own column multiplies a probability of 0 by -inf)
    check("dH", dH[:, :-1], *(x[:, :-1] for x in ref["dH"]))


