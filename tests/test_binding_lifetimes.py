"""Buffers that the Python binding allocates are held until the C call has enqueued its
work: given back earlier, another thread's allocation may take the same memory and use it
on the same stream before this call's kernels."""
import gc
import weakref

import pytest
import torch

import bit_quantized_fine_nf4_amd as nf4
from test_weight_binding import BF, F32, PARTS, M, Fake, h, o, r

V = 100


class Buffer(Fake):
    """A tensor with an address of its own."""
    last = 1 << 20

    def __init__(self, *a, **k):
        super().__init__(*a, **k)
        Buffer.last += 1 << 16
        self.address = Buffer.last

    def data_ptr(self):
        return self.address


def calls():
    B = Buffer
    W = nf4.NF4Weight(h=h, o=o, **{k: B(t, n) for k, (t, n) in PARTS.items()})
    X, dY, T, L1, L2, rng = B(BF, M, h), B(BF, M, o), B(BF, M, r), B(BF, h, r), B(BF, r, o), B(torch.int64, 2)
    w, rstd, head, labels, f = B(F32, h), B(F32, M), B(BF, V, h), B(torch.int64, M), B(F32, M)
    return dict(norm_fwd=lambda: nf4.qlora_norm_fwd(X, X, w, w, w),
                norm_bwd=lambda: nf4.qlora_norm_bwd(X, X, X, X, rstd, rstd, w, w, w, weight_grads=True),
                loss_fwd=lambda: nf4.qlora_loss_fwd(X, head, labels),
                loss_bwd=lambda: nf4.qlora_loss_bwd(X, head, labels, f, f, train_head=True),
                dropout=lambda: nf4.qlora_dropout(X, 0.5, rng),
                linear_fwd=lambda: nf4.qlora_linear_fwd_dropout(W, X, L1, L2, 1.0, 0.5, rng),
                linear_bwd=lambda: nf4.qlora_linear_bwd_dropout(W, X, T, dY, L1, L2, 1.0, 0.5, rng))


@pytest.mark.parametrize("name", ["norm_fwd", "norm_bwd", "loss_fwd", "loss_bwd", "dropout", "linear_fwd", "linear_bwd"])
def test_allocated_buffers_outlive_the_call(name, monkeypatch):
    made, seen = {}, []

    def empty(*shape, dtype, device):
        t = Buffer(dtype, *shape)
        made[t.address] = weakref.ref(t)
        return t

    def c_call(device, entry, *args):
        gc.collect()
        seen.append(entry)
        for a in args:
            if a in made:
                assert made[a]() is not None, f"{entry}: a buffer of the call is already gone"

    call = calls()[name]
    monkeypatch.setattr(nf4, "_call", c_call)
    monkeypatch.setattr(nf4.torch, "empty", empty)
    monkeypatch.setattr(nf4.torch, "empty_like", lambda t: empty(*t.shape, dtype=t.dtype, device=t.device))
    call()
    assert len(seen) == 1 and len(made) >= 1
