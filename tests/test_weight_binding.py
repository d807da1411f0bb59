"""What the Python binding refuses of an NF4 weight: parts of another type, too short, not
contiguous or somewhere else than the call's other tensors.  The C call takes bare
addresses and would read past them."""
import pytest
import torch

import bit_quantized_fine_nf4_amd as nf4

BF, F32 = torch.bfloat16, torch.float32
M, h, o, r = 4, 128, 192, 8
PARTS = dict(codes=(torch.uint8, h * o // 2), qabsmax=(torch.int8, h * o // 64), scale2=(F32, 2), mean=(F32, 1))


class Fake:
    """A tensor on cuda:0 as far as the checks can tell; nothing behind its address."""

    def __init__(self, dtype, *shape, index=0, whole=True):
        self.dtype, self.shape, self.index, self.whole = dtype, torch.Size(shape), index, whole
        self.device = torch.device("cuda", index) if index >= 0 else torch.device("cpu")
        self.is_cuda = index >= 0

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def is_contiguous(self):
        return self.whole

    def get_device(self):
        return self.index

    def data_ptr(self):
        raise AssertionError("an address was taken before the checks were through")


SPOILS = dict(dtype=lambda t, n: Fake(torch.float16, n), short=lambda t, n: Fake(t, n - 1),
              stride=lambda t, n: Fake(t, n, whole=False), host=lambda t, n: Fake(t, n, index=-1),
              other=lambda t, n: Fake(t, n, index=1))


def call(name, W, new, ws):
    """The call with every other tensor as it should be."""
    X, dY, T, L1, L2 = new(BF, M, h), new(BF, M, o), new(BF, M, r), new(BF, h, r), new(BF, r, o)
    Y, dX, dL1, dL2, rng = new(BF, M, o), new(BF, M, h), new(F32, h, r), new(F32, r, o), new(torch.int64, 2)
    if name == "fwd_dropout":
        return nf4.qlora_linear_fwd_dropout(W, X, L1, L2, 1.0, 0.5, rng, Y=Y, T=T, workspace=ws)
    if name == "bwd_dropout":
        return nf4.qlora_linear_bwd_dropout(W, X, T, dY, L1, L2, 1.0, 0.5, rng, dX, dL1, dL2, ws)
    return W.call("qlora_merge_adapter", None, None, 0, 1.0, None, nf4.QLORA_F32, None)


@pytest.mark.parametrize("spoil", SPOILS)
@pytest.mark.parametrize("part", PARTS)
@pytest.mark.parametrize("name", ["fwd_dropout", "bwd_dropout", "plain"])
def test_spoiled_weight(name, part, spoil):
    d = {k: Fake(t, n) for k, (t, n) in PARTS.items()}
    d[part] = SPOILS[spoil](*PARTS[part])
    if name == "plain" and part == "codes" and spoil == "other":
        part = "qabsmax"          # the plain calls go by the codes' device
    with pytest.raises(ValueError, match=part):
        call(name, nf4.NF4Weight(h=h, o=o, **d), Fake, Fake(torch.uint8, 1 << 20))


def test_host_weight():
    z = {k: torch.zeros(n, dtype=t) for k, (t, n) in PARTS.items()}
    with pytest.raises(ValueError, match="codes"):
        nf4.NF4Weight(h=h, o=o, **z).call("qlora_merge_adapter", None, None, 0, 1.0, None, nf4.QLORA_F32, None)


@pytest.mark.gpu
def test_parts_that_are_right():
    """Longer parts and other shapes of the same values are taken; results are the same."""
    dev = "cuda:0"
    g = torch.Generator().manual_seed(1)
    W = nf4.quantize_weight((torch.randn(o, h, generator=g) * 0.02).to(dev))
    X = torch.randn(M, h, generator=g).to(BF).to(dev)
    more = lambda t: torch.cat([t, t])
    V = nf4.NF4Weight(W.codes.view(-1, 1), more(W.qabsmax), more(W.scale2), W.mean.view(()), h, o)
    assert torch.equal(nf4.qlora_linear_fwd(W, X, None, None, 1.0)[0], nf4.qlora_linear_fwd(V, X, None, None, 1.0)[0])
    V.codes = W.codes
    L1, L2 = torch.zeros(h, r, dtype=BF, device=dev), torch.zeros(r, o, dtype=BF, device=dev)
    rng = torch.zeros(2, dtype=torch.int64, device=dev)
    Y = [nf4.qlora_linear_fwd_dropout(w, X, L1, L2, 1.0, 0.5, rng)[0] for w in (W, V)]
    assert torch.equal(*Y)


@pytest.mark.gpu
@pytest.mark.parametrize("spoil", ["short", "host", "dtype"])
@pytest.mark.parametrize("part", PARTS)
def test_spoiled_weight_on_the_gpu(part, spoil):
    dev = "cuda:0"
    d = {k: torch.zeros(n, dtype=t, device=dev) for k, (t, n) in PARTS.items()}
    d[part] = dict(short=d[part][1:], host=d[part].cpu(), dtype=d[part].to(torch.float16))[spoil]
    W = nf4.NF4Weight(h=h, o=o, **d)
    z = lambda t, *s: torch.zeros(*s, dtype=t, device=dev)
    X, dY, T, L1, L2 = z(BF, M, h), z(BF, M, o), z(BF, M, r), z(BF, h, r), z(BF, r, o)
    rng = z(torch.int64, 2)
    for f in (lambda: nf4.qlora_linear_fwd_dropout(W, X, L1, L2, 1.0, 0.5, rng),
              lambda: nf4.qlora_linear_bwd_dropout(W, X, T, dY, L1, L2, 1.0, 0.5, rng),
              lambda: nf4.qlora_linear_fwd(W, X, L1, L2, 1.0), lambda: nf4.qlora_linear_bwd(W, X, T, dY, L1, L2, 1.0),
              lambda: nf4.qlora_merge_adapter(W, L1, L2, 1.0), lambda: nf4.qlora_merge_requantize(W, L1, L2, 1.0)):
        with pytest.raises(ValueError):
            f()
    torch.cuda.synchronize()
