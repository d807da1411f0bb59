"""What the Python binding refuses before the C call: tensors that are not on the GPU, and on
it wrong types, shapes and strides."""
import pytest
import torch

import bit_quantized_fine_nf4_amd as nf4

BF, F32 = torch.bfloat16, torch.float32
M, h, o, r, V = 4, 64, 128, 8, 100


def tensors(device):
    e = lambda *s, t=BF: torch.zeros(*s, dtype=t, device=device)
    return dict(R=e(M, h), Y=e(M, h), dN=e(M, h), dR=e(M, h), w=e(h, t=F32), rstd=e(M, t=F32), H=e(M, h), head=e(V, h),
                labels=torch.zeros(M, dtype=torch.int64, device=device), lse=e(M, t=F32), dloss=e(M, t=F32),
                X=e(M, h), dY=e(M, o), L1=e(h, r), L2=e(r, o), T=e(M, r),
                rng=torch.zeros(2, dtype=torch.int64, device=device),
                codes=torch.zeros(h * o // 2, dtype=torch.uint8, device=device),
                qabsmax=torch.zeros(h * o // 64, dtype=torch.int8, device=device), scale2=e(1, t=F32), mean=e(1, t=F32))


def weight(d):
    return nf4.NF4Weight(d["codes"], d["qabsmax"], d["scale2"], d["mean"], h, o)


CALLS = dict(
    norm_fwd=(lambda d: nf4.qlora_norm_fwd(d["R"], d["Y"], d["w"]), ("R", "Y", "w")),
    norm_bwd=(lambda d: nf4.qlora_norm_bwd(d["dN"], d["dR"], d["R"], d["Y"], d["rstd"], w_pre=d["w"]),
              ("dN", "dR", "R", "Y", "rstd", "w")),
    loss_fwd=(lambda d: nf4.qlora_loss_fwd(d["H"], d["head"], d["labels"]), ("H", "head", "labels")),
    loss_bwd=(lambda d: nf4.qlora_loss_bwd(d["H"], d["head"], d["labels"], d["lse"], d["dloss"]),
              ("H", "head", "labels", "lse", "dloss")),
    dropout=(lambda d: nf4.qlora_dropout(d["X"], 0.5, d["rng"]), ("X", "rng")),
    linear_fwd=(lambda d: nf4.qlora_linear_fwd_dropout(weight(d), d["X"], d["L1"], d["L2"], 1.0, 0.5, d["rng"]),
                ("X", "L1", "L2", "rng", "codes")),
    linear_bwd=(lambda d: nf4.qlora_linear_bwd_dropout(weight(d), d["X"], d["T"], d["dY"], d["L1"], d["L2"], 1.0, 0.5,
                                                       d["rng"]), ("X", "T", "dY", "L1", "L2", "rng", "codes")))
SPOILS = dict(dtype=lambda t: t.to(torch.float16), shape=lambda t: torch.cat([t, t]).contiguous(),
              stride=lambda t: torch.stack([t, t], -1)[..., 0], host=lambda t: t.cpu())
# (more words, more tokens without anything else per token, and any shape are good calls)
GOOD = {("loss_fwd", "head", "shape"), ("loss_bwd", "head", "shape"), ("linear_fwd", "X", "shape"),
        ("dropout", "X", "shape")}
ARGS = [(c, a, s) for c, (_, args) in CALLS.items() for a in args for s in SPOILS if (c, a, s) not in GOOD]


@pytest.mark.parametrize("call", CALLS)
def test_host_tensors(call):
    with pytest.raises(ValueError):
        CALLS[call][0](tensors("cpu"))


@pytest.mark.gpu
@pytest.mark.parametrize("call,arg,spoil", ARGS)
def test_spoiled_argument(call, arg, spoil):
    d = tensors("cuda:0")
    d[arg] = SPOILS[spoil](d[arg])
    with pytest.raises(ValueError):
        CALLS[call][0](d)
    torch.cuda.synchronize()
