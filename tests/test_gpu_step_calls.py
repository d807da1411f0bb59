"""Calls that a user makes of the training step's operators besides the plain one: from two
host threads at once, each weight's gradient alone, streams' buffers given or not."""
import threading

import pytest
import torch

import workloads as wl
from test_gpu_norm import F32, dev, problem as norm_problem
from test_gpu_loss import problem as loss_problem

import bit_quantized_fine_nf4_amd as nf4

pytestmark = pytest.mark.gpu
DEV, BF = "cuda:0", torch.bfloat16


def make(seed, M=150, h=320, o=192, r=16, V=900):
    """One thread's step: norms, the linear with dropout, the loss, and back."""
    d = norm_problem(M, h, BF, True, True, seed=seed)
    w = dict(w_pre=dev(d["w_pre"]), w_post=dev(d["w_post"]), gate=dev(d["gate"]), alpha=0.5)
    R, Y, dRo = (dev(d[k]) for k in ("R", "Y", "dR_out"))
    wt, l1, l2, _, _ = wl.small_linear(h, o, r, M, seed=seed)
    W = nf4.quantize_weight(wt.to(DEV))
    l1, l2 = l1.to(DEV), l2.to(DEV)
    rng = torch.tensor([seed, 99], dtype=torch.int64, device=DEV)
    _, head, labels, dl = (t.to(DEV) for t in loss_problem(M, o, V, "some", seed=seed))

    def step():
        ro, n, p, q = nf4.qlora_norm_fwd(R, Y, **w)
        y, t = nf4.qlora_linear_fwd_dropout(W, n, l1, l2, 1.0, 0.2, rng)
        loss, lse = nf4.qlora_loss_fwd(y, head, labels)
        dy, dhead = nf4.qlora_loss_bwd(y, head, labels, lse, dl, train_head=True)
        dn, d1, d2 = nf4.qlora_linear_bwd_dropout(W, n, t, dy, l1, l2, 1.0, 0.2, rng)
        return (ro, n, y, loss, lse, dhead, d1, d2) + nf4.qlora_norm_bwd(dn, dRo, ro, Y, p, q, weight_grads=True, **w)
    return step


@pytest.mark.parametrize("own_streams", [True, False])
@pytest.mark.parametrize("M", [12, 150])
def test_two_threads(M, own_streams):
    """Every buffer a call allocates is its own until its work is enqueued."""
    steps = [make(s, M) for s in (1, 2)]
    want = [[t.clone() for t in s()] for s in steps]
    torch.cuda.synchronize()
    bad, errors = [0, 0], []
    gate = threading.Barrier(2)

    def work(k):
        try:
            with torch.cuda.stream(torch.cuda.Stream() if own_streams else torch.cuda.default_stream()):
                gate.wait(20)
                for _ in range(40):
                    got = steps[k]()
                    torch.cuda.current_stream().synchronize()
                    bad[k] += not all(torch.equal(a, b) for a, b in zip(got, want[k]))
        except Exception as e:  # noqa: BLE001 (reported below)
            errors.append(e)

    threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    assert not errors and bad == [0, 0]


@pytest.mark.parametrize("rt", [BF, F32])
@pytest.mark.parametrize("m,h", [(40, 200), (300, 5003), (300, 9000)])
def test_each_weights_gradient_alone(m, h, rt):
    d = norm_problem(m, h, rt, True, True)
    w = dict(w_pre=dev(d["w_pre"]), w_post=dev(d["w_post"]), gate=dev(d["gate"]), alpha=0.5)
    R, Y, dN, dRo = (dev(d[k]) for k in ("R", "Y", "dN", "dR_out"))
    p, q = (torch.rsqrt(t.float().square().mean(1) + 1e-5) for t in (R, Y))
    every = nf4.qlora_norm_bwd(dN, dRo, R, Y, p, q, weight_grads=True, **w)
    for i, name in ((2, "dw_pre"), (3, "dw_post"), (4, "dgate")):
        out = nf4.qlora_norm_bwd(dN, dRo, R, Y, p, q, **{name: torch.empty(h, device=DEV)}, **w)
        assert all(torch.equal(out[k], every[k]) for k in (0, 1, i))
        assert all(out[k] is None for k in (2, 3, 4) if k != i)


@pytest.mark.parametrize("m,h", [(5, 64), (300, 5003)])
def test_gate_without_norms_before_or_after(m, h):
    """The residual update alone, with a gate that is trained: no norm at either end."""
    d = norm_problem(m, h, F32, False, True, pre=False)
    Y, dRo, g = dev(d["Y"]), dev(d["dR_out"]), dev(d["gate"])
    dR, dY, a, b, dg = nf4.qlora_norm_bwd(None, dRo, None, Y, gate=g, alpha=0.5, weight_grads=True)
    assert a is b is None and torch.equal(dR, dRo)
    ref = 0.5 * (d["dR_out"].double() * d["Y"].double())
    bound = (m + 64) * 2.0 ** -24 * ref.abs().sum(0)
    assert torch.all((dg.cpu().double() - ref.sum(0)).abs() <= bound)
    du = 0.5 * d["gate"].double() * d["dR_out"].double()
    assert torch.all((dY.cpu().double() - du).abs() <= (2.0 ** -8 + 2.0 ** -22) * du.abs())
