"""A training step of the operators together: norm, three NF4 linears with dropout on their
adapters around a SiLU gate, norm with gate and residual scale, cross entropy, and all of
it backwards, against the formulas' gradients in float64.

Between the operators the tensors are bf16.  A rounding changes a tensor by at most 2^-8 of
its norm, and random matrices carry a relative error on unchanged to first order, so a
gradient is off by at most the number of rounded tensors on its way: forward N0, T (of the
adapters), G, U, H, Y, N1, backward G of the loss, dN1, dY, its U, dH, dG and dU, the two
dN0 and their sum, 16 of them: 2^-4 of the gradient's norm.  A bf16 residual stream adds R1
and dR: 18 * 2^-8.  With at most 16 tokens each product with a frozen weight adds up to
three (bf16 levels, scaled dY), four such products one after the other: 30 * 2^-8."""
import numpy as np
import pytest
import torch

import workloads as wl
from oracle import dropout as od
from parity import oracle_weight

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import bit_quantized_fine_nf4_amd as nf4  # noqa: E402

DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
S, P, ALPHA, EPS, SEED = 2.0, 0.25, 0.5, 1e-5, 11


def problem(M, h, f, V, r, stream, seed=0):
    """Parameters and inputs of one block (width h, inner width f) with an output head."""
    g = torch.Generator().manual_seed(97 * M + h + 5 * f + 1000 * seed)
    n = lambda *s, std=1.0: torch.randn(*s, generator=g) * std
    d = dict(R=n(M, h).to(stream), w0=1 + n(h, std=0.2), w1=1 + n(h, std=0.2), wp=1 + n(h, std=0.2), gate=n(h),
             head=(n(V, h) * 0.1).to(BF), labels=torch.randint(0, V, (M,), generator=g))
    d["labels"][torch.rand(M, generator=g) < 0.3] = -100
    d["labels"][0] = 1
    for k, (a, b) in dict(g=(h, f), u=(h, f), d=(f, h)).items():
        w, l1, l2, _, _ = wl.small_linear(a, b, r, 1, seed=seed + a + ord(k), lora_std=0.1)
        d[k], d[k + "1"], d[k + "2"] = w, l1, l2
    return d


def used(M, h, f):
    """Generator offsets of the three linears of one step, and the next step's."""
    a, b = M * h // 8, M * f // 8
    return dict(g=0, u=a, d=2 * a), 2 * a + b


def to_gpu(d):
    out = {k: v.to(DEV) for k, v in d.items() if k not in "gud"}
    out.update({k: nf4.quantize_weight(d[k].to(DEV)) for k in "gud"})
    out["at"], _ = used(*d["R"].shape, d["g"].shape[0])
    out["rng"] = {k: torch.tensor([SEED, v], device=DEV) for k, v in out["at"].items()}
    return out


def step(d):
    """Loss per token and every gradient: of the stream, the norms' weights, the adapters
    and the head."""
    lin = lambda k, x: nf4.qlora_linear_fwd_dropout(d[k], x, d[k + "1"], d[k + "2"], S, P, d["rng"][k])
    back = lambda k, x, t, dy: nf4.qlora_linear_bwd_dropout(d[k], x, t, dy, d[k + "1"], d[k + "2"], S, P, d["rng"][k])
    R = d["R"]
    _, N0, p0, _ = nf4.qlora_norm_fwd(R, w_pre=d["w0"], eps=EPS)
    G, Tg = lin("g", N0)
    Uu, Tu = lin("u", N0)
    H = nf4.qlora_silu_gate_fwd(G, Uu)
    Y, Td = lin("d", H)
    post = dict(w_pre=d["w1"], w_post=d["wp"], gate=d["gate"], alpha=ALPHA)
    R1, N1, p1, q1 = nf4.qlora_norm_fwd(R, Y, eps=EPS, **post)
    loss, lse = nf4.qlora_loss_fwd(N1, d["head"], d["labels"])
    live = (d["labels"] >= 0).float()
    dN1, dhead = nf4.qlora_loss_bwd(N1, d["head"], d["labels"], lse, live / live.sum(), train_head=True)
    dR1, dY, dw1, dwp, dgate = nf4.qlora_norm_bwd(dN1, None, R1, Y, p1, q1, weight_grads=True, **post)
    dH, dd1, dd2 = back("d", H, Td, dY)
    dG, dU = nf4.qlora_silu_gate_bwd(G, Uu, dH)
    dNg, dg1, dg2 = back("g", N0, Tg, dG)
    dNu, du1, du2 = back("u", N0, Tu, dU)
    dR, _, dw0, _, _ = nf4.qlora_norm_bwd(nf4.qlora_grad_sum([dNg, dNu]), dR1, R, rstd_pre=p0, w_pre=d["w0"],
                                          weight_grads=True, block=False)
    return dict(loss=loss, R=dR, w0=dw0, w1=dw1, wp=dwp, gate=dgate, head=dhead,
                g1=dg1, g2=dg2, u1=du1, u2=du2, d1=dd1, d2=dd2)


def exact(d, offset=0):
    """The same in float64 on the CPU, by autograd."""
    M, h = d["R"].shape
    f = d["g"].shape[0]
    at, _ = used(M, h, f)
    leaves = {k: d[k].double().requires_grad_() for k in
              ("R", "w0", "w1", "wp", "gate", "head", "g1", "g2", "u1", "u2", "d1", "d2")}
    L = leaves

    def lin(k, x):
        kept = torch.from_numpy(od.keep(SEED, offset + at[k], x.numel(), P).reshape(x.shape))
        W = torch.from_numpy(np.ascontiguousarray(oracle_weight(d[k]), dtype=np.float32)).to(BF).double().t()
        return x @ W + S * od.scale(P) * ((kept * x) @ L[k + "1"] @ L[k + "2"])

    norm = lambda x, w: x * torch.rsqrt(x.square().mean(1, keepdim=True) + EPS) * w
    N0 = norm(L["R"], L["w0"])
    Y = lin("d", torch.nn.functional.silu(lin("g", N0)) * lin("u", N0))
    R1 = L["R"] + ALPHA * L["gate"] * norm(Y, L["wp"])
    z = norm(R1, L["w1"]) @ L["head"].t()
    live = d["labels"] >= 0
    loss = torch.zeros(M, dtype=torch.float64)
    loss[live] = torch.logsumexp(z[live], 1) - z[live].gather(1, d["labels"][live][:, None])[:, 0]
    (loss.sum() / live.sum()).backward()
    return dict(loss=loss.detach(), **{k: v.grad for k, v in leaves.items()})


def close(got, ref, rounded):
    for k in ref:
        err = torch.linalg.norm(got[k].cpu().double() - ref[k]) / torch.linalg.norm(ref[k])
        assert err <= rounded * 2.0 ** -8, (k, float(err))


CASES = [(1, 64, 128, 100, 4, F32), (9, 192, 320, 300, 8, BF), (70, 128, 192, 515, 16, F32),
         (300, 256, 448, 1000, 33, BF)]


@pytest.mark.parametrize("M,h,f,V,r,stream", CASES)
def test_step(M, h, f, V, r, stream):
    print(f"step M={M} h={h} f={f} V={V} r={r} {stream}", flush=True)
    d = problem(M, h, f, V, r, stream)
    close(step(to_gpu(d)), exact(d), (30 if M <= 16 else 16) + 2 * (stream == BF))


@pytest.mark.parametrize("M,stream", [(12, F32), (150, BF)])
def test_captured_steps_beside_each_other(M, stream):
    """Two graphs of the step, each with its own inputs and an offset that it advances,
    replayed at the same time on two streams: each gives what eager calls give."""
    h, f, V, r = 128, 256, 700, 16
    sets = [problem(M, h, f, V, r, stream, seed) for seed in (1, 2)]
    gpu = [to_gpu(d) for d in sets]
    _, used_up = used(M, h, f)
    streams, graphs, held = [torch.cuda.Stream() for _ in sets], [], []
    for d, s in zip(gpu, streams):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            step(d)
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=s):
            held.append(step(d))
            for rng in d["rng"].values():
                rng[1:].add_(used_up)
    for k in range(3):
        for i, d in enumerate(gpu):  # other labels each time: another number of tokens with a loss
            d["labels"].copy_(problem(M, h, f, V, r, stream, 10 * k + i)["labels"])
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for d, out in zip(gpu, held):
            rng = {q: torch.tensor([SEED, v + k * used_up], device=DEV) for q, v in d["at"].items()}
            eager = step(dict(d, rng=rng))
            torch.cuda.synchronize()
            assert all(torch.equal(out[q], eager[q]) for q in eager), [q for q in eager if not torch.equal(out[q], eager[q])]
    d = dict(sets[0], labels=gpu[0]["labels"].cpu())
    close(held[0], exact(d, 2 * used_up), (30 if M <= 16 else 16) + 2 * (stream == BF))
