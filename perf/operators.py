"""The operators of a QLoRA training step around the frozen linears, as cases to measure.

Three groups, each in the directions that a step takes it:

  norm     the residual update after a block (optional norm of the block's output, a
           per-channel gate, a residual scale) together with the RMS norm before the
           next block, and its backward with the gradients of the three weights;
  dropout  inverted dropout from a counter-based generator whose mask is never stored:
           elementwise, and on the adapter branch of the NF4 linear, forward and backward;
  loss     softmax cross entropy of a bf16 output head over a large vocabulary without
           keeping the logits: loss alone, and loss with the gradient of the hidden
           states and, where the head is trained, of the head.

With `own` false `run` is the plain form in elementary torch operations; with `own`
true it makes the framework's calls.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DEVICE = "cuda:0"
EPS = 1e-5
IGNORED = -100

# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------


def listed():
    return [
        # one decoded token of the widest block: residual add and the next norm, launch-bound
        dict(name="norm_fwd_token", op="norm", grad=False, M=1, h=8192, res="bf16", post=False, gate=False, alpha=1.0),
        # a 2048-token batch of an 8192-wide block with norms on both sides and a gate
        dict(name="norm_fwd_block", op="norm", grad=False, M=2048, h=8192, res="bf16", post=True, gate=True, alpha=0.5),
        # the backward of a 4096-wide block whose residual stream is kept in float32, pre-norm only
        dict(name="norm_bwd_f32", op="norm", grad=True, M=4096, h=4096, res="f32", post=False, gate=False, alpha=1.0),
        # a ragged batch and an odd width (rows without 16-byte alignment), norms on both sides and a gate
        dict(name="norm_bwd_ragged", op="norm", grad=True, M=1777, h=5003, res="bf16", post=True, gate=True, alpha=0.25),
        # activations of a 2048-token batch, 8192 wide
        dict(name="dropout_elementwise", op="drop", M=2048, h=8192, p=0.1),
        # a 4096-wide attention projection with rank-16 adapters, 2048 tokens
        dict(name="dropout_linear_fwd", op="lin", grad=False, M=2048, h=4096, o=4096, r=16, p=0.05),
        # the backward of the same projection
        dict(name="dropout_linear_bwd", op="lin", grad=True, M=2048, h=4096, o=4096, r=16, p=0.05),
        # the backward of the widest feed-forward projection with rank-64 adapters
        dict(name="dropout_linear_bwd_wide", op="lin", grad=True, M=2048, h=8192, o=22016, r=64, p=0.1),
        # scoring a short answer: 16 tokens against a 32000-word vocabulary, bound by reading the head
        dict(name="loss_fwd_answer", op="loss", grad=False, M=16, h=4096, V=32000, ignored=0.0, train_head=False),
        # a training batch whose prompt tokens (a quarter) carry no loss, frozen head
        dict(name="loss_step_frozen", op="loss", grad=True, M=2048, h=8192, V=32000, ignored=0.25, train_head=False),
        # a ragged batch, a vocabulary that no tile divides, and a trained head
        dict(name="loss_step_ragged", op="loss", grad=True, M=1531, h=4096, V=50257, ignored=0.1, train_head=True),
        # the largest batch, trained head
        dict(name="loss_step_large", op="loss", grad=True, M=4096, h=8192, V=32000, ignored=0.0, train_head=True),
    ]


def _between(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], spread over the range's logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return min(hi, max(lo, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["norm", "norm", "drop", "lin", "lin", "loss", "loss"])
    if op == "norm":
        return dict(op=op, grad=rng.random() < 0.5, M=_between(rng, 1, 4096), h=_between(rng, 5, 16384),
                    res=rng.choice(["bf16", "f32"]), post=rng.random() < 0.5, gate=rng.random() < 0.5,
                    alpha=rng.choice([1.0, 0.5, 0.125]))
    if op == "drop":
        return dict(op=op, M=_between(rng, 1, 4096), h=_between(rng, 1, 11008), p=round(rng.uniform(0.0, 0.5), 3))
    if op == "lin":
        return dict(op=op, grad=rng.random() < 0.5, M=_between(rng, 1, 4096), h=_between(rng, 64, 8192, 64),
                    o=_between(rng, 64, 11008, 64), r=_between(rng, 1, 128), p=round(rng.uniform(0.0, 0.5), 3))
    return dict(op=op, grad=rng.random() < 0.6, M=_between(rng, 1, 4096), h=_between(rng, 64, 4096, 64),
                V=_between(rng, 100, 65536), ignored=rng.choice([0.0, 0.3, 0.75]), train_head=rng.random() < 0.5)


def _valid(case):
    """Tokens that carry a loss."""
    return case["M"] - int(case["ignored"] * case["M"])


def work(case):
    M, h = case["M"], case["h"]
    if case["op"] == "norm":
        b = 2 if case["res"] == "bf16" else 4
        weights = 4 * h * (1 + case["post"] + case["gate"])
        if not case["grad"]:
            return {"bytes": M * h * (4 + 2 * b) + weights + 4 * M * (1 + case["post"]),
                    "flops": M * h * (6 + 5 * case["post"])}
        y_read = 2 if case["post"] or case["gate"] else 0  # without them no gradient depends on Y
        return {"bytes": M * h * (4 + y_read + 3 * b) + 2 * weights + 4 * M * (1 + case["post"]),
                "flops": M * h * (12 + 10 * case["post"])}
    if case["op"] == "drop":
        return {"bytes": 4 * M * h, "flops": M * h}
    if case["op"] == "lin":
        o, r = case["o"], case["r"]
        codes = h * o // 2 + h * o // 64 + 4 * -(-h * o // 16384)
        factors = 2 * r * (h + o)
        if not case["grad"]:
            return {"bytes": codes + factors + 2 * M * (h + o + r), "flops": 2 * M * (h * o + r * (h + o))}
        return {"bytes": codes + factors + 2 * factors + 2 * M * (2 * h + o + r),
                "flops": 2 * M * (h * o + 2 * r * (h + o))}
    V, n = case["V"], _valid(case)
    parts = (1 + case["grad"] + (case["grad"] and case["train_head"]))
    return {"bytes": 2 * V * h * (1 + (case["grad"] and case["train_head"])) + 2 * n * h + 16 * M
            + (2 * M * h if case["grad"] else 0), "flops": 2 * n * V * h * parts}


# ---------------------------------------------------------------------------
# What a user's program has in hand
# ---------------------------------------------------------------------------


def _levels64():
    """The 16 NormalFloat levels: normal quantiles, 8 steps above zero and 7 below."""
    delta = (31.0 / 32.0 + 29.0 / 30.0) / 2.0
    up = torch.tensor([0.5 + (delta - 0.5) * k / 8.0 for k in range(1, 9)], dtype=torch.float64)
    down = torch.tensor([0.5 + (delta - 0.5) * k / 7.0 for k in range(7, 0, -1)], dtype=torch.float64)
    top = torch.special.ndtri(torch.tensor(delta, dtype=torch.float64))
    q = torch.cat([-torch.special.ndtri(down), torch.zeros(1, dtype=torch.float64), torch.special.ndtri(up)])
    return q / top


def _nf4_weight(o, h, gen):
    """A frozen weight [o][h] ~ N(0, 0.02) as its codes and double-quantized scales."""
    levels = _levels64()
    mids = ((levels[1:] + levels[:-1]) / 2).float().to(DEVICE)
    w = (torch.randn(o * h, generator=gen, device=DEVICE) * 0.02).view(-1, 64)
    amax = w.abs().amax(1)
    code = torch.bucketize((w / amax[:, None]).view(-1), mids, out_int32=True).to(torch.uint8).view(-1, 2)
    codes = code[:, 0] * 16 + code[:, 1]
    mean = amax.double().mean().float()
    n = amax.numel()
    c = torch.nn.functional.pad(amax - mean, (0, -n % 256)).view(-1, 256)
    scale2 = c.abs().amax(1) / 127.0
    step = torch.where(scale2 > 0, scale2, torch.ones_like(scale2))
    q = torch.round(c / step[:, None]).clamp(-127, 127).to(torch.int8).view(-1)[:n]
    return dict(codes=codes.contiguous(), qabsmax=q.contiguous(), scale2=scale2, mean=mean.reshape(1))


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    M, h = case["M"], case["h"]

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=gen, device=DEVICE) * std).to(dtype)

    s = dict(case=dict(case))
    if case["op"] == "norm":
        rt = torch.bfloat16 if case["res"] == "bf16" else torch.float32
        s["R"] = normal(M, h, std=2.0, dtype=rt)     # the residual stream (the stored result in a backward)
        s["Y"] = normal(M, h)                        # the block's output
        s["w_pre"] = 1 + normal(h, std=0.1, dtype=torch.float32)
        s["w_post"] = 1 + normal(h, std=0.1, dtype=torch.float32) if case["post"] else None
        s["gate"] = normal(h, std=0.5, dtype=torch.float32) if case["gate"] else None
        if case["grad"]:
            s["dN"] = normal(M, h)
            s["dR_out"] = normal(M, h, dtype=rt)
            s["rstd_pre"] = torch.rsqrt(s["R"].float().square().mean(1) + EPS)
            s["rstd_post"] = torch.rsqrt(s["Y"].float().square().mean(1) + EPS) if case["post"] else None
        return s
    if case["op"] == "loss":
        V = case["V"]
        s["H"] = normal(M, h)
        s["W"] = normal(V, h, std=0.02)
        labels = torch.randint(0, V, (M,), generator=gen, device=DEVICE)
        off = torch.randperm(M, generator=gen, device=DEVICE)[_valid(case):]
        labels[off] = IGNORED
        s["labels"] = labels
        if case["grad"]:
            s["dloss"] = torch.full((M,), 1.0 / _valid(case), device=DEVICE)  # the mean over the tokens with a loss
        return s
    # the generator's state lives on the GPU, so that a captured step can advance it
    s["rng"] = torch.tensor([seed * 2654435761 + 12345, 8 * seed + 3], dtype=torch.int64, device=DEVICE)
    s["X"] = normal(M, h)
    if case["op"] == "lin":
        o, r = case["o"], case["r"]
        s.update(_nf4_weight(o, h, gen), levels=_levels64().float().to(DEVICE))
        s["L1"], s["L2"], s["s"] = normal(h, r, std=0.01), normal(r, o, std=0.01), 0.25
        if case["grad"]:
            s["dY"] = normal(M, o)
            s["T"] = ((s["X"].float() * _keep(s["rng"], M * h, case["p"]).view(M, h)) @ s["L1"].float()).bfloat16()
    return s


# ---------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------


def _threshold(p):
    """Elements whose 16 random bits are below it are dropped; the rest are scaled by
    65536 / (65536 - threshold), so the result is unbiased at this probability."""
    return round(p * 65536)


def _philox(key, counter):
    """Philox 4x32 with 7 rounds (Salmon, Moraes, Dror and Shaw, 2011) on 64-bit
    counters: four 32-bit words each, in int64."""
    low = 0xFFFFFFFF
    k0, k1 = key & low, (key >> 32) & low
    x0, x1 = counter & low, (counter >> 32) & low
    x2, x3 = torch.zeros_like(x0), torch.zeros_like(x0)
    for _ in range(7):
        a, b = x0 * 0xD2511F53, x2 * 0xCD9E8D57  # the low 64 bits, which hold the whole product
        x0, x1, x2, x3 = ((b >> 32) & low) ^ x1 ^ k0, b & low, ((a >> 32) & low) ^ x3 ^ k1, a & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    return x0, x1, x2, x3


def _keep(rng, n, p):
    """Whether each of n elements is kept: element e has the (e % 8)-th 16-bit piece of
    the block with counter offset + e / 8."""
    blocks = torch.arange((n + 7) // 8, device=rng.device) + rng[1]
    words = torch.stack(_philox(rng[0], blocks), 1)
    bits = torch.stack((words & 0xFFFF, words >> 16), 2).view(-1)[:n]
    return bits >= _threshold(p)


def _w_hat(s):
    """The bf16 dequantization of the frozen weight, [o][h], in float32."""
    case = s["case"]
    codes = s["codes"].int()
    w = s["levels"][torch.stack((codes >> 4, codes & 15), 1).view(-1)].view(-1, 64)
    q = s["qabsmax"].float()
    a = q * s["scale2"].repeat_interleave(256)[: q.numel()] + s["mean"]
    return (w * a[:, None]).bfloat16().float().view(case["o"], case["h"])


def _plain_norm(s):
    case, alpha = s["case"], s["case"]["alpha"]
    R, Y = s["R"].float(), s["Y"].float()
    g = alpha if s["gate"] is None else alpha * s["gate"]
    if not case["grad"]:
        rstd_post, u = None, Y
        if case["post"]:
            rstd_post = torch.rsqrt(Y.square().mean(1) + EPS)
            u = Y * rstd_post[:, None] * s["w_post"]
        r = R + g * u
        rstd_pre = torch.rsqrt(r.square().mean(1) + EPS)
        n = r * rstd_pre[:, None] * s["w_pre"]
        return dict(R_out=r.to(s["R"].dtype), N=n.bfloat16(), rstd_pre=rstd_pre, rstd_post=rstd_post)
    dN, x = s["dN"].float(), R * s["rstd_pre"][:, None]
    d = dN * s["w_pre"]
    dr = s["dR_out"].float() + s["rstd_pre"][:, None] * (d - x * (d * x).mean(1, keepdim=True))
    out = dict(dR=dr.to(s["R"].dtype), dw_pre=(dN * x).sum(0))
    du, u = dr * g, Y
    if case["post"]:
        y = Y * s["rstd_post"][:, None]
        u = y * s["w_post"]
        out["dw_post"] = (du * y).sum(0)
        d = du * s["w_post"]
        out["dY"] = (s["rstd_post"][:, None] * (d - y * (d * y).mean(1, keepdim=True))).bfloat16()
    else:
        out["dY"] = du.bfloat16()
    if case["gate"]:
        out["dgate"] = (alpha * dr * u).sum(0)
    return out


def _plain_lin(s):
    case = s["case"]
    M, h, p = case["M"], case["h"], case["p"]
    keep = _keep(s["rng"], M * h, p).view(M, h).float()
    scale = s["s"] * 65536.0 / (65536 - _threshold(p))
    X, L1, L2, W = s["X"].float(), s["L1"].float(), s["L2"].float(), _w_hat(s)
    if not case["grad"]:
        T = (X * keep) @ L1
        return dict(Y=(X @ W.t() + scale * (T @ L2)).bfloat16(), T=T.bfloat16())
    dY = s["dY"].float()
    U = dY @ L2.t()
    return dict(dX=(dY @ W + scale * keep * (U @ L1.t())).bfloat16(), dL1=scale * ((X * keep).t() @ U),
                dL2=scale * (s["T"].float().t() @ dY))


def _plain_loss(s):
    case = s["case"]
    H, W, labels = s["H"].float(), s["W"].float(), s["labels"]
    live = (labels >= 0) & (labels < case["V"])
    at = torch.where(live, labels, torch.zeros_like(labels))[:, None]
    z = H @ W.t()
    top = z.amax(1, keepdim=True)
    e = torch.exp(z - top)
    total = e.sum(1, keepdim=True)
    lse = (top + torch.log(total))[:, 0]
    zero = torch.zeros_like(lse)
    out = dict(loss=torch.where(live, lse - z.gather(1, at)[:, 0], zero), lse=torch.where(live, lse, zero))
    if case["grad"]:
        G = e / total
        G.scatter_add_(1, at, -torch.ones_like(lse)[:, None])
        G = G * torch.where(live, s["dloss"], zero)[:, None]
        out["dH"] = (G @ W).bfloat16()
        if case["train_head"]:
            out["dW"] = (G.t() @ H).bfloat16()
    return out


def _plain(s):
    case = s["case"]
    if case["op"] == "norm":
        return _plain_norm(s)
    if case["op"] == "loss":
        return _plain_loss(s)
    if case["op"] == "lin":
        return _plain_lin(s)
    keep = _keep(s["rng"], case["M"] * case["h"], case["p"]).view(case["M"], case["h"])
    return (s["X"].float() * keep * (65536.0 / (65536 - _threshold(case["p"])))).bfloat16()


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------


def _framework(s):
    import bit_quantized_fine_nf4_amd as nf4

    case = s["case"]
    if case["op"] == "norm":
        weights = dict(w_pre=s["w_pre"], w_post=s["w_post"], gate=s["gate"], alpha=case["alpha"])
        if not case["grad"]:
            R_out, N, rstd_pre, rstd_post = nf4.qlora_norm_fwd(s["R"], s["Y"], eps=EPS, **weights)
            return dict(R_out=R_out, N=N, rstd_pre=rstd_pre, rstd_post=rstd_post)
        dR, dY, dw_pre, dw_post, dgate = nf4.qlora_norm_bwd(
            s["dN"], s["dR_out"], s["R"], s["Y"], s["rstd_pre"], s["rstd_post"], weight_grads=True, **weights)
        return {k: v for k, v in dict(dR=dR, dY=dY, dw_pre=dw_pre, dw_post=dw_post, dgate=dgate).items()
                if v is not None}
    if case["op"] == "drop":
        return nf4.qlora_dropout(s["X"], case["p"], s["rng"])
    if case["op"] == "lin":
        W = nf4.NF4Weight(s["codes"], s["qabsmax"], s["scale2"], s["mean"], case["h"], case["o"])
        if not case["grad"]:
            Y, T = nf4.qlora_linear_fwd_dropout(W, s["X"], s["L1"], s["L2"], s["s"], case["p"], s["rng"])
            return dict(Y=Y, T=T)
        dX, dL1, dL2 = nf4.qlora_linear_bwd_dropout(W, s["X"], s["T"], s["dY"], s["L1"], s["L2"], s["s"],
                                                    case["p"], s["rng"])
        return dict(dX=dX, dL1=dL1, dL2=dL2)
    loss, lse = nf4.qlora_loss_fwd(s["H"], s["W"], s["labels"])
    out = dict(loss=loss, lse=lse)
    if case["grad"]:
        dH, dW = nf4.qlora_loss_bwd(s["H"], s["W"], s["labels"], lse, s["dloss"], train_head=case["train_head"])
        out["dH"] = dH
        if case["train_head"]:
            out["dW"] = dW
    return out


def run(state):
    return _framework(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------


def _kept64(rng, n, p):
    """The kept elements, from the generator's definition in NumPy's unsigned integers."""
    seed, offset = (int(v) % (1 << 64) for v in rng.tolist())
    count = np.arange(-(-n // 8), dtype=np.uint64) + np.uint64(offset)
    word = [(count & np.uint64(0xFFFFFFFF)), count >> np.uint64(32), np.zeros_like(count), np.zeros_like(count)]
    for i in range(7):
        key = [np.uint64((seed + i * 0x9E3779B9) % (1 << 32)), np.uint64(((seed >> 32) + i * 0xBB67AE85) % (1 << 32))]
        first, second = word[0] * np.uint64(0xD2511F53), word[2] * np.uint64(0xCD9E8D57)
        word = [(second >> np.uint64(32)) ^ word[1] ^ key[0], second & np.uint64(0xFFFFFFFF),
                (first >> np.uint64(32)) ^ word[3] ^ key[1], first & np.uint64(0xFFFFFFFF)]
    halves = np.stack([w.astype(np.uint32) for w in word], 1).view(np.uint16).reshape(-1)[:n]  # low half first
    return torch.from_numpy(halves.astype(np.int32) >= int(round(p * 65536))).to(DEVICE)


def _exact_norm(s):
    case = s["case"]
    d = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor)}
    alpha = case["alpha"]
    gate = d.get("gate", torch.ones(case["h"], dtype=torch.float64, device=DEVICE))
    if not case["grad"]:
        block = d["Y"]
        rstd_post = None
        if case["post"]:
            rstd_post = 1 / torch.sqrt((block ** 2).mean(-1) + EPS)
            block = torch.einsum("mh,m,h->mh", block, rstd_post, d["w_post"])
        r = d["R"] + alpha * gate * block
        rstd_pre = 1 / torch.sqrt((r ** 2).mean(-1) + EPS)
        return dict(R_out=r, N=torch.einsum("mh,m,h->mh", r, rstd_pre, d["w_pre"]), rstd_pre=rstd_pre,
                    rstd_post=rstd_post)
    h = case["h"]
    rp = d["rstd_pre"][:, None]
    # d/dr of w_h r_h (mean r^2 + eps)^(-1/2): rstd w_h on the diagonal, -rstd^3 / h in r r^T
    dot = (d["dN"] * d["w_pre"] * d["R"]).sum(-1, keepdim=True)
    dr = d["dR_out"] + rp * d["w_pre"] * d["dN"] - rp ** 3 / h * dot * d["R"]
    out = dict(dR=dr, dw_pre=(d["dN"] * d["R"] * rp).sum(0))
    dblock = alpha * gate * dr
    if not case["post"]:
        out["dY"], block = dblock, d["Y"]
    else:
        rq = d["rstd_post"][:, None]
        dot = (dblock * d["w_post"] * d["Y"]).sum(-1, keepdim=True)
        out["dY"] = rq * d["w_post"] * dblock - rq ** 3 / h * dot * d["Y"]
        out["dw_post"] = (dblock * d["Y"] * rq).sum(0)
        block = d["Y"] * rq * d["w_post"]
    if case["gate"]:
        out["dgate"] = alpha * (dr * block).sum(0)
    return out


def _exact_lin(s):
    case = s["case"]
    M, h, o, p = case["M"], case["h"], case["o"], case["p"]
    t = int(round(p * 65536))
    scale = s["s"] * (65536 / (65536 - t))
    kept = _kept64(s["rng"], M * h, p).view(M, h).double()
    table = _levels64().float().to(DEVICE)
    byte = s["codes"].long()
    w = torch.empty(o * h, device=DEVICE)
    w[0::2], w[1::2] = table[byte // 16], table[byte % 16]
    nb = o * h // 64
    block = torch.arange(nb, device=DEVICE)
    # the rebuilt scale and the weight are rounded where the format says: float32 twice, then bf16
    a = s["qabsmax"].float() * s["scale2"][block // 256]
    a = a + s["mean"]
    W = (w.view(nb, 64) * a[:, None]).to(torch.bfloat16).double().view(o, h)
    X, L1, L2 = s["X"].double(), s["L1"].double(), s["L2"].double()
    if not case["grad"]:
        T = (kept * X).mm(L1)
        return dict(Y=X.mm(W.t()) + scale * T.mm(L2), T=T)
    dY = s["dY"].double()
    U = dY.mm(L2.t())
    return dict(dX=dY.mm(W) + scale * kept * U.mm(L1.t()), dL1=scale * (kept * X).t().mm(U),
                dL2=scale * s["T"].double().t().mm(dY))


def _exact_loss(s):
    case = s["case"]
    M, V = case["M"], case["V"]
    rows = torch.nonzero((s["labels"] >= 0) & (s["labels"] < V))[:, 0]
    H, W, label = s["H"][rows].double(), s["W"].double(), s["labels"][rows]
    logp = torch.log_softmax(H.mm(W.t()), 1)
    picked = logp[torch.arange(rows.numel(), device=DEVICE), label]
    z = (H * W[label]).sum(1)
    loss = torch.zeros(M, dtype=torch.float64, device=DEVICE)
    lse = torch.zeros(M, dtype=torch.float64, device=DEVICE)
    loss[rows], lse[rows] = -picked, z - picked
    out = dict(loss=loss, lse=lse)
    if case["grad"]:
        G = logp.exp_()
        G[torch.arange(rows.numel(), device=DEVICE), label] -= 1
        G *= s["dloss"][rows].double()[:, None]
        dH = torch.zeros(M, case["h"], dtype=torch.float64, device=DEVICE)
        dH[rows] = G.mm(W)
        out["dH"] = dH
        if case["train_head"]:
            out["dW"] = G.t().mm(H)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(s)
    if case["op"] == "loss":
        return _exact_loss(s)
    if case["op"] == "lin":
        return _exact_lin(s)
    kept = _kept64(s["rng"], case["M"] * case["h"], case["p"]).view(case["M"], case["h"])
    return torch.where(kept, s["X"].double() * 65536 / (65536 - int(round(case["p"] * 65536))), 0.0)
