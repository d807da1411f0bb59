"""Attention over spans in float64 with bounds on the GPU's results, for the tests of its edges.

Bounds, with u = 2^-24, r = 2^-8 (half a bf16 step) and n the number of keys or rows summed:
  z    ez = 2 d u sum scale|q||k| + 8 u (|z| + |lse|), with a cap 16 u |z| more, with a bias
       4 u |slope| |i - j| more
  p    relative: ep = ez + 8 u, and where lse enters (backward) el more
  lse  el = max ep + (n + 64) u + 4 u |lse|
  O    sum p (ep + r + 2 n u) |v| + |O| (max ep + (n + 64) u) + r |O|
  D    eD = sum |dO| eO + 2 d u sum |dO||O|, or summed from p and dP (`own`, a truth value a row):
       sum p |dP| (ep + el + 2 n u) + 2 d u sum p |dO||v|
  dS   eS = |dS| (ep + r + 4 u) + p (2 d u sum |dO||v| + eD), with a cap 32 u p |dP - D| more
  dQ   scale sum eS |k| + 2 n u scale sum |dS||k| + r |dQ|;  dK alike over rows and heads;
  dV   sum p (ep + r + 2 n u) |dO| + r |dV|
all times 1 + 2^-5 for the products of two errors; a sum may lose n 2^-120 by underflow.

A capped score z = cap tanh(t), t = x / cap, is within 16 u of itself, whatever the cap.  With
t2 = 2 t log2(e) off by 4 u (two roundings of the factor, a quotient's, the product's):
  small t: t2 P(t2^2), a polynomial with a factor of 3 u, and a product: 8 u;
  large t, |tanh| >= 0.46: exp(2 t) is off by 8 |t| u for t2 and 2 u of its own, and
     1 - 2 / (e + 1) by half of that times 1 - tanh^2, at most 4 u tanh + 1.7 u tanh, by the
     reciprocal's 2 u (1 - tanh) <= 2.4 u tanh, and a rounding u: under 10 u;
and the factor cap log2(e) and its product 3 u.  Its slope 1 - tanh^2 is off by twice that."""
import numpy as np
import torch

U, R = 2.0 ** -24, 2.0 ** -8
TINY = 2.0 ** -120
BF = torch.bfloat16
DEV = "cuda:0"


def problem(M, hq, hk, d, spans, seed=0, std=1.5):
    g = torch.Generator().manual_seed(1000 * seed + 7 * M + 3 * hq + d)
    n = lambda h, s=1.0: (torch.randn(M, h, d, generator=g) * s).to(BF).to(DEV)
    return dict(Q=n(hq, std), K=n(hk), V=n(hk), dO=n(hq),
                spans=torch.as_tensor(np.asarray(spans), dtype=torch.int32).to(DEV))


def run(nf4, p, **form):
    O, lse = nf4.qlora_attn_fwd(p["Q"], p["K"], p["V"], p["spans"], **form)
    dQ, dK, dV = nf4.qlora_attn_bwd(p["dO"], p["Q"], p["K"], p["V"], O, lse, p["spans"], **form)
    return dict(O=O, lse=lse, dQ=dQ, dK=dK, dV=dV)


def reference(p, scale, cap=0.0, slopes=None, own=None):
    """Results and bounds, head by head."""
    Q, K, V, dO = (p[x].double() for x in ("Q", "K", "V", "dO"))
    M, hq, d = Q.shape
    group = hq // K.shape[1]
    j = torch.arange(M, device=DEV)
    seen = (j >= p["spans"][:, :1]) & (j < p["spans"][:, 1:])
    any_ = seen.any(1)
    own = torch.zeros_like(any_) if own is None else torch.as_tensor(own, device=DEV).expand(M)
    away = (j[:, None] - j).abs().double()
    out = {k: torch.zeros_like(x) for k, x in dict(O=Q, dQ=Q, dK=K, dV=V).items()}
    out["lse"] = torch.zeros(hq, M, dtype=torch.float64, device=DEV)
    err = {k: torch.zeros_like(x) for k, x in out.items()}
    nk, nq = float(seen.sum(1).max()), float(seen.sum(0).max()) * group
    for h in range(hq):
        g = h // group
        q, k, v, do = Q[:, h], K[:, g], V[:, g], dO[:, h]
        z = scale * q @ k.t()
        ez = 2 * d * U * scale * (q.abs() @ k.abs().t())
        slack = torch.ones_like(z)
        if cap:
            th = torch.tanh(z / cap)
            z, slack = cap * th, 1 - th * th
            ez = ez + 16 * U * z.abs()
        if slopes is not None:
            z = z - slopes[h].double() * away
            ez = ez + 4 * U * slopes[h].double().abs() * away
        z = z.masked_fill(~seen, -torch.inf)
        lse = torch.logsumexp(z, 1)
        safe = torch.where(any_, lse, 0.0)
        w = torch.where(seen, torch.exp(z - safe[:, None]), 0.0)
        ep = torch.where(seen, ez + 8 * U * (1 + torch.where(seen, z.abs(), 0.0) + safe.abs()[:, None]), 0.0)
        top = ep.amax(1)
        el = top + (nk + 64) * U + 4 * U * safe.abs()
        O = w @ v
        eO = (w * (ep + R + 2 * nk * U)) @ v.abs() + O.abs() * (top + (nk + 64) * U)[:, None] + R * O.abs()
        out["lse"][h], err["lse"][h] = torch.where(any_, lse, -torch.inf), el
        out["O"][:, h], err["O"][:, h] = O, eO + nk * TINY
        eb = ep + el[:, None]
        dP, most = do @ v.t(), do.abs() @ v.abs().t()
        eD = (do.abs() * eO).sum(1) + 2 * d * U * (do.abs() * O.abs()).sum(1)
        eD = torch.where(own, (w * ((eb + 2 * nk * U) * dP.abs() + 2 * d * U * most)).sum(1), eD)
        rest = dP - (do * O).sum(1, keepdim=True)
        dS = w * rest * slack
        eS = dS.abs() * (eb + R + 4 * U) + w * (2 * d * U * most + eD[:, None])
        if cap:
            eS = eS + 32 * U * w * rest.abs()
        out["dQ"][:, h] = scale * dS @ k
        err["dQ"][:, h] = scale * ((eS + 2 * nk * U * dS.abs()) @ k.abs()) + nk * TINY
        out["dK"][:, g] += scale * dS.t() @ q
        err["dK"][:, g] += scale * ((eS + 2 * nq * U * dS.abs()).t() @ q.abs()) + nq * TINY
        out["dV"][:, g] += w.t() @ do
        err["dV"][:, g] += (w * (eb + R + 2 * nq * U)).t() @ do.abs() + nq * TINY
    for k in ("dQ", "dK", "dV"):
        err[k] += R * out[k].abs()
    return out, {k: e * (1 + 2.0 ** -5) for k, e in err.items()}


def check(got, ref, norms=None):
    """Every value within its bound, and each tensor within `norms` of its norm, 1e-2 (the
    tolerance of the framework's bf16 outputs) where it has none there."""
    out, err = ref
    for name, x in got.items():
        x, y = x.double(), out[name]
        if name == "lse":
            assert torch.equal(x == -torch.inf, y == -torch.inf), name
            x, y = torch.where(y == -torch.inf, 0.0, x), torch.where(y == -torch.inf, 0.0, y)
        off = (x - y).abs()
        bad = ~(off <= err[name])
        assert not bad.any(), (name, int(bad.sum()), bad.nonzero()[:3].tolist(), x[bad][:3].tolist(), y[bad][:3].tolist())
        if y.norm() > 0 and name != "lse":
            far = float((x - y).norm() / y.norm())
            assert far <= (norms or {}).get(name, 1e-2), (name, far)
