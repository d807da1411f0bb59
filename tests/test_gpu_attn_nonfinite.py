"""Infinities and NaN in attention: they reach every result that the formulas let them reach,
and no other value changes by a bit.  Of a NaN at one value e of

  Q_i    the whole rows i of O, lse and dQ; dK and dV of the keys that i sees
  K_j    the whole rows of O, lse and dQ of the queries that see j; dK and dV of the keys that
         such a query sees
  V_j    value e of the queries' O; their dQ, and dK of the keys that they see (through D); dV
         stays
  dO_i   dQ of i, dK of the keys that i sees, and value e of their dV

A key whose scores are all -inf has the weight zero: as if it were not seen, but for 0 * inf at
its value e of dQ."""
import pytest
import torch

import oracle
from attention_bounds import BF, DEV, problem, run

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import bit_quantized_fine_nf4_amd as nf4  # noqa: E402

NAN, INF = float("nan"), float("inf")
# heads of 64 and 128 values and narrower ones; one and two groups of waves, and dK's and dV's
# sums in one, two and several parts, by workgroups (those of 128 queries or keys times heads)
SHAPES = [(150, 2, 1, 64, 0.0), (300, 4, 2, 128, 0.0), (300, 4, 4, 40, 5.0), (1300, 52, 52, 64, 0.0),
          (1100, 64, 64, 128, 0.0), (700, 12, 2, 64, 0.0)]


def spans_of(kind, M):
    if kind == "causal":
        return oracle.spans([0, M], M)
    s = oracle.spans([0, M // 3, M], M, causal=False)          # whole documents, and rows without a key
    s[M // 5:M // 5 + 9] = 0
    return s


def expect(p, what, at, hk_of):
    """Where a value of each result must not be finite."""
    M, hq, d = p["Q"].shape
    hk = p["K"].shape[1]
    i, h, e = at
    j = torch.arange(M, device=DEV)
    seen = (j >= p["spans"][:, :1]) & (j < p["spans"][:, 1:])
    bad = dict(O=torch.zeros(M, hq, d, dtype=torch.bool, device=DEV), lse=torch.zeros(hq, M, dtype=torch.bool, device=DEV),
               dK=torch.zeros(M, hk, d, dtype=torch.bool, device=DEV))
    bad["dQ"], bad["dV"] = torch.zeros_like(bad["O"]), torch.zeros_like(bad["dK"])
    if what in ("Q", "dO"):
        if not bool(seen[i].any()):
            return bad
        rows, heads, g = torch.zeros(M, dtype=torch.bool, device=DEV), [h], hk_of(h)
        rows[i] = True
    else:
        rows, g = seen[:, i], h
        heads = [x for x in range(hq) if hk_of(x) == h]
    keys = seen[rows].any(0)
    for x in heads:
        bad["dQ"][rows, x] = True
        if what in ("Q", "K"):
            bad["O"][rows, x], bad["lse"][x, rows] = True, True
        elif what == "V":
            bad["O"][rows, x, e] = True
    bad["dK"][keys, g] = True
    if what == "dO":
        bad["dV"][keys, g, e] = True
    elif what != "V":
        bad["dV"][keys, g] = True
    return bad


def compare(got, clean, bad):
    for k, x in got.items():
        finite = torch.isfinite(x)
        wrong = torch.isfinite(clean[k]) & (finite == bad[k])
        assert not wrong.any(), (k, int(wrong.sum()), wrong.nonzero()[:4].tolist(), int(bad[k].sum()))
        keep = ~bad[k]
        assert torch.equal(x[keep], clean[k][keep]), k


def spoiled(M, hq, hk, d, cap, kind, what, value, results):
    """Results of a problem with one value that is not finite, here and there, against those without."""
    print(f"attn nonfinite M={M} hq={hq} hk={hk} d={d} cap={cap} {kind} {what} {value}", flush=True)
    p = problem(M, hq, hk, d, spans_of(kind, M))
    call = (lambda q: run(nf4, q, cap=cap)) if "dQ" in results else (
        lambda q: dict(zip(("O", "lse"), nf4.qlora_attn_fwd(q["Q"], q["K"], q["V"], q["spans"], cap=cap))))
    clean = call(p)
    heads = hq if what in ("Q", "dO") else hk
    for i, h, e in ((3, 0, 0), (M // 2 + 1, heads - 1, d - 1), (M - 1, heads // 2, 5), (70, 0, d // 2), (M // 5 + 2, 0, 1)):
        q = dict(p)
        q[what] = p[what].clone()
        q[what][i, h, e] = value
        bad = expect(p, what, (i, h, e), lambda x: x // (hq // hk))
        got = call(q)
        compare({k: got[k] for k in results}, clean, bad)


@pytest.mark.parametrize("what", ["Q", "K"])
@pytest.mark.parametrize("kind", ["causal", "documents"])
@pytest.mark.parametrize("M,hq,hk,d,cap", SHAPES)
def test_rows_of_a_nan(M, hq, hk, d, cap, kind, what):
    spoiled(M, hq, hk, d, cap, kind, what, NAN, ("O", "lse"))


@pytest.mark.parametrize("value", [NAN, INF, -INF])
@pytest.mark.parametrize("kind", ["causal", "documents"])
@pytest.mark.parametrize("M,hq,hk,d,cap", SHAPES)
def test_columns_of_a_value(M, hq, hk, d, cap, kind, value):
    spoiled(M, hq, hk, d, cap, kind, "V", value, ("O", "lse"))


@pytest.mark.parametrize("what,value", [("Q", NAN), ("K", NAN), ("V", NAN), ("V", INF), ("dO", NAN), ("dO", INF)])
@pytest.mark.parametrize("kind", ["causal", "documents"])
@pytest.mark.parametrize("M,hq,hk,d,cap", SHAPES)
def test_gradients(M, hq, hk, d, cap, kind, what, value):
    spoiled(M, hq, hk, d, cap, kind, what, value, ("dQ", "dK", "dV"))


@pytest.mark.parametrize("M,hq,hk,d,cap", [s for s in SHAPES if s[4] == 0.0])
def test_scores_of_minus_infinity(M, hq, hk, d, cap):
    p = problem(M, hq, hk, d, oracle.spans([0, M], M))
    j, e = M // 2 + 1, 7
    p["Q"][:, :, e] = -1.0
    p["K"][j, :, e] = INF                                      # every score of key j: -inf
    got = run(nf4, p)
    seen = torch.arange(M, device=DEV) >= j
    for k in ("O", "lse", "dV"):
        assert bool(torch.isfinite(got[k]).all()), k
    assert not got["dV"][j].any() and not got["dK"][j].any()
    bad = torch.zeros_like(got["dQ"], dtype=torch.bool)
    bad[seen, :, e] = True
    assert torch.equal(~torch.isfinite(got["dQ"]), bad)
    # the same without that key: spans cannot leave one key out, so the formulas in float64
    q, k, v, do = (p[x].double() for x in ("Q", "K", "V", "dO"))
    k, v = k.repeat_interleave(hq // hk, 1), v.repeat_interleave(hq // hk, 1)
    row = M - 1
    keep = torch.arange(M, device=DEV) != j
    z = d ** -0.5 * torch.einsum("hd,jhd->hj", q[row], k[keep])
    w = torch.softmax(z, 1)
    O = torch.einsum("hj,jhd->hd", w, v[keep])
    dP = torch.einsum("hd,jhd->hj", do[row], v[keep])
    dS = w * (dP - (w * dP).sum(1, keepdim=True))
    dQ = d ** -0.5 * torch.einsum("hj,jhd->hd", dS, k[keep])
    at = torch.arange(d, device=DEV) != e
    assert float((got["O"][row] - O).norm() / O.norm()) < 1e-2
    assert float((got["dQ"][row][:, at] - dQ[:, at]).norm() / dQ[:, at].norm()) < 1e-2


def test_one_new_token():
    """The same of one new token: a NaN of a query or a seen key reaches its whole row, of a
    value its value."""
    B, hq, hk, d, page, width = 4, 4, 2, 64, 16, 40
    g = torch.Generator().manual_seed(11)
    k, v = (torch.randn(B * width, hk, page, d, generator=g).to(BF).to(DEV) for _ in range(2))
    table = torch.randperm(B * width, generator=g).view(B, width).to(torch.int32).to(DEV)
    lens = torch.tensor([3, 129, 640, 0], dtype=torch.int32, device=DEV)
    q = torch.randn(B, hq, d, generator=g).to(BF).to(DEV)
    call = lambda q, k, v: nf4.qlora_decode_attn(q, k, v, table, lens)
    clean = call(q, k, v)
    for b, n in enumerate(lens.tolist()):
        spoiled = q.clone()
        spoiled[b, 1, 3] = NAN
        bad = torch.zeros_like(clean, dtype=torch.bool)
        bad[b, 1] = n > 0
        compare(dict(O=call(spoiled, k, v)), dict(O=clean), dict(O=bad))
        for j in {0, n // 2, n - 1} if n else ():
            at = (int(table[b, j // page]), 1, j % page, 9)
            spoiled = k.clone()
            spoiled[at] = NAN
            bad = torch.zeros_like(clean, dtype=torch.bool)
            bad[b, 2:] = True
            compare(dict(O=call(q, spoiled, v)), dict(O=clean), dict(O=bad))
            spoiled = v.clone()
            spoiled[at] = INF
            bad = torch.zeros_like(clean, dtype=torch.bool)
            bad[b, 2:, 9] = True
            compare(dict(O=call(q, k, spoiled)), dict(O=clean), dict(O=bad))
