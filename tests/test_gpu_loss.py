"""GPU parity of the cross entropy without kept logits (qlora_loss_fwd, qlora_loss_bwd)
against float64.

Bounds, with u = 2^-24 and mag(z) = sum |H||W| of a logit:
  z     ez = 2 h u mag(z): h float32 additions; the factor 2 because the matrix cores'
        internal rounding is not specified as to-nearest
  lse   el = max ez + (256 + 4 range(z)) u + 2 u |lse|: at most 64 additions per lane and
        tile, 8 joins and one wave's sum of tiles (under 256 in all); an exponential's
        argument is rounded twice, relative to its size, and the exponential once
  loss  el + ez + u |loss|
  G     P (ez + el + (4 + 2 |z - lse|) u) |dloss| + 6 u |G| (dloss over the largest and
        back, each a few roundings), then half a bf16 step 2^-8 |G|
  dH    sum |error of G| |W| + 2 (V + 32) u sum |G||W|, then 2^-8 |dH|; dW alike over tokens
(the 32: partial sums of the vocabulary's splits).
Underflow: a float32 below TINY = 2^-126 may be flushed to 0 (the hardware exponential
and the matrix cores flush subnormals), an error of at most TINY.  P, its product with
dloss / max |dloss| and its bf16 operand each may: TINY (|dloss| + 2 max |dloss|) more on
G, which the products carry on through |W| or |H| as above; and TINY on each result."""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import bit_quantized_fine_nf4_amd as nf4  # noqa: E402

DEV = "cuda:0"
U = 2.0 ** -24
TINY = 2.0 ** -126
BF = torch.bfloat16


def problem(M, h, V, skip, scale=1.0, seed=0):
    g = torch.Generator().manual_seed(17 * M + 3 * h + V + 1000 * seed)
    H = (torch.randn(M, h, generator=g) * scale).to(BF)
    W = (torch.randn(V, h, generator=g) * 0.2).to(BF)
    labels = torch.randint(0, V, (M,), generator=g)
    labels[0], labels[-1] = V - 1, 0          # the ends of the vocabulary
    if skip == "some":
        labels[torch.rand(M, generator=g) < 0.4] = -100
        labels[M // 2] = V                     # one past the last word
    elif skip == "most":
        labels[: M - 1] = -1
    elif skip == "all":
        labels[:] = -100
    dead = (labels < 0) | (labels >= V)
    H[dead] = float("nan")                     # prompt rows may hold anything
    if skip == "some" and M > 4:
        H[dead.nonzero()[0, 0]] = float("inf")
    dl = torch.randn(M, generator=g)
    dl[dead] = float("nan")
    return H, W, labels, dl


def reference(H, W, labels, dl):
    """Values and bounds, in float64 on the tensors' device."""
    H, W, dl = H.double(), W.double(), dl.double()
    V, h = W.shape
    live = ((labels >= 0) & (labels < V)).nonzero()[:, 0]
    H, dl, y = H[live], dl[live], labels[live]
    row = torch.arange(len(live), device=H.device)
    z, mag = H @ W.t(), H.abs() @ W.t().abs()
    ez = 2 * h * U * mag
    lse = torch.logsumexp(z, 1)
    el = ez.amax(1) + (256 + 4 * (z.amax(1) - z.amin(1))) * U + 2 * U * lse.abs() if len(live) else lse
    loss = lse - z[row, y]
    P = torch.exp(z - lse[:, None])
    eG = P * (ez + el[:, None] + (4 + 2 * (z - lse[:, None]).abs()) * U)
    G = P.clone()
    G[row, y] -= 1
    G, eG = G * dl[:, None], eG * dl.abs()[:, None]
    top = dl.abs().max() if len(live) else 0.0
    eG = eG + (2.0 ** -8 + 6 * U) * G.abs() + TINY * (dl.abs()[:, None] + 2 * top)
    dH, dW = G @ W, G.t() @ H
    eH = eG @ W.abs() + 2 * (V + 32) * U * (G.abs() @ W.abs()) + 2.0 ** -8 * dH.abs()
    eW = eG.t() @ H.abs() + 2 * (len(live) + 32) * U * (G.abs().t() @ H.abs()) + 2.0 ** -8 * dW.abs()
    return live, dict(loss=(loss, el + ez[row, y] + U * loss.abs()), lse=(lse, el), dH=(dH, eH), dW=(dW, eW))


def check(name, got, ref, bound):
    err = (got.double() - ref).abs()
    bad = ~(err <= bound + TINY)
    assert not bad.any(), (name, int(bad.sum()), bad.nonzero()[:3].tolist(), got[bad][:3].tolist(), ref[bad][:3].tolist())


def run(H, W, labels, dl):
    loss, lse = nf4.qlora_loss_fwd(H, W, labels)
    dH, dW = nf4.qlora_loss_bwd(H, W, labels, lse, dl, train_head=True)
    frozen, none = nf4.qlora_loss_bwd(H, W, labels, lse, dl)
    assert none is None and torch.equal(frozen, dH)
    return dict(loss=loss, lse=lse, dH=dH, dW=dW)


def compare(got, H, W, labels, dl):
    live, ref = reference(H, W, labels, dl)
    dead = torch.ones(len(labels), dtype=torch.bool, device=labels.device)
    dead[live] = False
    for k in ("loss", "lse", "dH"):
        assert torch.all(got[k][dead] == 0), k
        check(k, got[k][live], *ref[k])
    check("dW", got["dW"], *ref["dW"])


SHAPES = [(1, 64, 1), (1, 64, 100), (1, 1024, 3001), (3, 128, 129), (16, 192, 1000), (31, 64, 128), (32, 64, 257),
          (33, 64, 300), (64, 256, 511), (65, 128, 512), (128, 64, 700), (129, 320, 513), (300, 256, 1000),
          (257, 64, 5000), (513, 576, 770), (1024, 64, 300), (1025, 64, 300),
          (300, 192, 30011), (513, 256, 13500)]


@pytest.mark.parametrize("skip", ["none", "some", "most", "all"])
@pytest.mark.parametrize("M,h,V", SHAPES)
def test_parity(M, h, V, skip):
    print(f"loss M={M} h={h} V={V} skip={skip}", flush=True)
    t = [x.to(DEV) for x in problem(M, h, V, skip)]
    compare(run(*t), *t)


def test_against_the_oracle():
    M, h, V = 21, 128, 333
    H, W, labels, dl = problem(M, h, V, "some")
    got = run(*(x.to(DEV) for x in (H, W, labels, dl)))
    H, W, dl, y = H.double().numpy(), W.double().numpy(), dl.double().numpy(), labels.tolist()
    loss, lse = oracle.loss_fwd(H, W, y)
    dH, dW = oracle.loss_bwd(H, W, y, dl)
    for k, ref in (("loss", loss), ("lse", lse), ("dH", dH), ("dW", dW)):
        g = got[k].cpu().double().numpy()
        assert np.linalg.norm(g - ref) <= (1e-2 if g.ndim == 2 else 1e-5) * np.linalg.norm(ref), k


@pytest.mark.parametrize("scale", [1e-3, 40.0])
def test_flat_and_peaked_distributions(scale):
    """Logits near zero, and logits of hundreds, whose exponentials underflow."""
    t = [x.to(DEV) for x in problem(70, 256, 900, "some", scale)]
    compare(run(*t), *t)


def test_mean_gradient_is_no_worse_than_its_rounding():
    """One dloss for all tokens: what is left is dH's own rounding (2^-8 at most, under
    1.8e-3 of the norm for values spread over a binade)."""
    H, W, labels, _ = (x.to(DEV) for x in problem(300, 256, 2000, "none"))
    dl = torch.full((300,), 1 / 300, device=DEV)
    _, lse = nf4.qlora_loss_fwd(H, W, labels)
    dH, dW = nf4.qlora_loss_bwd(H, W, labels, lse, dl, train_head=True)
    _, ref = reference(H, W, labels, dl)
    for got, (r, _) in ((dH, ref["dH"]), (dW, ref["dW"])):
        assert torch.linalg.norm(got.double() - r) <= 2.2e-3 * torch.linalg.norm(r)
    zero, _ = nf4.qlora_loss_bwd(H, W, labels, lse, 0 * dl)
    assert torch.all(zero == 0)


@pytest.mark.parametrize("h", [64, 192])
def test_pieces_of_the_vocabulary(h):
    """More tokens than one piece of the vocabulary holds: three pieces, the last ragged."""
    M, V = 33000, 9001
    t = [x.to(DEV) for x in problem(M, h, V, "some")]
    got = run(*t)
    compare(got, *t)
    again = run(*t)
    assert all(torch.equal(got[k], again[k]) for k in got)


@pytest.mark.parametrize("M", [3, 100])
def test_pieces_of_the_vocabulary_for_few_tokens(M):
    """A vocabulary past one piece's 2^20 entries."""
    t = [x.to(DEV) for x in problem(M, 64, (1 << 20) + 777, "none")]
    compare(run(*t), *t)


def test_few_tokens_of_a_head_past_the_cache():
    """A head of more than 256 MB, which is read another way."""
    t = [x.to(DEV) for x in problem(9, 1024, 140001, "some")]
    compare(run(*t), *t)


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("M", [20, 70, 300])
def test_a_gradient_that_is_not_finite_stays_with_its_token(M, bad):
    H, W, labels, dl = (x.to(DEV) for x in problem(M, 256, 600, "none"))
    dl[7] = 0
    _, lse = nf4.qlora_loss_fwd(H, W, labels)
    live, ref = reference(H, W, labels, dl)
    dl[7] = bad
    dH, _ = nf4.qlora_loss_bwd(H, W, labels, lse, dl)
    assert not torch.isfinite(dH[7]).any()
    others = torch.arange(M, device=DEV) != 7
    check("dH", dH[others], ref["dH"][0][others], ref["dH"][1][others])
    alone, _ = nf4.qlora_loss_bwd(H, W, labels, lse, torch.full_like(dl, bad))
    assert not torch.isfinite(alone).any()


def test_gradient_by_differences():
    """A float64 difference of the oracle's loss along a random direction."""
    H, W, labels, _ = problem(12, 64, 50, "some")
    live = (labels >= 0) & (labels < 50)
    H[~live] = 0
    dl = torch.ones(12)
    d = [x.to(DEV) for x in (H, W, labels, dl)]
    _, lse = nf4.qlora_loss_fwd(*d[:3])
    dH, dW = nf4.qlora_loss_bwd(*d[:3], lse, d[3], train_head=True)
    rng = np.random.default_rng(3)
    h64, w64, y = H.double().numpy(), W.double().numpy(), labels.tolist()
    a, b = rng.standard_normal(h64.shape), rng.standard_normal(w64.shape)
    f = lambda e: oracle.loss_fwd(h64 + e * a, w64 + e * b, y)[0].sum()
    diff = (f(1e-5) - f(-1e-5)) / 2e-5
    got = (dH.double().cpu().numpy() * a).sum() + (dW.double().cpu().numpy() * b).sum()
    size = np.sqrt((dH.double().cpu().numpy() * a) ** 2).sum() + np.sqrt((dW.double().cpu().numpy() * b) ** 2).sum()
    assert abs(got - diff) <= 2.0 ** -7 * size      # two bf16 roundings of every term


def test_neighbours_are_left_alone():
    M, h, V = 45, 192, 301
    H, W, labels, dl = (x.to(DEV) for x in problem(M, h, V, "some"))
    guard = lambda n, t: torch.full((n + 256,), 7.0, dtype=t, device=DEV)
    big = dict(loss=guard(M, torch.float32), lse=guard(M, torch.float32), dH=guard(M * h, BF), dW=guard(V * h, BF))
    nf4.qlora_loss_fwd(H, W, labels, loss=big["loss"][:M], lse=big["lse"][:M])
    ws = torch.full((nf4.workspace_size(nf4.QLORA_OP_LOSS_BWD, M, h, V) + 512,), 255, dtype=torch.uint8, device=DEV)
    nf4.qlora_loss_bwd(H, W, labels, big["lse"][:M], dl, dH=big["dH"][: M * h].view(M, h),
                       dW=big["dW"][: V * h].view(V, h), workspace=ws[:-512])
    assert torch.all(ws[-512:] == 255)
    for t, n in zip(big.values(), (M, M, M * h, V * h)):
        assert torch.all(t[n:] == 7.0)
    compare(dict(loss=big["loss"][:M], lse=big["lse"][:M], dH=big["dH"][: M * h].view(M, h),
                 dW=big["dW"][: V * h].view(V, h)), H, W, labels, dl)


def test_captured_step():
    """One captured graph, replayed with other labels (another number of tokens with a
    loss) and other values, between eager calls."""
    M, h, V = 140, 128, 700
    bufs = [x.to(DEV) for x in problem(M, h, V, "some")]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(*bufs)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run_captured(*bufs)
    for k, skip in enumerate(("none", "all", "some", "most")):
        for b, x in zip(bufs, problem(M, h, V, skip, seed=k + 1)):
            b.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        eager = run(*bufs)
        assert all(torch.equal(held[key], eager[key]) for key in eager), skip
        compare(eager, *bufs)


def run_captured(H, W, labels, dl):
    loss, lse = nf4.qlora_loss_fwd(H, W, labels)
    dH, dW = nf4.qlora_loss_bwd(H, W, labels, lse, dl, train_head=True)
    return dict(loss=loss, lse=lse, dH=dH, dW=dW)
