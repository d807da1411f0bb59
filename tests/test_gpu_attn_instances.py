"""Biased and capped attention at sizes that take each instance of its kernels: one and two groups of
waves (above 512 workgroups of 128 queries forward, 256 to 512 of the queries' gradients), keys'
gradients in one, two and more parts (bounds: attention_bounds.py); and what the other tests of
attention look at less closely."""
import threading

import pytest
import torch

import oracle
from attention_bounds import BF, DEV, check, problem, reference, run

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import bit_quantized_fine_nf4_amd as nf4  # noqa: E402


def geometric(heads):
    return (2.0 ** (-8.0 * torch.arange(1, heads + 1) / heads)).float().to(DEV)


@pytest.mark.parametrize("M,hq,hk", [(1100, 64, 64), (1030, 120, 120), (1100, 48, 12), (700, 16, 2), (500, 66, 66)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cap,bias", [(0.0, True), (30.0, False), (2.0, True)])
def test_every_form(M, hq, hk, d, cap, bias):
    print(f"attn instances M={M} hq={hq} hk={hk} d={d} cap={cap} bias={bias}", flush=True)
    p = problem(M, hq, hk, d, oracle.spans([0, 30, M - 5], M))
    slopes = geometric(hq) if bias else None
    check(run(nf4, p, cap=cap, slopes=slopes), reference(p, d ** -0.5, cap, slopes))


def test_growing_scores_by_tensor():
    """Scores that grow along the keys.  dQ and dK keep little of what their sums cancel (a sum of dS
    that is zero times what the keys share), so these are held by each value's bound alone; O and dV
    have nothing that cancels."""
    M, d = 700, 64
    p = problem(M, 2, 2, d, oracle.spans([0, M], M, causal=False))
    p["K"] = (p["K"].float() * 0.1 + torch.arange(M, device=DEV)[:, None, None] * 0.02).to(BF)
    p["Q"] = (p["Q"].float() * 0.1 + 1.0).to(BF)
    for _ in range(2):
        check(run(nf4, p), reference(p, d ** -0.5), dict(dQ=float("inf"), dK=float("inf")))
        p["K"] = p["K"].flip(0).contiguous()


def test_documents_out_of_order():
    """Bounds that decrease give some spans; attention over them is that of the spans as they are."""
    M = 600
    documents = torch.tensor([0, 900, -5, 40, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    for causal in (True, False):
        spans = nf4.qlora_attn_spans(documents, M, causal=causal, window=70)
        assert int(spans[:, 0].min()) >= 0 and int(spans[:, 1].max()) <= M
        p = problem(M, 2, 1, 64, spans.cpu())
        check(run(nf4, p), reference(p, 0.125))


def test_two_threads_end():
    """Forward, backward and one new token from two threads, both of which end."""
    sets = [problem(M, 4, 2, 64, oracle.spans([0, M - 3], M)) for M in (130, 900)]
    want = [run(nf4, p) for p in sets]
    torch.cuda.synchronize()
    rounds, errors, gate = [0, 0], [], threading.Barrier(2)

    def work(k):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                gate.wait(20)
                for _ in range(20):
                    got = run(nf4, sets[k])
                    torch.cuda.current_stream().synchronize()
                    assert all(torch.equal(got[x], want[k][x]) for x in got)
                    rounds[k] += 1
        except BaseException as e:  # noqa: BLE001 (reported below)
            errors.append(e)

    threads = [threading.Thread(target=work, args=(k,), daemon=True) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    assert not errors and rounds == [20, 20] and not any(t.is_alive() for t in threads), (errors, rounds)
