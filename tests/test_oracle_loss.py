"""Pins of the loss oracle (oracle/loss.py): closed forms and central differences."""
import numpy as np

import oracle


def test_closed_forms():
    H = np.array([[1.0, 0.0], [0.0, 0.0], [5.0, 5.0]])
    W = np.array([[np.log(2.0), 9.0], [0.0, 9.0], [0.0, 9.0]])
    loss, lse = oracle.loss_fwd(H, W, [0, 2, -100])
    assert np.allclose(lse, [np.log(4.0), np.log(3.0), 0.0], rtol=1e-15)   # 2 + 1 + 1, and three equal words
    assert np.allclose(loss, [np.log(2.0), np.log(3.0), 0.0], rtol=1e-15)
    G = oracle.loss_grad(H, W, [0, 2, 3], [1.0, 3.0, 1.0])                  # 3 is no word of three
    assert np.allclose(G, [[-0.5, 0.25, 0.25], [1.0, 1.0, -2.0], [0, 0, 0]], atol=1e-15)


def test_backward_by_differences():
    rng = np.random.default_rng(2)
    H, W = rng.standard_normal((5, 4)), rng.standard_normal((7, 4))
    labels, dl = [3, -1, 0, 6, 7], rng.standard_normal(5)
    H[1] = np.nan                                   # a token without a loss may hold anything
    dH, dW = oracle.loss_bwd(H, W, labels, dl)
    value = lambda H, W: float(np.sum(oracle.loss_fwd(H, W, labels)[0] * dl))
    for arg, grad in ((H, dH), (W, dW)):
        for at in np.ndindex(arg.shape):
            keep = arg[at]
            arg[at] = keep + 1e-6
            hi = value(H, W)
            arg[at] = keep - 1e-6
            lo = value(H, W)
            arg[at] = keep
            if arg is H and at[0] in (1, 4):
                assert at[0] == 1 or grad[at] == 0.0
            else:
                assert abs((hi - lo) / 2e-6 - grad[at]) < 1e-8
