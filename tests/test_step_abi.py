"""Refusals of the training step's operators around the linears, on the CPU: every bad
argument is turned away before anything is launched."""
import ctypes

import pytest

nf4 = pytest.importorskip("bit_quantized_fine_nf4_amd")
lib = nf4.lib

OK, INV, UNS = nf4.QLORA_OK, nf4.QLORA_ERR_INVALID_VALUE, nf4.QLORA_ERR_UNSUPPORTED
A = [ctypes.c_void_p(0x100000 + 0x10000 * i) for i in range(24)]   # distinct, aligned, never dereferenced
ODD = ctypes.c_void_p(0x100002)
NAN = float("nan")


def norm_fwd(R=A[0], dt=1, Y=A[1], w_post=A[2], gate=A[3], alpha=1.0, w_pre=A[4], eps=1e-6, M=4, h=64, R_out=A[5],
             N=A[6], rq=A[7], rp=A[8]):
    return lib.qlora_norm_fwd(R, dt, Y, w_post, gate, alpha, w_pre, eps, M, h, R_out, N, rq, rp, None)


def norm_bwd(dN=A[0], dR_out=A[1], dt=1, R_out=A[2], Y=A[3], rq=A[4], rp=A[5], w_post=A[6], gate=A[7], alpha=1.0,
             w_pre=A[8], M=4, h=64, dR=A[9], dY=A[10], dwp=A[11], dwq=A[12], dg=A[13], ws=A[14], wb=1 << 30):
    return lib.qlora_norm_bwd(dN, dR_out, dt, R_out, Y, rq, rp, w_post, gate, alpha, w_pre, M, h, dR, dY, dwp, dwq, dg,
                              ws, wb, None)


@pytest.mark.parametrize("bad", [
    dict(R=None), dict(dt=2), dict(M=0), dict(h=0), dict(M=-1), dict(R=ODD), dict(Y=ODD), dict(w_pre=ODD),
    dict(rp=ODD), dict(eps=0.0), dict(eps=NAN), dict(eps=float("inf")), dict(alpha=NAN), dict(N=None), dict(R_out=None),
    dict(Y=None), dict(Y=None, w_post=None), dict(Y=None, w_post=None, gate=None),   # R_out is then R
    dict(Y=None, w_post=None, gate=None, R_out=None, w_pre=None), dict(N=A[0]), dict(N=A[5]), dict(R_out=A[1]),
])
def test_norm_fwd_refusals(bad):
    assert norm_fwd(**bad) == INV


@pytest.mark.parametrize("bad", [
    dict(dR=None), dict(dt=3), dict(M=0), dict(h=-1), dict(dN=None), dict(R_out=None), dict(rp=None), dict(dR=ODD),
    dict(w_pre=None), dict(w_pre=None, dwp=None, dR_out=None), dict(dY=None), dict(Y=None), dict(rq=None),
    dict(w_post=None), dict(gate=None), dict(alpha=NAN), dict(ws=None), dict(wb=16), dict(ws=ctypes.c_void_p(0x100010)),
    dict(dR=A[0]), dict(dR=A[2]), dict(dR=A[10]), dict(dY=A[0]), dict(dY=A[1]), dict(dY=A[3]),
    dict(w_post=None, dwq=None, Y=None),      # the gate's gradient needs Y
])
def test_norm_bwd_refusals(bad):
    assert norm_bwd(**bad) == INV


def test_norm_limits():
    assert norm_fwd(h=16385) == UNS and norm_bwd(h=16385) == UNS
    assert norm_fwd(M=1 << 40, h=64) == UNS and norm_bwd(M=1 << 40, h=64) == UNS
    assert nf4.workspace_size(nf4.QLORA_OP_NORM_BWD, 5, 100) % 256 == 0
    for a, b in ((0, 64), (4, 0), (4, 16385)):
        with pytest.raises(nf4.QloraError):
            nf4.workspace_size(nf4.QLORA_OP_NORM_BWD, a, b)


def loss_fwd(H=A[0], W=A[1], lab=A[2], M=4, h=64, V=100, loss=A[3], lse=A[4], ws=A[5], wb=1 << 40):
    return lib.qlora_loss_fwd(H, W, lab, M, h, V, loss, lse, ws, wb, None)


def loss_bwd(H=A[0], W=A[1], lab=A[2], lse=A[3], dl=A[4], M=4, h=64, V=100, dH=A[5], dW=A[6], ws=A[7], wb=1 << 40):
    return lib.qlora_loss_bwd(H, W, lab, lse, dl, M, h, V, dH, dW, ws, wb, None)


@pytest.mark.parametrize("call", [loss_fwd, loss_bwd])
@pytest.mark.parametrize("bad", [
    dict(H=None), dict(W=None), dict(lab=None), dict(lse=None), dict(M=0), dict(V=0), dict(h=0), dict(h=100),
    dict(H=ODD), dict(W=ODD), dict(lab=ODD), dict(ws=None), dict(wb=256), dict(ws=ctypes.c_void_p(0x100010)),
])
def test_loss_refusals(call, bad):
    assert call(**bad) == INV


def test_loss_own_refusals():
    assert loss_fwd(loss=None) == INV and loss_fwd(loss=A[4]) == INV
    assert loss_bwd(dl=None) == INV and loss_bwd(dH=None) == INV and loss_bwd(dH=ODD) == INV
    assert loss_bwd(dH=A[0]) == INV and loss_bwd(dH=A[6]) == INV and loss_bwd(dW=A[1]) == INV
    for call in (loss_fwd, loss_bwd):
        assert call(h=(1 << 20) + 64) == UNS and call(V=(1 << 24) + 1) == UNS and call(M=1 << 25) == UNS
        assert call(M=1 << 20, V=1 << 20) == UNS      # too many tiles
    for op in (nf4.QLORA_OP_LOSS_FWD, nf4.QLORA_OP_LOSS_BWD):
        assert nf4.workspace_size(op, 100, 128, 1000) % 256 == 0
        for a, b, c in ((0, 64, 10), (4, 65, 10), (4, 64, 0), (1 << 20, 64, 1 << 20)):
            with pytest.raises(nf4.QloraError):
                nf4.workspace_size(op, a, b, c)
    # the backward's workspace follows a piece of the vocabulary, not the whole of it
    small, large = (nf4.workspace_size(nf4.QLORA_OP_LOSS_BWD, 65536, 64, V) for V in (8192, 131072))
    assert large == small


def drop(x=A[0], dt=1, n=10, p=0.1, rng=A[1], out=A[2]):
    return lib.qlora_dropout(x, dt, n, p, rng, out, None)


BAD_DROP = [dict(p=-0.1), dict(p=1.0), dict(p=NAN), dict(p=0.999999), dict(rng=None), dict(rng=ctypes.c_void_p(0x100004))]


@pytest.mark.parametrize("bad", BAD_DROP + [dict(x=None), dict(out=None), dict(dt=2), dict(n=0), dict(x=ODD), dict(out=ODD)])
def test_dropout_refusals(bad):
    assert drop(**bad) == INV
    assert drop(n=(1 << 40) + 1) == UNS


def weight(h=128, o=64, codes=A[20]):
    return nf4.NF4WeightT(codes.value if codes else None, A[21].value, A[22].value, A[23].value, h, o)


def lin_fwd(W=None, cb=0, X=A[0], M=4, L1=A[1], L2=A[2], r=8, p=0.1, rng=A[3], Y=A[4], T=A[5], ws=A[6], wb=1 << 40):
    return lib.qlora_linear_fwd_dropout(ctypes.byref(W or weight()), cb, X, M, L1, L2, r, 1.0, p, rng, Y, T, ws, wb, None)


def lin_bwd(W=None, cb=0, X=A[0], T=A[5], dY=A[7], M=4, L1=A[1], L2=A[2], r=8, p=0.1, rng=A[3], dX=A[8], dL1=A[9],
            dL2=A[10], ws=A[6], wb=1 << 40):
    return lib.qlora_linear_bwd_dropout(ctypes.byref(W or weight()), cb, X, T, dY, M, L1, L2, r, 1.0, p, rng, dX, dL1,
                                        dL2, ws, wb, None)


@pytest.mark.parametrize("call", [lin_fwd, lin_bwd])
@pytest.mark.parametrize("bad", BAD_DROP + [
    dict(cb=3), dict(X=None), dict(X=ODD), dict(M=0), dict(M=(1 << 31) + 1), dict(L1=None), dict(L2=None), dict(r=-1),
    dict(r=129), dict(T=None), dict(T=ODD), dict(ws=None), dict(wb=64), dict(ws=ctypes.c_void_p(0x100010)),
    dict(W=weight(h=100)), dict(W=weight(o=32)), dict(W=weight(codes=None)), dict(W=weight(codes=ODD)),
])
def test_linear_dropout_refusals(call, bad):
    assert call(**bad) == INV


def test_linear_dropout_own_refusals():
    assert lin_fwd(Y=None) == INV
    for k in ("dY", "dX", "dL1", "dL2"):
        assert lin_bwd(**{k: None}) == INV and lin_bwd(**{k: ODD}) == INV
    assert lin_fwd(r=0, Y=None) == INV and lin_bwd(r=0, dY=None) == INV     # the plain linear's own checks
    op = nf4.QLORA_OP_LINEAR_DROPOUT
    for M, h, o, r in ((1, 64, 64, 1), (16, 1024, 1024, 64), (2048, 8192, 22016, 64)):
        assert nf4.workspace_size(op, M, h, o, r) >= nf4.workspace_size(nf4.QLORA_OP_LINEAR_FWD, M, h, o, r)
    assert nf4.workspace_size(op, 17, 64, 64, 0) == 0
    with pytest.raises(nf4.QloraError):
        nf4.workspace_size(op, 0, 64, 64, 8)
    big = weight(h=1 << 20, o=64)
    assert lin_bwd(W=big, M=1 << 31, wb=(1 << 62)) == UNS                   # too many token splits
