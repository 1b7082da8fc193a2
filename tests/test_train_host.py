"""The training operators' refusals, on a machine without a GPU: the C ABI
validates before it touches CUDA, the Python binding before it calls the ABI."""
import ctypes

import pytest
import torch

NULL = None


@pytest.fixture(scope="module")
def lib():
    from transformer_ffn_gb300 import build
    build.build()
    import transformer_ffn_gb300 as tffn
    return tffn.load()


@pytest.fixture(scope="module")
def tffn(lib):
    import transformer_ffn_gb300
    return transformer_ffn_gb300


def _ln_fwd(lib, X=16, R=NULL, gamma=16, beta=16, eps=1e-5, dtype=0, pdtype=0, T=4, N=64, Y=16, S=NULL, mean=16,
            rstd=16):
    return lib.layer_norm_forward(X, R, gamma, beta, ctypes.c_float(eps), dtype, pdtype, T, N, Y, S, mean, rstd, NULL)


@pytest.mark.parametrize("bad", [
    dict(X=NULL), dict(Y=NULL), dict(mean=NULL), dict(rstd=NULL), dict(R=16), dict(T=-1), dict(N=0), dict(N=-8),
    dict(dtype=2), dict(pdtype=-1), dict(eps=-1.0), dict(eps=float("nan")), dict(X=17), dict(X=18, dtype=1),
    dict(gamma=17), dict(beta=18, pdtype=1), dict(mean=18), dict(rstd=17), dict(T=1 << 31),
])
def test_layer_norm_forward_refuses(lib, bad):
    assert _ln_fwd(lib, **bad) == -1
    assert lib.tffn_last_launch_count() == 0


def _ln_bwd(lib, dY=16, S=16, gamma=16, mean=16, rstd=16, dS=NULL, dtype=0, pdtype=0, T=4, N=64, dX=16, dgamma=16,
            dbeta=16):
    return lib.layer_norm_backward(dY, S, gamma, mean, rstd, dS, dtype, pdtype, T, N, dX, dgamma, dbeta, NULL)


@pytest.mark.parametrize("bad", [
    dict(dY=NULL), dict(S=NULL), dict(mean=NULL), dict(rstd=NULL), dict(dX=NULL), dict(dgamma=NULL),
    dict(dbeta=NULL), dict(T=-1), dict(N=0), dict(dtype=3), dict(pdtype=2), dict(dY=17), dict(dS=17),
    dict(dgamma=18), dict(dX=18, dtype=1),
])
def test_layer_norm_backward_refuses(lib, bad):
    assert _ln_bwd(lib, **bad) == -1


def _glu_fwd(lib, X=16, W1=16, W3=16, W2=16, act=3, M=8, N=64, O=64, P=64, Y=16, G=16, U=16):
    return lib.ffn_glu_forward_train(X, W1, W3, W2, act, M, N, O, P, Y, G, U, NULL)


@pytest.mark.parametrize("bad", [
    dict(X=NULL), dict(W1=NULL), dict(W3=NULL), dict(W2=NULL), dict(Y=NULL), dict(G=NULL), dict(U=NULL),
    dict(M=-1), dict(N=12), dict(O=0), dict(P=4), dict(act=4), dict(act=-1), dict(X=24), dict(U=18),
])
def test_glu_forward_train_refuses(lib, bad):
    assert _glu_fwd(lib, **bad) == -1


def _glu_bwd(lib, dY=16, X=16, W1=16, W3=16, W2=16, G=16, U=16, act=3, M=8, N=64, O=64, P=64, dX=16, dW1=16, dW3=16,
             dW2=16):
    return lib.ffn_glu_backward(dY, X, W1, W3, W2, G, U, act, M, N, O, P, dX, dW1, dW3, dW2, NULL)


@pytest.mark.parametrize("bad", [
    dict(dY=NULL), dict(X=NULL), dict(W1=NULL), dict(W3=NULL), dict(W2=NULL), dict(G=NULL), dict(U=NULL),
    dict(dX=NULL), dict(dW1=NULL), dict(dW3=NULL), dict(dW2=NULL), dict(M=-1), dict(N=20), dict(O=4), dict(P=0),
    dict(act=9), dict(dY=8), dict(dW1=24), dict(M=0, dW2=NULL),
])
def test_glu_backward_refuses(lib, bad):
    assert _glu_bwd(lib, **bad) == -1


def _muon(lib, G=16, dtype=0, batch=1, m=8, n=8, steps=5, out=16):
    return lib.muon_orthogonalize(G, dtype, batch, m, n, steps, out, NULL)


@pytest.mark.parametrize("bad", [
    dict(G=NULL), dict(out=NULL), dict(dtype=2), dict(batch=-1), dict(m=-1), dict(n=-1), dict(steps=0),
    dict(steps=65), dict(m=(1 << 18) + 1), dict(n=1 << 20), dict(batch=70000), dict(G=18, dtype=1), dict(out=17),
])
def test_muon_refuses(lib, bad):
    assert _muon(lib, **bad) == -1


def test_empty_calls_touch_nothing(lib):
    assert _ln_fwd(lib, T=0, X=NULL, Y=NULL, mean=NULL, rstd=NULL) == 0
    assert _ln_bwd(lib, T=0, dY=NULL, S=NULL, mean=NULL, rstd=NULL, dX=NULL, dgamma=NULL, dbeta=NULL) == 0
    assert _glu_fwd(lib, M=0, X=NULL, Y=NULL, G=NULL, U=NULL) == 0
    assert _muon(lib, batch=0, G=NULL, out=NULL) == 0
    assert _muon(lib, m=0, G=NULL, out=NULL) == 0
    assert lib.tffn_last_launch_count() == 0


def test_workspace_sizes(tffn):
    base = tffn.layer_norm_workspace_bytes(0, 1)
    assert tffn.layer_norm_workspace_bytes(4096, 8192) >= base + 2 * 8192 * 4
    assert tffn.layer_norm_workspace_bytes(-1, 8) == 0 and tffn.layer_norm_workspace_bytes(1, 0) == 0
    # the backward pass keeps dG, dU and H
    assert tffn.ffn_glu_train_workspace_bytes(4096, 14336) >= 3 * 4096 * 14336 * 2
    assert tffn.ffn_glu_train_workspace_bytes(16, 12) == 0 and tffn.ffn_glu_train_workspace_bytes(-1, 64) == 0
    # two copies of X, A and B
    assert tffn.muon_workspace_bytes(1, 1024, 4096) >= (2 * 1024 * 4096 + 2 * 1024 * 1024) * 2
    assert tffn.muon_workspace_bytes(1, 0, 8) == 0 and tffn.muon_workspace_bytes(1, 1 << 19, 8) == 0


def test_binding_refuses(tffn):
    bf = torch.bfloat16
    X, v = torch.zeros(4, 64, dtype=bf), torch.zeros(64, dtype=bf)
    W1, W2 = torch.zeros(64, 64, dtype=bf), torch.zeros(64, 64, dtype=bf)
    stat = torch.zeros(4)
    with pytest.raises(ValueError, match="CUDA device"):      # no path computes on the host
        tffn.layer_norm_forward(X, v, v)
    with pytest.raises(ValueError, match="CUDA device"):
        tffn.layer_norm_backward(X, X, v, stat, stat)
    with pytest.raises(ValueError, match="CUDA device"):
        tffn.ffn_glu_forward_train(X, W1, W1, W2)
    with pytest.raises(ValueError, match="CUDA device"):
        tffn.muon_orthogonalize(X)
    with pytest.raises(TypeError):
        tffn.layer_norm_forward(X.half(), v, v)
    with pytest.raises(TypeError):
        tffn.ffn_glu_forward_train(X.float(), W1, W1, W2)
    with pytest.raises(TypeError):
        tffn.muon_orthogonalize(None)
    with pytest.raises(ValueError, match="dimensions"):
        tffn.layer_norm_forward(X[0], v, v)
    with pytest.raises(ValueError, match="dimensions"):
        tffn.muon_orthogonalize(X[0])
    with pytest.raises(ValueError, match="contiguous"):
        tffn.muon_orthogonalize(X.t())
