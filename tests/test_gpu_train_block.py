"""The training operators together: a block's training step, streams, CUDA
graphs, and caller-owned and poisoned workspaces."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))
BF = torch.bfloat16


def _glu(M=300, N=256, O=1096, P=256, seed=1):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, std=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(BF)
    return (normal(M, N), normal(N, O, std=N ** -0.5), normal(N, O, std=N ** -0.5), normal(O, P, std=O ** -0.5),
            normal(M, P))


def _everything(tffn, X, W1, W3, W2, dY, m, gamma, beta, stream=None):
    Z, S, mean, rstd = tffn.layer_norm_forward(X, gamma, beta, residual=dY, stream=stream)
    Y, G, U = tffn.ffn_glu_forward_train(Z, W1, W3, W2, stream=stream)
    dZ, dW1, dW3, dW2 = tffn.ffn_glu_backward(dY, Z, W1, W3, W2, G, U, stream=stream)
    dX, dgamma, dbeta = tffn.layer_norm_backward(dZ, S, gamma, mean, rstd, dS=dY, stream=stream)
    return [Z, S, mean, rstd, Y, G, U, dZ, dW1, dW3, dW2, dX, dgamma, dbeta, tffn.muon_orthogonalize(m, stream=stream)]


def _operands(seed=1):
    X, W1, W3, W2, dY = _glu(seed=seed)
    return (X, W1, W3, W2, dY, torch.randn((256, 1096), device="cuda"), torch.ones(256, device="cuda"),
            torch.zeros(256, device="cuda"))


def test_block_learns(cuda_lib):
    """Thirty steps of the example: the loss falls by more than half."""
    import train_block
    losses = train_block.train(steps=30)
    assert losses[-1] < 0.5 * losses[0] and all(b < 1.05 * a for a, b in zip(losses, losses[1:]))


def test_block_gradient_against_differences(cuda_lib):
    """The gradient of the example's block against central differences of its
    64-bit forward pass: off by the operators' bf16 roundings, 1 % of the norms."""
    import train_block
    N, O, T, h = 64, 192, 50, 1e-4
    block = train_block.Block(N, O, seed=3)
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    X = torch.randn((T, N), generator=g, device="cuda").to(BF)
    dY = torch.randn((T, N), generator=g, device="cuda").to(BF)
    _, saved = block.forward(X)
    dX, _ = block.backward(dY, saved)

    def loss(x):
        z = torch.nn.functional.layer_norm(x, (N,), block.gamma.double(), block.beta.double(), 1e-5)
        a = z @ block.W1.double()
        return ((x + (torch.nn.functional.silu(a) * (z @ block.W3.double())) @ block.W2.double()) * dY.double()).sum()
    d = dX.double()
    V = d / d.norm() + torch.randn(d.shape, device="cuda", dtype=torch.float64) / d.numel() ** 0.5
    x = X.double()
    diff = float((loss(x + h * V) - loss(x - h * V)) / (2 * h))
    assert abs(float((d * V).sum()) - diff) <= 1e-2 * float(d.norm() * V.norm())


def test_other_stream(cuda_lib):
    """On a stream of the caller's: the same bits, results usable after a wait."""
    ops = _operands()
    want = _everything(cuda_lib, *ops)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = _everything(cuda_lib, *ops, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    with torch.cuda.stream(side):
        got = _everything(cuda_lib, *ops)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    cuda_lib.check()


def test_cuda_graph(cuda_lib):
    ops = list(_operands())
    want = _everything(cuda_lib, *ops)        # also sizes the workspace
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _everything(cuda_lib, *ops)
    for seed in (1, 2):
        fresh = _operands(seed)
        for a, b in zip(ops, fresh):
            a.copy_(b)
        want = _everything(cuda_lib, *ops)
        for _ in range(3):
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    cuda_lib.check()


def test_poisoned_workspace(cuda_lib):
    """A caller's workspace whose data region holds NaN before every call: a read
    of something not yet written would show."""
    ops = _operands()
    want = _everything(cuda_lib, *ops)
    torch.cuda.synchronize()
    need = max(cuda_lib.ffn_glu_train_workspace_bytes(300, 1096), cuda_lib.layer_norm_workspace_bytes(300, 256),
               cuda_lib.muon_workspace_bytes(1, 256, 1096))
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    data = 5 << 20
    cuda_lib.set_workspace(ws)
    try:
        for _ in range(3):
            X, W1, W3, W2, dY, m, gamma, beta = ops
            got = []
            for call in range(5):
                ws[data:] = 255
                if call == 0:
                    Z, S, mean, rstd = cuda_lib.layer_norm_forward(X, gamma, beta, residual=dY)
                    got += [Z, S, mean, rstd]
                elif call == 1:
                    Y, G, U = cuda_lib.ffn_glu_forward_train(Z, W1, W3, W2)
                    got += [Y, G, U]
                elif call == 2:
                    grads = cuda_lib.ffn_glu_backward(dY, Z, W1, W3, W2, G, U)
                    got += list(grads)
                elif call == 3:
                    got += list(cuda_lib.layer_norm_backward(grads[0], S, gamma, mean, rstd, dS=dY))
                else:
                    got.append(cuda_lib.muon_orthogonalize(m))
            cuda_lib.check()
            assert all(torch.equal(a, b) for a, b in zip(got, want))
            # the counters are left at zero
            assert not ws[256 + (4 << 20):data].any()
    finally:
        cuda_lib.set_workspace(None)


def test_workspace_too_small(cuda_lib):
    X, W1, W3, W2, dY = _glu()
    ws = torch.zeros(6 << 20, dtype=torch.uint8, device="cuda")
    cuda_lib.set_workspace(ws)
    try:
        for call in (lambda: cuda_lib.ffn_glu_forward_train(X, W1, W3, W2),
                     lambda: cuda_lib.muon_orthogonalize(torch.ones((512, 4096), device="cuda"))):
            with pytest.raises(cuda_lib.TffnError) as e:
                call()
            assert e.value.code == -5
    finally:
        cuda_lib.set_workspace(None)


def test_interleaved_with_inference(cuda_lib):
    """Training and inference calls share the workspace in stream order."""
    X, W1, W3, W2, dY = _glu(M=260)
    y = cuda_lib.ffn_glu_forward(X, W1, W3, W2)
    d = cuda_lib.ffn_glu_forward(X[:9].contiguous(), W1, W3, W2)
    Y, G, U = cuda_lib.ffn_glu_forward_train(X, W1, W3, W2)
    grads = cuda_lib.ffn_glu_backward(dY, X, W1, W3, W2, G, U)
    for _ in range(4):
        assert torch.equal(cuda_lib.ffn_glu_forward(X, W1, W3, W2), y)
        a = cuda_lib.ffn_glu_backward(dY, X, W1, W3, W2, G, U)
        assert torch.equal(cuda_lib.ffn_glu_forward(X[:9].contiguous(), W1, W3, W2), d)
        assert all(torch.equal(p, q) for p, q in zip(a, grads))
        cuda_lib.muon_orthogonalize(W1)
        assert torch.equal(cuda_lib.ffn_glu_forward_train(X, W1, W3, W2)[0], Y)
    cuda_lib.check()


def test_wait_timeout_is_reported_and_recovered(cuda_lib):
    """A tile that is never counted: the products that wait for it give up after
    the limit, the call is reported, and the next calls are right again."""
    ops = _operands()
    X, W1, W3, W2, dY, m, _, _ = ops
    Y, G, U = cuda_lib.ffn_glu_forward_train(X, W1, W3, W2)
    calls = (lambda: cuda_lib.ffn_glu_forward_train(X, W1, W3, W2),
             lambda: cuda_lib.ffn_glu_backward(dY, X, W1, W3, W2, G, U),
             lambda: [cuda_lib.muon_orthogonalize(m)])
    want = [call() for call in calls]
    cuda_lib.check()
    limit = cuda_lib.set_option(cuda_lib.OPT_WAIT_LIMIT_MS, 100)
    try:
        for call in calls:
            cuda_lib.set_option(cuda_lib.OPT_SKIP_FLAG, 0)
            call()
            cuda_lib.set_option(cuda_lib.OPT_SKIP_FLAG, -1)
            with pytest.raises(cuda_lib.TffnError) as e:
                cuda_lib.check()
            assert e.value.code == -4
            cuda_lib.check()
    finally:
        cuda_lib.set_option(cuda_lib.OPT_SKIP_FLAG, -1)
        cuda_lib.set_option(cuda_lib.OPT_WAIT_LIMIT_MS, limit)
    for call, w in zip(calls, want):
        assert all(torch.equal(a, b) for a, b in zip(call(), w))
    cuda_lib.check()
