"""The gated FFN's training forward and backward pass against the formulas in
64 bits.

Tolerances: an output is stored in bf16 (eight significant bits, half a unit is
at most 2^-8 of it) and summed in fp32 from products of operands of which some
were rounded to bf16 on the way (H, dG, dU: 2^-8 of each term, so at most 2^-8
of the sum of the terms' magnitudes) with an accumulation error of at most K 2^-24 of that same sum.
Independent roundings add in quadrature, each 1.7e-3 of the norm (2^-8 / sqrt(3)
times 0.75, the mean over a binade): two of them 2.4e-3; 4e-3 is allowed."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _inputs(M, N, O, P, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, std=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(BF)
    return (normal(M, N), normal(N, O, std=N ** -0.5), normal(N, O, std=N ** -0.5), normal(O, P, std=O ** -0.5),
            normal(M, P, std=0.1))


def _act(name, x):
    """The activation and its derivative in 64 bits."""
    if name == "none":
        return x, torch.ones_like(x)
    if name == "relu":
        return x.clamp_min(0), (x > 0).double()
    if name == "silu":
        s = torch.sigmoid(x)
        return x * s, s * (1 + x * (1 - s))
    c = 0.7978845608028654
    t = torch.tanh(c * (x + 0.044715 * x ** 3))
    return 0.5 * x * (1 + t), 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * c * (1 + 0.134145 * x * x)


def _close(got, want, terms, K, what, norm=4e-3):
    """terms: the sum of the magnitudes of the products that make `want`."""
    err = (got.double() - want).abs()
    bound = 2.0 ** -8 * want.abs() + (2.0 ** -8 + (K + 64) * 2.0 ** -24) * terms * 1.01 + 1e-30
    bad = ~(err <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} out of bound"
    if want.numel() >= 4096:
        assert float(err.norm() / want.norm()) <= norm, f"{what}: {float(err.norm() / want.norm()):.2e} of the norm"


def _check(tffn, X, W1, W3, W2, dY, act):
    Y, G, U = tffn.ffn_glu_forward_train(X, W1, W3, W2, act)
    tffn.check()
    x, w1, w3, w2, dy = (t.double() for t in (X, W1, W3, W2, dY))
    g, u = x @ w1, x @ w3
    a, _ = _act(act, g)
    N, O, P, M = X.shape[1], W1.shape[1], W2.shape[1], X.shape[0]
    _close(G, g, (x.abs() @ w1.abs()) * 2.0 ** -9, N, "G")
    _close(U, u, (x.abs() @ w3.abs()) * 2.0 ** -9, N, "U")
    # H carries the fp32 errors of G and U too: a few 2^-24 of their terms
    _close(Y, (a * u) @ w2, (a * u).abs() @ w2.abs() + 1e-4 * (x.abs() @ w1.abs() + 1).mean(), O, "Y")

    grads = tffn.ffn_glu_backward(dY, X, W1, W3, W2, G, U, act)
    tffn.check()
    g, u = G.double(), U.double()
    a, d = _act(act, g)
    dh = dy @ w2.t()
    noise = (dy.abs() @ w2.abs().t()) * ((P + 64) * 2.0 ** -24)   # dH's own fp32 error
    dg, du, h = dh * u * d, dh * a, a * u
    tg, tu = dg.abs() + 512 * noise * (u * d).abs() + 1e-5 * dh.abs(), du.abs() + 512 * noise * a.abs() + 1e-5 * dh.abs()
    want = (dg @ w1.t() + du @ w3.t(), x.t() @ dg, x.t() @ du, h.t() @ dy)
    terms = (tg @ w1.abs().t() + tu @ w3.abs().t(), x.abs().t() @ tg, x.abs().t() @ tu, h.abs().t() @ dy.abs())
    for name, got, w, t, K in zip(("dX", "dW1", "dW3", "dW2"), grads, want, terms, (2 * O, M, M, M)):
        _close(got, w, t, K, name)
    return (Y, G, U), grads


SHAPES = [
    (1, 8, 8, 8),              # one token, the smallest sizes
    (1, 256, 1024, 256), (2, 72, 200, 136), (16, 512, 2048, 512),
    (64, 256, 1024, 256),      # one row band, narrow tiles
    (127, 64, 72, 64), (128, 128, 128, 128), (129, 136, 264, 200),
    (255, 320, 520, 64), (256, 256, 256, 256), (257, 64, 1032, 320),
    (300, 1544, 136, 72),      # N > O
    (513, 64, 384, 1096),      # P > O
    (700, 520, 1416, 264),     # sizes that end inside a tile everywhere
    (1003, 2056, 5528, 2056),  # several tasks per CTA pair
    (2100, 1024, 2048, 512),   # more bands than one raster group
    (40, 4096, 512, 4096),     # long reductions in parts
]


@pytest.mark.parametrize("M,N,O,P", SHAPES)
def test_forward_and_backward(cuda_lib, M, N, O, P):
    _check(cuda_lib, *_inputs(M, N, O, P, M + O), "silu")


@pytest.mark.parametrize("act", ["none", "relu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("M,N,O,P", [(70, 136, 328, 200), (600, 256, 1160, 256)])
def test_activations(cuda_lib, act, M, N, O, P):
    X, W1, W3, W2, dY = _inputs(M, N, O, P, 17)
    _check(cuda_lib, X, (W1.float() * 3).to(BF), W3, W2, dY, act)   # gates well into both tails


@pytest.mark.parametrize("M", [33, 300, 4096])
def test_forward_equals_inference(cuda_lib, M):
    """Y is the inference entry point's, up to the order of its fp32 sums."""
    X, W1, W3, W2, _ = _inputs(M, 512, 1536, 512, M)
    Y, _, _ = cuda_lib.ffn_glu_forward_train(X, W1, W3, W2)
    y = cuda_lib.ffn_glu_forward(X, W1, W3, W2, "silu")
    assert float((Y.float() - y.float()).norm() / y.float().norm()) < 4e-3


def test_large_gates(cuda_lib):
    """Gates beyond the exponential's range: the activations' limits, no NaN."""
    M, N, O, P = 40, 64, 128, 64
    X, W1, W3, W2, dY = _inputs(M, N, O, P, 5)
    for act in ("silu", "gelu_tanh", "relu"):
        for scale in (300.0, 3e8, 1e18):
            G = (torch.randn((M, O), device="cuda") * scale).to(BF)
            U = torch.ones((M, O), device="cuda", dtype=BF)
            dX, dW1, dW3, dW2 = cuda_lib.ffn_glu_backward(dY, X, W1, W3, W2, G, U, act)
            for t in (dX, dW1, dW3, dW2):
                assert torch.isfinite(t).all()
            dh = dY.double() @ W2.double().t()
            a, d = _act(act, G.double())
            want = X.double().t() @ (dh * d)
            assert float((dW1.double() - want).norm() / want.norm()) < 4e-3
            want = (a.t() @ dY.double())
            assert float((dW2.double() - want).norm() / want.norm()) < 4e-3


def test_nan_stays_in_its_token(cuda_lib):
    X, W1, W3, W2, _ = _inputs(300, 128, 512, 128, 6)
    want = cuda_lib.ffn_glu_forward_train(X, W1, W3, W2)
    Z = X.clone()
    Z[131, 5] = float("nan")
    got = cuda_lib.ffn_glu_forward_train(Z, W1, W3, W2)
    keep = torch.arange(300, device="cuda") != 131
    for g, w in zip(got, want):
        assert torch.equal(g[keep], w[keep]) and torch.isnan(g[131]).all()


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_gradients_against_differences(cuda_lib, act):
    """Directional derivatives of the 64-bit forward pass by central differences.
    A gradient is off by at most 4e-3 of its norm (above), so its product with a
    direction V is off by at most 4e-3 |grad| |V|; G and U are the forward
    pass's bf16 values, which moves the true gradient by as much again."""
    M, N, O, P, h = 90, 128, 256, 128, 1e-4
    X, W1, W3, W2, dY = _inputs(M, N, O, P, 7)
    _, G, U = cuda_lib.ffn_glu_forward_train(X, W1, W3, W2, act)
    grads = cuda_lib.ffn_glu_backward(dY, X, W1, W3, W2, G, U, act)
    base = [t.double() for t in (X, W1, W3, W2)]

    def loss(x, w1, w3, w2):
        return (((_act(act, x @ w1)[0] * (x @ w3)) @ w2) * dY.double()).sum()
    for i, grad in enumerate(grads):
        gd = grad.double()
        V = gd / gd.norm() + torch.randn(gd.shape, device="cuda", dtype=torch.float64) / gd.numel() ** 0.5
        up, down = list(base), list(base)
        up[i], down[i] = base[i] + h * V, base[i] - h * V
        diff = float((loss(*up) - loss(*down)) / (2 * h))
        assert abs(float((gd * V).sum()) - diff) <= 1e-2 * float(gd.norm() * V.norm())


def test_results_repeat(cuda_lib):
    for M, N, O, P in ((16, 1024, 4096, 1024), (700, 512, 1536, 256)):
        X, W1, W3, W2, dY = _inputs(M, N, O, P, 8)
        a, b = (cuda_lib.ffn_glu_forward_train(X, W1, W3, W2) for _ in range(2))
        assert all(torch.equal(p, q) for p, q in zip(a, b))
        a, b = (cuda_lib.ffn_glu_backward(dY, X, W1, W3, W2, a[1], a[2]) for _ in range(2))
        assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_no_rows(cuda_lib):
    X, W1, W3, W2, dY = _inputs(4, 64, 128, 64, 9)
    Y, G, U = cuda_lib.ffn_glu_forward_train(X[:0], W1, W3, W2)
    assert Y.shape == (0, 64) and G.shape == (0, 128)
    dX, dW1, dW3, dW2 = cuda_lib.ffn_glu_backward(dY[:0], X[:0], W1, W3, W2, G, U)
    assert dX.shape == (0, 64) and not dW1.any() and not dW3.any() and not dW2.any()


def test_refusals(cuda_lib):
    X, W1, W3, W2, dY = _inputs(8, 64, 128, 64, 10)
    _, G, U = cuda_lib.ffn_glu_forward_train(X, W1, W3, W2)
    with pytest.raises(TypeError):
        cuda_lib.ffn_glu_forward_train(X, W1.float(), W3, W2)
    with pytest.raises(ValueError):
        cuda_lib.ffn_glu_forward_train(X, W1, W3[:, :64], W2)
    with pytest.raises(ValueError):
        cuda_lib.ffn_glu_forward_train(X, W1, W3, W2[:64])
    with pytest.raises(ValueError):
        cuda_lib.ffn_glu_forward_train(X, W1.t(), W3, W2)
    with pytest.raises(KeyError):
        cuda_lib.ffn_glu_forward_train(X, W1, W3, W2, "tanh")
    with pytest.raises(ValueError):
        cuda_lib.ffn_glu_backward(dY[:4], X, W1, W3, W2, G, U)
    with pytest.raises(TypeError):
        cuda_lib.ffn_glu_backward(dY, X, W1, W3, W2, G.float(), U)
    odd = torch.zeros((8, 60), dtype=BF, device="cuda")      # not a multiple of 8
    with pytest.raises(cuda_lib.TffnError):
        cuda_lib.ffn_glu_forward_train(odd, torch.zeros((60, 128), dtype=BF, device="cuda"),
                                       torch.zeros((60, 128), dtype=BF, device="cuda"), W2)
