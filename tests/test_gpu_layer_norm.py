"""Layer norm's forward and backward pass against the formulas in 64 bits.

Tolerances, with u = 2^-24 (fp32) and w = half a unit in the last place of the
stored type (2^-8 relative for bf16's eight significant bits, u for fp32).  A row's sum runs over 16
values per thread and then a tree, so it is off by at most 32 u times the sum
of magnitudes; divided by N that is 32 u mean|S|, which the statistics, xh and
dX see multiplied by rstd.  64 u times the magnitudes that enter covers the
few further roundings."""
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
W = {torch.bfloat16: 2.0 ** -8, torch.float32: U}
BF, F32 = torch.bfloat16, torch.float32


def _rows(T, N, dtype, seed, outlier=True):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn((T, N), generator=g, device="cuda") * 1.5 + 0.25
    if outlier:
        x[:, N // 2] *= 30.0
    return x.to(dtype)


def _params(N, dtype, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1000)
    return ((1 + 0.2 * torch.randn(N, generator=g, device="cuda")).to(dtype),
            (0.2 * torch.randn(N, generator=g, device="cuda")).to(dtype))


def _close(got, want, bound, what):
    err = (got.double() - want).abs()
    bad = ~(err <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} out of bound, worst {float((err - bound).max()):.3e}"


def _check_forward(tffn, X, gamma, beta, R, eps=1e-5):
    Y, S, mean, rstd = tffn.layer_norm_forward(X, gamma, beta, residual=R, eps=eps)
    tffn.check()
    dtype = X.dtype
    want_S = X if R is None else (X.double() + R.double()).to(dtype)
    assert torch.equal(S, want_S)
    s = want_S.double()
    m = s.mean(1, keepdim=True)
    r = 1 / torch.sqrt(((s - m) ** 2).mean(1, keepdim=True) + eps)
    a = s.abs().mean(1, keepdim=True)
    _close(mean, m[:, 0], 64 * U * a[:, 0], "mean")
    # the variance is off by 64 u of itself and by the square of the mean's error
    _close(rstd, r[:, 0], r[:, 0] * (64 * U + (64 * U * a[:, 0] * r[:, 0]) ** 2), "rstd")
    g = 1.0 if gamma is None else gamma.double()
    b = 0.0 if beta is None else beta.double()
    y = (s - m) * r * g + b
    slack = 64 * U * ((s.abs() + a) * r * (abs(g) if gamma is None else g.abs()) + (y - b).abs() + y.abs())
    _close(Y, y, W[dtype] * y.abs() + slack, "Y")
    return Y, S, mean, rstd


def _check_backward(tffn, dY, S, gamma, mean, rstd, dS):
    dX, dgamma, dbeta = tffn.layer_norm_backward(dY, S, gamma, mean, rstd, dS=dS)
    tffn.check()
    T, N = dY.shape
    r, m = rstd.double()[:, None], mean.double()[:, None]
    xh = (S.double() - m) * r
    dy = dY.double()
    gy = dy if gamma is None else dy * gamma.double()
    dx = r * (gy - gy.mean(1, keepdim=True) - xh * (gy * xh).mean(1, keepdim=True))
    slack = 64 * U * r * (gy.abs() + gy.abs().mean(1, keepdim=True) + xh.abs() * (gy * xh).abs().mean(1, keepdim=True))
    if dS is not None:
        dx = dx + dS.double()
        slack = slack + 4 * U * dS.double().abs()
    _close(dX, dx, W[dY.dtype] * dx.abs() + slack, "dX")
    # a column: a thread's rows one after another (at most T / 2 of them), then CTAs in strands of 16
    depth = (T + 1) // 2 + 64
    _close(dgamma, (dy * xh).sum(0), (depth + 4) * U * (dy * xh).abs().sum(0), "dgamma")
    _close(dbeta, dy.sum(0), depth * U * dy.abs().sum(0), "dbeta")
    return dX, dgamma, dbeta


SHAPES = [
    # one token, one column, rows shorter than a vector
    (1, 1), (1, 8), (3, 2), (5, 3), (1, 4096),
    # a warp's rows, around its limits; odd widths start between words
    (64, 256), (37, 255), (37, 257), (1000, 511), (9, 512), (2500, 513),
    # a block's rows
    (33, 1021), (300, 1024), (17, 1025), (700, 2048), (11, 2047), (40, 4093), (400, 4096), (3, 4097),
    (50, 8190), (13, 8191), (320, 8192),
    # longer than a block's registers
    (4, 8193), (7, 16384), (2, 20001),
]


@pytest.mark.parametrize("T,N", SHAPES)
@pytest.mark.parametrize("dtype,ptype", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)])
@pytest.mark.parametrize("residual", [False, True])
def test_forward_and_backward(cuda_lib, T, N, dtype, ptype, residual):
    X, R = _rows(T, N, dtype, T + N), _rows(T, N, dtype, T + N + 1) if residual else None
    gamma, beta = _params(N, ptype, N)
    _, S, mean, rstd = _check_forward(cuda_lib, X, gamma, beta, R)
    dY = _rows(T, N, dtype, T + N + 2)
    dS = _rows(T, N, dtype, T + N + 3, outlier=False) if residual else None
    _check_backward(cuda_lib, dY, S, gamma, mean, rstd, dS)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_without_parameters(cuda_lib, dtype):
    X = _rows(30, 384, dtype, 5)
    _, S, mean, rstd = _check_forward(cuda_lib, X, None, None, None)
    assert S is X
    _check_backward(cuda_lib, _rows(30, 384, dtype, 6), S, None, mean, rstd, None)
    gamma, beta = _params(384, F32, 7)
    _check_forward(cuda_lib, X, gamma, None, None)
    _check_forward(cuda_lib, X, None, beta, None)


def test_without_weight_gradients(cuda_lib):
    X = _rows(100, 640, BF, 8)
    gamma, beta = _params(640, F32, 8)
    _, S, mean, rstd = cuda_lib.layer_norm_forward(X, gamma, beta)
    dY = _rows(100, 640, BF, 9)
    want = cuda_lib.layer_norm_backward(dY, S, gamma, mean, rstd)[0]
    dX, dgamma, dbeta = cuda_lib.layer_norm_backward(dY, S, gamma, mean, rstd, weight_grads=False)
    assert dgamma is None and dbeta is None and torch.equal(dX, want)


@pytest.mark.parametrize("N", [96, 1021, 4096])
def test_unaligned_tensors(cuda_lib, N):
    """Contiguous tensors that start one element into their storage."""
    def shifted(t):
        s = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        s[1:] = t.reshape(-1)
        return s[1:].view(t.shape)
    for dtype in (BF, F32):
        X, R = shifted(_rows(20, N, dtype, N)), shifted(_rows(20, N, dtype, N + 1))
        gamma, beta = (shifted(t) for t in _params(N, BF, N))
        _, S, mean, rstd = _check_forward(cuda_lib, X, gamma, beta, R)
        _check_backward(cuda_lib, shifted(_rows(20, N, dtype, N + 2)), S, gamma, mean, rstd, X)


def test_constant_rows(cuda_lib):
    """A row without variance: xh is 0 and rstd 1 / sqrt(eps)."""
    X = torch.full((6, 1000), 3.5, device="cuda", dtype=BF)
    gamma, beta = _params(1000, F32, 1)
    Y, S, mean, rstd = cuda_lib.layer_norm_forward(X, gamma, beta)
    assert torch.equal(mean, torch.full_like(mean, 3.5))
    assert torch.equal(Y, beta.to(BF).expand(6, 1000))
    dX, dgamma, _ = cuda_lib.layer_norm_backward(_rows(6, 1000, BF, 2), S, gamma, mean, rstd)
    assert torch.isfinite(dX).all() and torch.equal(dgamma, torch.zeros_like(dgamma))


def test_nan_and_inf_stay_in_their_row(cuda_lib):
    for N in (333, 512, 1024, 8192):
        X = _rows(40, N, BF, N)
        gamma, beta = _params(N, F32, N)
        want = cuda_lib.layer_norm_forward(X, gamma, beta)[0]
        Z = X.clone()
        Z[7, 0], Z[8, N - 1], Z[39, N // 3] = float("nan"), float("inf"), float("-inf")
        Y = cuda_lib.layer_norm_forward(Z, gamma, beta)[0]
        keep = torch.ones(40, dtype=torch.bool, device="cuda")
        keep[[7, 8, 39]] = False
        assert torch.equal(Y[keep], want[keep])
        assert torch.isnan(Y[7]).all() and torch.isnan(Y[8]).any() and torch.isnan(Y[39]).any()


def test_gradients_against_differences(cuda_lib):
    """<dX, V>, <dgamma, v> and <dbeta, v> against central differences of the
    64-bit forward pass: their error is O(h^2) = 1e-8 of the third derivative,
    the kernel's an fp32 rounding of each entry."""
    T, N, eps, h = 23, 301, 1e-5, 1e-4
    X = _rows(T, N, F32, 3, outlier=False)
    gamma, beta = _params(N, F32, 3)
    dY = _rows(T, N, F32, 4, outlier=False)
    _, S, mean, rstd = cuda_lib.layer_norm_forward(X, gamma, beta, eps=eps)
    dX, dgamma, dbeta = cuda_lib.layer_norm_backward(dY, S, gamma, mean, rstd)

    def loss(x, g, b):
        m = x.mean(1, keepdim=True)
        return (((x - m) / torch.sqrt(((x - m) ** 2).mean(1, keepdim=True) + eps) * g + b) * dY.double()).sum()
    x, g, b = X.double(), gamma.double(), beta.double()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(9)
    for which, grad in ((0, dX), (1, dgamma), (2, dbeta)):
        V = torch.randn(grad.shape, generator=gen, device="cuda", dtype=torch.float64)
        args = [x, g, b]
        up, down = list(args), list(args)
        up[which], down[which] = args[which] + h * V, args[which] - h * V
        diff = float((loss(*up) - loss(*down)) / (2 * h))
        got = float((grad.double() * V).sum())
        scale = float((grad.double().abs() * V.abs()).sum())
        assert abs(got - diff) <= 1e-5 * scale


def test_results_repeat(cuda_lib):
    X, R = _rows(5000, 1024, BF, 1), _rows(5000, 1024, BF, 2)
    gamma, beta = _params(1024, F32, 1)
    a = cuda_lib.layer_norm_forward(X, gamma, beta, residual=R)
    b = cuda_lib.layer_norm_forward(X, gamma, beta, residual=R)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    a = cuda_lib.layer_norm_backward(R, X, gamma, a[2], a[3], dS=R)
    b = cuda_lib.layer_norm_backward(R, X, gamma, b[2], b[3], dS=R)
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_more_than_32_bits_of_elements(cuda_lib):
    """T x N past 2^31: the last rows of a large tensor against the same rows alone."""
    T, N = 270001, 8000
    gamma, beta = _params(N, F32, 1)
    X = torch.empty((T, N), dtype=BF, device="cuda").normal_(generator=torch.Generator(device="cuda").manual_seed(4))
    Y, _, mean, rstd = cuda_lib.layer_norm_forward(X, gamma, beta)
    tail = X[-50:].clone()
    y, _, m, r = cuda_lib.layer_norm_forward(tail, gamma, beta)
    assert torch.equal(Y[-50:], y) and torch.equal(mean[-50:], m) and torch.equal(rstd[-50:], r)
    dX = cuda_lib.layer_norm_backward(X, X, gamma, mean, rstd, weight_grads=False)[0]
    assert torch.equal(dX[-50:], cuda_lib.layer_norm_backward(tail, tail, gamma, m, r, weight_grads=False)[0])


def test_empty(cuda_lib):
    gamma, beta = _params(64, F32, 1)
    X = torch.empty((0, 64), dtype=BF, device="cuda")
    Y, S, mean, rstd = cuda_lib.layer_norm_forward(X, gamma, beta)
    assert Y.shape == (0, 64) and mean.shape == (0,)
    dX, dgamma, dbeta = cuda_lib.layer_norm_backward(X, X, gamma, mean, rstd)
    assert dX.shape == (0, 64) and not dgamma.any() and not dbeta.any()


def test_refusals(cuda_lib):
    X, (gamma, beta) = _rows(4, 64, BF, 1), _params(64, F32, 1)
    with pytest.raises(TypeError):
        cuda_lib.layer_norm_forward(X, gamma, beta.to(BF))
    with pytest.raises(ValueError):
        cuda_lib.layer_norm_forward(X, gamma[:63], beta)
    with pytest.raises(TypeError):
        cuda_lib.layer_norm_forward(X, gamma, beta, residual=X.float())
    with pytest.raises(ValueError):
        cuda_lib.layer_norm_forward(X, gamma, beta, residual=X[:3])
    with pytest.raises(cuda_lib.TffnError):
        cuda_lib.layer_norm_forward(X, gamma, beta, eps=-1.0)
    _, S, mean, rstd = cuda_lib.layer_norm_forward(X, gamma, beta)
    with pytest.raises(ValueError):
        cuda_lib.layer_norm_backward(X, S, gamma, mean[:2], rstd)
    with pytest.raises(TypeError):
        cuda_lib.layer_norm_backward(X, S, gamma, mean, rstd.double())
    with pytest.raises(ValueError):
        cuda_lib.layer_norm_backward(X, S.cpu(), gamma, mean, rstd)
