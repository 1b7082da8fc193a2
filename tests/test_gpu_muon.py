"""muon_orthogonalize against the iteration in 64 bits.

Tolerance (of the result's norm): X, A and the polynomial's matrix are rounded
to fp16 (rms 2^-11 / sqrt(3) times 0.75 = 2.1e-4 of their norms) three times in
each of five steps, and a relative error of X grows by at most the polynomial's
slope, 3.44, in a step while it grows X itself by as much, and shrinks after;
the matrix's rounding counts up to 3.44 times where it multiplies X.  In
quadrature sqrt(15) 2.1e-4 3.44 = 2.8e-3, with bf16's 1.7e-3 on the result
3.3e-3; 5e-3 is allowed."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
A, B, C = 3.4445, -4.7750, 2.0315


def _exact(G, steps=5):
    X = G.double()
    tall = X.shape[-2] > X.shape[-1]
    if tall:
        X = X.mT
    X = X / (torch.linalg.matrix_norm(X, keepdim=True) + 1e-7)
    for _ in range(steps):
        S = X @ X.mT
        X = A * X + (B * S + C * S @ S) @ X
    return X.mT if tall else X


def _matrix(*shape, dtype=F32, seed=0, scale=1e-3):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _check(tffn, G, steps=5, tol=5e-3):
    out = tffn.muon_orthogonalize(G, steps=steps)
    tffn.check()
    assert out.dtype == BF and out.shape == G.shape
    want = _exact(G, steps)
    err = (out.double() - want).flatten(-2).norm(dim=-1) / want.flatten(-2).norm(dim=-1)
    assert float(err.max()) <= tol, f"{float(err.max()):.2e}"
    return out


SHAPES = [
    (1, 1), (1, 100), (100, 1), (2, 3), (8, 8), (29, 48), (64, 64), (50, 9000), (3000, 16),
    (127, 129), (128, 256), (256, 128), (255, 257), (256, 256), (257, 255), (256, 1024), (1024, 256),
    (513, 520), (600, 2000), (2000, 333), (1000, 1000), (1100, 4104), (4096, 1024),
]


@pytest.mark.parametrize("m,n", SHAPES)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_against_64_bits(cuda_lib, m, n, dtype):
    _check(cuda_lib, _matrix(m, n, dtype=dtype, seed=m + n))


@pytest.mark.parametrize("batch,m,n", [(2, 100, 300), (3, 700, 520), (8, 256, 1024), (5, 1030, 250), (70, 33, 17),
                                       (1, 64, 64), (3, 64, 31)])
def test_stacks(cuda_lib, batch, m, n):
    G = _matrix(batch, m, n, seed=batch)
    G *= torch.logspace(-3, 3, batch, device="cuda")[:, None, None]   # each entry is normalised by itself
    out = _check(cuda_lib, G)
    # an entry of a stack is the matrix alone
    alone = cuda_lib.muon_orthogonalize(G[batch - 1].contiguous())
    assert float((out[batch - 1].float() - alone.float()).norm() / alone.float().norm()) < 4e-3


def test_large_stack(cuda_lib):
    """More entries than one launch's counters hold."""
    out = _check(cuda_lib, _matrix(3000, 72, 80, seed=4), tol=8e-3)     # the worst of 3000 small matrices
    assert cuda_lib.last_launch_count() > 3
    assert torch.isfinite(out).all()
    _check(cuda_lib, _matrix(3000, 24, 40, seed=4))


@pytest.mark.parametrize("m,n", [(31, 33), (32, 4000), (33, 33), (63, 65), (64, 14336), (5000, 64), (65, 65), (64, 1),
                                 (33, 1000)])
@pytest.mark.parametrize("steps", [1, 5, 8])
def test_small_sides(cuda_lib, m, n, steps):
    """A side of at most 64 is iterated in fp32: only the result's rounding to
    bf16 (1.7e-3 of its norm) is left; 2.2e-3 is allowed.  (65 is not small.)"""
    _check(cuda_lib, _matrix(m, n, seed=m + n), steps=steps, tol=2.2e-3 if min(m, n) <= 64 else 5e-3)
    _check(cuda_lib, _matrix(3, m, n, seed=m + n, dtype=BF), steps=steps, tol=2.2e-3 if min(m, n) <= 64 else 5e-3)


@pytest.mark.parametrize("steps", [1, 2, 5, 6, 10, 11])
def test_steps(cuda_lib, steps):
    _check(cuda_lib, _matrix(192, 320, seed=steps), steps=steps)
    _check(cuda_lib, _matrix(320, 190, seed=steps), steps=steps)


def test_singular_values_end_near_one(cuda_lib):
    """A matrix with singular values between 1 and 30."""
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    U, _ = torch.linalg.qr(torch.randn((300, 300), generator=g, device="cuda", dtype=torch.float64))
    V, _ = torch.linalg.qr(torch.randn((900, 300), generator=g, device="cuda", dtype=torch.float64))
    G = (U * torch.logspace(0, 1.477, 300, device="cuda", dtype=torch.float64)) @ V.t()
    s = torch.linalg.svdvals(cuda_lib.muon_orthogonalize(G.float()).double())
    # the iteration maps such values into [0.67, 1.21]; the rounding moves them by under 2 %
    assert float(s.min()) > 0.65 and float(s.max()) < 1.24


@pytest.mark.parametrize("scale", [1e-30, 1e-12, 1e-3, 1.0, 1e15, 1e25])
def test_scales(cuda_lib, scale):
    """Norms far below the 1e-7 (the result is then nearly zero, as defined) and
    norms whose square passes fp32's range."""
    G = _matrix(96, 160, seed=3, scale=scale)
    out = cuda_lib.muon_orthogonalize(G).double()
    want = _exact(G)
    if scale == 1e-30:
        assert not out.any()    # X itself, 1e-23, is far below any step of fp16
    else:
        assert float((out - want).norm() / want.norm()) <= 5e-3


def test_zero_and_nan(cuda_lib):
    G = torch.zeros((3, 40, 72), device="cuda")
    assert not cuda_lib.muon_orthogonalize(G).any()
    G[0] = _matrix(40, 72, seed=1)
    G[2] = _matrix(40, 72, seed=2)
    want = cuda_lib.muon_orthogonalize(G)
    G[1, 3, 4] = float("nan")
    out = cuda_lib.muon_orthogonalize(G)
    assert torch.isnan(out[1]).all()
    assert torch.equal(out[0], want[0]) and torch.equal(out[2], want[2])


def test_unaligned(cuda_lib):
    """A contiguous matrix that starts one element into its storage."""
    for dtype in (BF, F32):
        s = torch.empty(200 * 328 + 1, dtype=dtype, device="cuda")
        G = s[1:].view(200, 328)
        G.copy_(_matrix(200, 328, dtype=dtype, seed=6))
        want = cuda_lib.muon_orthogonalize(G.clone())
        assert torch.equal(cuda_lib.muon_orthogonalize(G), want)


def test_results_repeat(cuda_lib):
    for G in (_matrix(1024, 2048, seed=7), _matrix(4, 700, 300, seed=8)):
        assert torch.equal(cuda_lib.muon_orthogonalize(G), cuda_lib.muon_orthogonalize(G))


def test_empty_and_refusals(cuda_lib):
    assert cuda_lib.muon_orthogonalize(torch.empty((0, 8), device="cuda")).shape == (0, 8)
    assert cuda_lib.muon_orthogonalize(torch.empty((0, 4, 8), device="cuda")).shape == (0, 4, 8)
    G = _matrix(16, 24)
    with pytest.raises(TypeError):
        cuda_lib.muon_orthogonalize(G.half())
    with pytest.raises(ValueError):
        cuda_lib.muon_orthogonalize(G.t())
    with pytest.raises(ValueError):
        cuda_lib.muon_orthogonalize(G[0])
    with pytest.raises(cuda_lib.TffnError):
        cuda_lib.muon_orthogonalize(G, steps=0)
