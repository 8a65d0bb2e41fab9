"""Orthogonalised updates on the GPU against the iteration in 64 bits.

Tolerance.  Operands are rounded to 11 bits (2^-12 at most, 2^-13 or so on average) three times a
step; in a 64-bit simulation of those roundings the result of 5 steps is 1e-3 to 1.7e-3 off (2-norm)
for spectra from flat to steep, so 2e-3 is allowed for them, and 2^-9 for the output's rounding.
Few-entry matrices do not average: their tolerance is the sum of 15 roundings of 2^-12, grown by the
iteration's slope near 1 (at most 3.5) in each step they pass: 8e-3.
"""
import math

import pytest
import torch

import compressed_pseudo_gradient_gb300 as spl

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
COEF = spl.NEWTON_SCHULZ


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def iterate(u, steps=5, coef=COEF, eps=1e-7):
    x = u.double()
    tall = x.shape[-2] > x.shape[-1]
    x = x.mT if tall else x
    x = x / (x.square().sum((-2, -1), keepdim=True).sqrt() + eps)
    for _ in range(steps):
        a = x @ x.mT
        x = coef[0] * x + (coef[1] * a + coef[2] * (a @ a)) @ x
    return x.mT if tall else x


def off(got, ref):
    return ((got.double() - ref).norm() / ref.norm()).item()


def limit(m, n):
    return (2e-3 if min(m, n) >= 32 else 8e-3) + 2.0 ** -9


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("m,n", [(1, 1), (1, 7), (9, 1), (2, 2), (8, 8), (17, 33), (64, 64), (63, 65), (100, 257),
                                 (128, 128), (129, 127), (200, 1000), (1000, 136), (256, 256), (257, 511), (384, 640),
                                 (513, 700), (1000, 999), (96, 5000), (700, 2100),
                                 # around the sizes that one cluster holds
                                 (128, 4096), (100, 4001), (4096, 31), (128, 4097), (64, 1100), (700, 128), (129, 256),
                                 (256, 130), (255, 255), (256, 257), (200, 136)])
def test_matrix(m, n, dtype):
    u = torch.randn(m, n, generator=gen(m * n), device=DEV).to(dtype) * 1e-3
    got = spl.orthogonalize(u)
    assert got.dtype == torch.bfloat16 and got.shape == (m, n)
    assert off(got, iterate(u)) <= limit(m, n)


@pytest.mark.parametrize("batch,m,n", [(1, 24, 5000), (1, 32, 9001), (2, 48, 6000), (1, 100, 5000), (1, 128, 8192),
                                       (40, 48, 4096)])
def test_few_long_rows(batch, m, n):
    """Few rows average roundings less, and are multiplied in two planes: still 2e-3 before the output's
    rounding, whose 1.7e-3 (2-norm, mantissas spread evenly) adds in quadrature."""
    u = torch.randn(batch, m, n, generator=gen(m), device=DEV)
    u *= torch.exp(math.log(100) * torch.rand(batch, m, 1, generator=gen(n), device=DEV))
    for x in (u, u.mT.contiguous()):
        got, ref = spl.orthogonalize(x), iterate(x)
        for i in range(batch):
            assert off(got[i], ref[i]) <= math.hypot(2e-3, 1.7e-3)


@pytest.mark.parametrize("batch,m,n", [(12, 520, 1100), (3, 2100, 2300), (1, 2560, 3000)])
@pytest.mark.parametrize("tall", [False, True])
def test_many_tiles(batch, m, n, tall):
    """Enough 256 x 256 tiles for pairs of CTAs, ragged ones among them."""
    u = torch.randn(batch, *((n, m) if tall else (m, n)), generator=gen(m), device=DEV)
    got, ref = spl.orthogonalize(u), iterate(u)
    for i in range(batch):
        assert off(got[i], ref[i]) <= limit(m, n)


@pytest.mark.parametrize("power", [0.0, 0.5, 1.0, 1.5, 2.0])
@pytest.mark.parametrize("m,n", [(256, 256), (300, 900)])
def test_spread_of_singular_values(m, n, power):
    """Orthogonal factors times a falling spectrum: small directions are not lost to the large ones'
    rounding."""
    g = gen(5)
    q1 = torch.linalg.qr(torch.randn(m, m, generator=g, device=DEV, dtype=torch.float64))[0]
    q2 = torch.linalg.qr(torch.randn(n, m, generator=g, device=DEV, dtype=torch.float64))[0]
    s = torch.arange(1, m + 1, device=DEV).double() ** -power
    u = ((q1 * s) @ q2.T).float()
    assert off(spl.orthogonalize(u), iterate(u)) <= limit(m, n)


def test_result_is_nearly_orthogonal():
    """For a well-spread matrix 5 steps bring every singular value to 0.68 .. 1.14."""
    u = torch.randn(300, 700, generator=gen(1), device=DEV)
    s = torch.linalg.svdvals(spl.orthogonalize(u).float())
    assert 0.65 <= s.min() and s.max() <= 1.16


@pytest.mark.parametrize("batch,m,n,extra", [(3, 40, 72, 0), (5, 130, 50, 6), (2, 300, 260, 3), (7, 1, 5, 1)])
def test_stack_of_strided_matrices(batch, m, n, extra):
    u = torch.randn(batch, m + 1, n + extra, generator=gen(batch), device=DEV).bfloat16()[:, :m, :n]
    u *= torch.logspace(-6, 2, batch, device=DEV)[:, None, None]
    got = spl.orthogonalize(u)
    ref = iterate(u)
    for i in range(batch):
        assert off(got[i], ref[i]) <= limit(m, n)
        assert torch.equal(spl.orthogonalize(u[i]), got[i])


@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_momentum(nesterov, dtype):
    g = gen(3)
    for shape in ((90, 200), (2, 150, 70)):
        m = torch.randn(shape, generator=g, device=DEV)
        m64 = m.double()
        for _ in range(3):
            u = torch.randn(shape, generator=g, device=DEV).to(dtype)
            got = spl.orthogonalize(u, momentum=m, mu=0.9, nesterov=nesterov)
            mu = torch.tensor(0.9, dtype=torch.float32).double().item()
            m64 = mu * m64 + u.double()
            assert (m.double() - m64).abs().max() <= 3 * 2.0 ** -24 * 8 * m64.abs().max()
            v = u.double() + mu * m64 if nesterov else m64
            assert off(got, iterate(v)) <= limit(90, 200)
            m64 = m.double()


def test_steps_and_coefficients():
    u = torch.randn(120, 300, generator=gen(2), device=DEV)
    for steps, coef in ((1, COEF), (2, COEF), (8, COEF), (6, (1.5, -0.5, 0.0)), (3, (2.0, -1.5, 0.5))):
        got = spl.orthogonalize(u, steps=steps, coefficients=coef)
        assert off(got, iterate(u, steps, coef)) <= limit(120, 300) * max(1.0, steps / 5)


def test_zeros_and_nonfinite():
    flags = torch.zeros(1, dtype=torch.int32, device=DEV)
    assert (spl.orthogonalize(torch.zeros(40, 60, device=DEV), flags=flags) == 0).all()
    assert spl.flags_status(flags) == 0
    u = torch.randn(2, 40, 60, device=DEV)
    u[1, 3, 4] = math.inf
    got = spl.orthogonalize(u, flags=flags)
    assert spl.flags_status(flags) == 4
    assert torch.isfinite(got[0]).all() and torch.isnan(got[1]).all()


@pytest.mark.parametrize("size", [1e-12, 1e-5, 1.0, 1e9])
def test_scale_of_the_update_does_not_matter(size):
    u = torch.randn(64, 200, generator=gen(7), device=DEV)
    assert off(spl.orthogonalize(u * size, eps=0.0), iterate(u, eps=0.0)) <= limit(64, 200)


def test_same_bits_on_another_stream_with_a_kept_workspace():
    u = torch.randn(300, 500, generator=gen(6), device=DEV)
    a = spl.orthogonalize(u)
    ws = torch.full((spl.orthogonalize_workspace(u.shape),), 255, dtype=torch.uint8, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        v = u * 1
        for _ in range(3):
            b = spl.orthogonalize(v, workspace=ws)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(a, b)


def test_refusals():
    u = torch.randn(20, 30, device=DEV)
    for call in (lambda: spl.orthogonalize(u.t()), lambda: spl.orthogonalize(u[0]),
                 lambda: spl.orthogonalize(u[:0]), lambda: spl.orthogonalize(u, momentum=u[:10]),
                 lambda: spl.orthogonalize(u, out=torch.empty(30, 20, dtype=torch.bfloat16, device=DEV)),
                 lambda: spl.orthogonalize(u, workspace=torch.empty(10, dtype=torch.uint8, device=DEV)),
                 lambda: spl.orthogonalize(u.expand(3, 20, 30))):
        with pytest.raises(ValueError):
            call()
    for kw in (dict(steps=0), dict(coefficients=(9.0, 0.0, 0.0)), dict(eps=-1.0)):
        with pytest.raises(spl.SplError):
            spl.orthogonalize(u, **kw)
    with pytest.raises(TypeError):
        spl.orthogonalize(u.double())
