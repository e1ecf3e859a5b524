"""How exact the orthogonalisation's products are: beside the same iteration in
32-bit products, both against 64 bits.

A value held as two halves is off by up to 2^-22 of itself, a 32-bit one by 2^-24: a
factor of 4 in what the operands bring, as the sums are added up in 32 bits on both
sides.  A product's result, as halves again, adds 2^-22 where 32-bit values happen to
be exact.  So the whole error may be 4 times that of 32-bit products and 2^-22 of the
result's norm.  Sums that the tensor cores cut off over 256 of k are off by 7e-7 in one
round and pass neither bound.

A 1 x n matrix is its norm's chain of scalars: a factor a + b t + c t^2 is off by
(3.4445 + 4.775 + 2.0315) / 0.70 = 15 times its terms' 2^-21, five of them by 75 2^-21,
and the map multiplies a relative error by at most 1.8 a round where it does not shrink
it: below 300 2^-21 = 1.4e-4 of each element.  (Without the lower halves 2e-2.)"""
import pytest
import torch

import sharded_optimizer_step_gb300 as ss

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ss.build()
    tf32 = torch.backends.cuda.matmul.allow_tf32
    torch.backends.cuda.matmul.allow_tf32 = False
    yield
    torch.backends.cuda.matmul.allow_tf32 = tf32
    assert ss.device_status() == 0


def _quintic(u, rounds):
    """In u's own type."""
    a, b, c = ss.QUINTIC
    x = u / (u.norm() + 1e-7)
    tall = x.shape[0] > x.shape[1]
    x = x.T if tall else x
    for _ in range(rounds):
        g = x @ x.T
        x = a * x + (b * g + c * (g @ g)) @ x
    return x.T if tall else x


def _spectra(m, n, g):
    q, _ = torch.linalg.qr(torch.randn(m, m, generator=g, device=DEV, dtype=torch.float64))
    p, _ = torch.linalg.qr(torch.randn(n, m, generator=g, device=DEV, dtype=torch.float64))
    yield "random", torch.randn(m, n, generator=g, device=DEV)
    yield "decaying", (q * torch.logspace(0, -5, m, device=DEV, dtype=torch.float64)) @ p.T
    part = torch.zeros(m, device=DEV, dtype=torch.float64)
    part[:max(1, m // 4)] = 1
    yield "a quarter of the rank", (q * part) @ p.T
    yield "one direction", q[:, :1] @ p[:, :1].T
    yield "two sizes", (q * torch.where(part > 0, 1.0, 1e-2)) @ p.T


def _off(got, want):
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.parametrize("shape", [(64, 64), (256, 256), (100, 1000), (256, 2048), (700, 700),
                                   (520, 2050), (1024, 4096), (3000, 770)])
@pytest.mark.parametrize("rounds", [1, 3, 4, 5])
def test_as_exact_as_32_bit_products(shape, rounds):
    g = torch.Generator(device=DEV).manual_seed(sum(shape))
    m, n = min(shape), max(shape)
    for name, u in _spectra(m, n, g):
        u = (u if shape[0] <= shape[1] else u.T).float().contiguous()
        want = _quintic(u.double(), rounds)
        plain = _off(_quintic(u, rounds), want)
        off = _off(ss.orthogonalize(u, rounds=rounds), want)
        assert off <= 4 * plain + 2.0 ** -22, (name, off, plain)


@pytest.mark.parametrize("shape", [(1, 1), (1, 7), (9, 1), (1, 300)])
def test_rows_element_by_element(shape):
    u = torch.randn(*shape, generator=torch.Generator(device=DEV).manual_seed(3), device=DEV)
    want = _quintic(u.double(), 5)
    got = ss.orthogonalize(u).double()
    assert bool(((got - want).abs() <= 300 * 2.0 ** -21 * want.abs()).all())


@pytest.mark.parametrize("shape", [(150, 170), (256, 256), (600, 2050), (3, 5)])
@pytest.mark.parametrize("size", [1e18, 6e18, 1.8e19])
def test_elements_whose_squares_fit(shape, size):
    """Squares below 3.4e38 whose sum is not: the norm is formed all the same.  (An
    element beyond gives NaNs.)"""
    g = torch.Generator(device=DEV).manual_seed(7)
    small = torch.randn(*shape, generator=g, device=DEV).clamp(-1, 1)
    u = small * size
    want = _quintic(u.double(), 5)
    off, plain = _off(ss.orthogonalize(u), want), _off(_quintic(small, 5), want)
    assert off <= 4 * plain + 2.0 ** -22, (off, plain)
    u[-1, -1] = 1.9e19
    assert bool(torch.isnan(ss.orthogonalize(u)).all())


def test_a_step_on_elements_whose_squares_fit():
    g = torch.Generator(device=DEV).manual_seed(8)
    params = [torch.randn(300, 200, generator=g, device=DEV).bfloat16() for _ in range(2)]
    grad = torch.randn(300, 200, generator=g, device=DEV)
    opt = ss.TensorMuon(params, ss.Muon(lr=1.0, weight_decay=0.0))
    before = opt.master.clone()
    opt.step([grad, grad * 2.0 ** 61])                  # the same direction
    a, b = (opt.view(opt.master, k) - opt.view(before, k) for k in (0, 1))
    # the masters' own roundings, 2^-24 of values up to 4, beside the results'
    assert float((a - b).norm()) <= 1e-5 * float(a.norm()) + 2.0 ** -22 * 245
