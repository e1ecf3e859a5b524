"""The oracle of the embedding, layer norm and the orthogonalised step against
things other than itself: torch's own layers and their autograd in float64,
singular value decompositions, and differences."""
import numpy as np
import pytest
import torch

from oracle import model_ops as OM


def _rand(seed, *shape):
    return np.random.default_rng(seed).normal(size=shape)


def test_embedding_against_torch():
    table, ids = _rand(1, 13, 5), np.array([3, 0, 12, 3, -1, 13, 7, 3])
    keep = (ids >= 0) & (ids < 13)
    t = torch.tensor(table, requires_grad=True)
    rows = torch.nn.functional.embedding(torch.tensor(ids[keep]), t) * 2.5
    got = OM.embedding(table, ids, 2.5)
    assert np.array_equal(got[keep], rows.detach().numpy()) and not got[~keep].any()
    d = _rand(2, len(ids), 5)
    (rows * torch.tensor(d[keep])).sum().backward()
    assert np.allclose(OM.embedding_grad(d, ids, 13, 2.5), t.grad.numpy(), rtol=1e-14, atol=1e-14)


@pytest.mark.parametrize("affine", [False, True])
def test_layer_norm_against_torch(affine):
    x, d = _rand(3, 6, 17) * 3 + 1, _rand(4, 6, 17)
    w, b = (_rand(5, 17), _rand(6, 17)) if affine else (None, None)
    tx, tw, tb = (torch.tensor(v, requires_grad=True) if v is not None else None
                  for v in (x, w, b))
    y = torch.nn.functional.layer_norm(tx, (17,), tw, tb, 1e-5)
    out, mean, rstd = OM.layer_norm(x, w, b, 1e-5)
    assert np.allclose(out, y.detach().numpy(), rtol=1e-12, atol=1e-12)
    assert np.allclose(mean, x.mean(1)) and np.allclose(rstd, (x.var(1) + 1e-5) ** -0.5)
    y.backward(torch.tensor(d))
    d_x, d_w, d_b = OM.layer_norm_grad(d, x, mean, rstd, w)
    assert np.allclose(d_x, tx.grad.numpy(), rtol=1e-11, atol=1e-11)
    if affine:
        assert np.allclose(d_w, tw.grad.numpy(), rtol=1e-11, atol=1e-11)
        assert np.allclose(d_b, tb.grad.numpy(), rtol=1e-11, atol=1e-11)


@pytest.mark.parametrize("shape", [(7, 7), (5, 19), (23, 4), (1, 6), (6, 1)])
@pytest.mark.parametrize("rounds,abc", [(5, OM.QUINTIC), (3, (1.5, -0.5, 0.0)),
                                        (2, (1.875, -1.25, 0.375))])
def test_orthogonalize_acts_on_the_singular_values(shape, rounds, abc):
    u = _rand(sum(shape), *shape)
    p, s, q = np.linalg.svd(u, full_matrices=False)
    s = s / (np.sqrt((s * s).sum()) + 1e-7)
    for _ in range(rounds):
        s = abc[0] * s + abc[1] * s ** 3 + abc[2] * s ** 5
    assert np.allclose(OM.orthogonalize(u, rounds, abc), (p * s) @ q, rtol=0, atol=1e-12)


def test_orthogonalize_brings_singular_values_near_one():
    s = np.linalg.svd(OM.orthogonalize(_rand(9, 40, 60)), compute_uv=False)
    assert 0.65 < s.min() and s.max() < 1.25
    # the cubic iteration settles on the nearest matrix with orthonormal rows
    x = OM.orthogonalize(_rand(9, 10, 30), 40, (1.5, -0.5, 0.0))
    p, _, q = np.linalg.svd(_rand(9, 10, 30), full_matrices=False)
    assert np.allclose(x, p @ q, atol=1e-9)


def test_muon_step_by_hand():
    # a 1 x 1 matrix: u / |u| = 1 but for eps, f five times from 1, by hand below
    f = 1.0
    for _ in range(5):
        f = 3.4445 * f - 4.7750 * f ** 3 + 2.0315 * f ** 5
    p, m = OM.muon_step(np.array([[2.0]]), np.array([[0.5]]), np.array([[4.0]]), 0.1, 0.5, 0.01,
                        0.0, eps=0.0)
    assert m[0, 0] == 2.25 and abs(p[0, 0] - (2.0 - 0.002 - 0.1 * f)) < 1e-12
    assert OM.muon_scale(8, 2, 0.0) == 2.0 and OM.muon_scale(2, 8, 0.0) == 1.0
    assert OM.muon_scale(9, 16, 0.25) == 1.0
    # without nesterov the update is the momentum's direction
    a, _ = OM.muon_step(np.zeros((2, 3)), _rand(1, 2, 3), _rand(2, 2, 3), 1.0, 0.9, 0.0, 0.0,
                        nesterov=False)
    m = 0.9 * _rand(1, 2, 3) + 0.1 * _rand(2, 2, 3)
    assert np.allclose(a, -OM.orthogonalize(m), atol=1e-12)
