"""Every tile and grouping of rounds of the matrices' kernel, by the name that
``last_kernel`` gives, held to the iteration in 64 bits: alone, as a step of weights,
skipped, in a graph, on a stream of its own, and with waits that run out.

Bounds are those of test_gpu_matrix_precision.py: 4 times the error of 32-bit products
and 2^-22 of the norm."""
import math

import pytest
import torch

import sharded_optimizer_step_gb300 as ss

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


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


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


# lists that the rule sends to each tile and grouping on 152 SMs: wide, tall, odd
LISTS = {
    "<128, 64>": [(256, 300), (299, 65), (1, 70), (130, 1000)],
    "<128, 64>, rounds in twos": [(520, 2050), (2050, 520), (1500, 600)],
    "<128, 128>": [(300, 300)] * 50 + [(299, 310), (129, 300), (300, 1)],
    "<128, 128>, rounds in twos": [(520, 2050)] * 10 + [(2049, 513), (515, 1999)],
    "<256, 256>": [(397, 411)] * 30 + [(411, 397)] * 8 + [(400, 130), (2, 400)],
    "<256, 256>, rounds in twos": [(1024, 1024), (1024, 4096), (4096, 1024)] * 2 + [
        (1000, 4100), (4093, 515), (777, 1025)],
}


def _only_here():
    if torch.cuda.get_device_properties(0).multi_processor_count != 152:
        pytest.skip("the lists are those of 152 SMs")


def _quintic(u, rounds=5, abc=ss.QUINTIC):
    a, b, c = abc
    x = u / (u.norm() + 1e-7)
    tall = x.shape[0] > x.shape[1]
    x = x.T if tall else x
    for _ in range(rounds):
        g = x @ x.T
        x = a * x + (b * g + c * (g @ g)) @ x
    return x.T if tall else x


def _bound(u, want, rounds=5, abc=ss.QUINTIC):
    """Of the norm of the error."""
    plain = float((_quintic(u.float(), rounds, abc).double() - want).norm())
    return 4 * plain + 2.0 ** -22 * float(want.norm())


@pytest.mark.parametrize("which", LISTS)
@pytest.mark.parametrize("rounds", [5, 3])
def test_every_tile_and_grouping(which, rounds):
    _only_here()
    g = _gen(len(which) + rounds)
    us = [torch.randn(*s, generator=g, device=DEV) * 1e-3 for s in LISTS[which]]
    outs = [torch.full_like(u, 7.0) for u in us]
    ss.orthogonalize(us, out=outs, rounds=rounds)
    if rounds == 5:
        assert ss.last_kernel() == "matrix_rounds" + which
    again = ss.orthogonalize(us, rounds=rounds)
    for u, o, r in zip(us, outs, again):
        want = _quintic(u.double(), rounds)
        # a scalar's chain has its own bound: 300 2^-21
        most = _bound(u, want, rounds) if min(u.shape) > 1 else 300 * 2.0 ** -21 * float(want.norm())
        assert float((o.double() - want).norm()) <= most, u.shape
        assert torch.equal(o, r), u.shape


@pytest.mark.parametrize("which", LISTS)
@pytest.mark.parametrize("rounds,abc", [(8, (1.5, -0.5, 0.0)), (6, (1.875, -1.25, 0.375)),
                                        (4, (-1.5, 0.5, 0.0)), (2, ss.QUINTIC), (7, ss.QUINTIC)])
def test_every_tile_with_other_rounds_and_coefficients(which, rounds, abc):
    """2^-22 in every round.  Of a piece's four additions at full size each is cut off, by
    2^-24 of what is there by then on average (a quarter, a half, three quarters, all of
    it): 2.5 2^-24 of the result, towards zero.  One product with X in a round, or one with X
    and one of the two rounds' factors in two: 2.5 2^-24 a round of all products on X's way,
    five eighths of 2^-22; the halves' roundings go to either side and take less than the
    rest.  All rounds' add up, where 32-bit products round to either side."""
    _only_here()
    g = _gen(rounds)
    us = [torch.randn(*s, generator=g, device=DEV) for s in LISTS[which] if min(s) > 2]
    for u, o in zip(us, ss.orthogonalize(us, rounds=rounds, coefficients=abc)):
        want = _quintic(u.double(), rounds, abc)
        most = _bound(u, want, rounds, abc) + (rounds - 1) * 2.0 ** -22 * float(want.norm())
        assert float((o.double() - want).norm()) <= most, u.shape


@pytest.mark.parametrize("which", LISTS)
@pytest.mark.parametrize("out", [BF, torch.float16])
def test_every_tile_in_16_bits(which, out):
    _only_here()
    g = _gen(len(which))
    us = [torch.randn(*s, generator=g, device=DEV).to(BF) for s in LISTS[which]]
    for u, o in zip(us, ss.orthogonalize(us, out=[torch.empty_like(u, dtype=out) for u in us])):
        want = _quintic(u.double())
        err = ((o.double() - want).abs() - torch.finfo(out).eps / 2 * want.abs()).clamp(min=0)
        sub = 2.0 ** -25 * math.sqrt(u.numel()) if out is torch.float16 else 0.0
        most = _bound(u, want) if min(u.shape) > 1 else 300 * 2.0 ** -21 * float(want.norm())
        assert float(err.norm()) <= most * (1 + torch.finfo(out).eps) + sub, u.shape


@pytest.mark.parametrize("which", LISTS)
def test_every_tile_steps_weights(which):
    _only_here()
    g = _gen(31)
    shapes = LISTS[which]
    start = [(torch.randn(*s, generator=g, device=DEV) * 0.05).to(BF) for s in shapes]
    hp = ss.Muon(lr=2e-3, weight_decay=0.1)
    coef = torch.tensor([0.25], device=DEV)
    grads = [torch.randn(*s, generator=g, device=DEV).to(BF) for s in shapes]
    skip = torch.zeros(1, dtype=torch.int32, device=DEV)

    def steps(how):
        params = [p.clone() for p in start]
        opt = ss.TensorMuon(params, hp)
        lst = ss.TensorList(grads)
        opt.step(lst, grad_coef=coef)
        assert ss.last_kernel() == "matrix_rounds" + which
        first = opt.master.clone(), opt.m.clone()
        if how == "graph":
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                opt.step(lst, grad_coef=coef, skip=skip)
            graph.replay()
            skip.fill_(1)
            graph.replay()                                 # nothing
            skip.zero_()
        elif how == "stream":
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            opt.step(lst, grad_coef=coef, stream=s)
            s.synchronize()
        else:
            skip.fill_(1)
            opt.step(lst, grad_coef=coef, skip=skip)       # nothing
            skip.zero_()
            assert torch.equal(first[0], opt.master) and torch.equal(first[1], opt.m)
            opt.workspace.buf.fill_(255)
            opt.step(lst, grad_coef=coef)
        return first, opt, params

    first, opt, params = steps("eager")
    for k, (p, grad) in enumerate(zip(start, grads)):
        m = 0.05 * 0.25 * grad.double()
        u = 0.95 * m + 0.05 * 0.25 * grad.double()
        s = hp.lr * hp.match_rms * math.sqrt(max(p.shape))
        ortho = _quintic(u)
        want = p.double() * (1 - hp.lr * hp.weight_decay) - s * ortho
        assert float((opt.view(first[1], k).double() - m).abs().max()) <= 4 * 2.0 ** -24 * float(
            m.abs().max())
        # u's two roundings move the result by what the iteration makes of 2^-23 of it: within
        # what 32-bit products are held to; the weights' own two roundings
        most = (_bound(u, ortho) if min(p.shape) > 1 else 300 * 2.0 ** -21 * float(ortho.norm()))
        assert float((opt.view(first[0], k).double() - want).norm()) <= 2 * s * most + 3 * 2.0 ** -24 \
            * float(want.norm()), p.shape
        assert torch.equal(params[k], opt.view(opt.master, k).to(BF))
    for how in ("graph", "stream"):
        _, other, others = steps(how)
        assert torch.equal(other.master, opt.master) and torch.equal(other.m, opt.m), how
        assert all(torch.equal(a, b) for a, b in zip(params, others)), how


@pytest.mark.parametrize("which", LISTS)
def test_waits_that_run_out(which):
    """Every tile's way out: reported, and the next call is right."""
    _only_here()
    us = [torch.randn(*s, generator=_gen(15), device=DEV) for s in LISTS[which]]
    want = ss.orthogonalize(us)
    torch.cuda.synchronize()
    before = ss.set_tma_wait_ns(1)
    try:
        ss.orthogonalize(us)
        torch.cuda.synchronize()
    finally:
        ss.set_tma_wait_ns(before)
    assert ss.device_status(clear=True) & 3
    assert ss.device_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(ss.orthogonalize(us), want))
