"""Orthogonalised matrices and the step that uses them, on the GPU against the
quintic iteration in 64 bits.

A value held as two halves is off by 2^-23 of itself, the product left out
2^-22, so an element of a product is off by 2^-21 of the sum of its terms'
magnitudes; the tensor cores cut off their sums of 256 k at the last bit, 48
times by half a bit of what is there by then, a quarter of the result on average:
48 / 4 / 2 * 2^-23 = 7e-7 of it, downwards.  A round multiplies the settled
values' errors by at most 1.7 or so and adds some 6 such products' errors, so
after five rounds each singular value is off by a few 1e-5 at the worst, the
result in norm by that times the root of its short side: below 1e-3 for sides up
to 1024.  That is asserted of the norm of the whole error (1e-3, not of the
result's norm, which is up to 30); one product of single halves misses it
by 2e-3 to 2e-2 of the norm.  What is measured is 4e-6 to 1e-5 of the norm."""
import math

import pytest
import torch

import sharded_optimizer_step_gb300 as ss

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
ABS = 1e-3


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ss.build()
    yield
    assert ss.device_status() == 0


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _quintic(u, rounds=5, abc=ss.QUINTIC, eps=1e-7):
    a, b, c = abc
    x = u.double()
    x = x / (x.square().sum().sqrt() + eps)
    tall = x.shape[0] > x.shape[1]
    x = x.T if tall else x
    for _ in range(rounds):
        g = x @ x.T
        x = a * x + (b * g + c * g @ g) @ x
    return x.T if tall else x


def _check(got, want, what=""):
    err = (got.double() - want).abs() - torch.finfo(got.dtype).eps / 2 * want.abs()
    err = err.clamp(min=0.0)
    assert bool(torch.isfinite(got).all()), what
    off = float(err.square().sum().sqrt())
    assert off <= ABS, (what, off, float(want.norm()))


SHAPES = [(1, 1), (1, 7), (9, 1), (5, 5), (64, 64), (127, 129), (128, 128), (129, 127),
          (130, 257), (300, 40), (40, 1000), (256, 256), (384, 640), (700, 300), (513, 511)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dt,out_dt", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f32"),
                                       ("bf16", "f16")])
def test_orthogonalize(shape, dt, out_dt):
    u = (torch.randn(*shape, generator=_gen(sum(shape)), device=DEV) * 1e-3).to(DT[dt])
    out = torch.full(shape, 7.0, dtype=DT[out_dt], device=DEV)
    assert ss.orthogonalize(u, out=out) is out
    _check(out, _quintic(u), shape)


def _spectra(m, n, g):
    q, _ = torch.linalg.qr(torch.randn(m, m, generator=g, device=DEV, dtype=torch.float64))
    p, _ = torch.linalg.qr(torch.randn(n, m, generator=g, device=DEV, dtype=torch.float64))
    yield "decaying", (q * torch.logspace(0, -5, m, device=DEV, dtype=torch.float64)) @ p.T
    yield "one direction", q[:, :1] @ p[:, :1].T
    yield "equal", q @ p.T
    steps = torch.ones(m, device=DEV, dtype=torch.float64)
    steps[m // 2:] = 1e-2
    yield "two sizes", (q * steps) @ p.T


@pytest.mark.parametrize("m,n", [(130, 200), (256, 1024), (512, 512)])
def test_spectra(m, n):
    for name, u in _spectra(m, n, _gen(m)):
        u = u.float()
        _check(ss.orthogonalize(u), _quintic(u), name)
        _check(ss.orthogonalize(u.T.contiguous()), _quintic(u.T), name + ", tall")


@pytest.mark.parametrize("size", [1e-30, 1e-12, 1.0, 1e15])
def test_sizes_of_values(size):
    u = torch.randn(150, 170, generator=_gen(1), device=DEV) * size
    # squares below 2^-126 lose bits of the norm, which eps outweighs by then
    _check(ss.orthogonalize(u), _quintic(u), size)


def test_lists_of_all_sizes_and_more_than_a_group():
    g = _gen(2)
    shapes = [(k % 37 + 1, (k * 7) % 150 + 1) for k in range(150)] + [(0, 5), (300, 200), (4, 0)]
    us = [torch.randn(*s, generator=g, device=DEV).bfloat16() for s in shapes]
    outs = ss.orthogonalize(us)
    for u, o in zip(us, outs):
        assert o.shape == u.shape and o.dtype == u.dtype
        if u.numel():
            _check(o, _quintic(u), u.shape)
    alone = [ss.orthogonalize(u) for u in us]
    assert all(torch.equal(p, q) for p, q in zip(outs, alone))
    assert ss.orthogonalize([]) == []


def test_rounds_and_coefficients():
    u = torch.randn(100, 140, generator=_gen(4), device=DEV)
    for rounds, abc in ((1, ss.QUINTIC), (2, ss.QUINTIC), (12, ss.QUINTIC), (8, (1.5, -0.5, 0.0)),
                        (6, (1.875, -1.25, 0.375))):
        got = ss.orthogonalize(u, rounds=rounds, coefficients=abc)
        want = _quintic(u, rounds, abc)
        _check(got, want, (rounds, abc))
    # the cubic iteration settles: rows become orthonormal
    got = ss.orthogonalize(u, rounds=24, coefficients=(1.5, -0.5, 0.0))
    assert float((got @ got.T - torch.eye(100, device=DEV)).abs().max()) < 1e-4


def test_zeros_and_values_that_are_not_finite():
    z = torch.zeros(40, 60, device=DEV)
    assert not ss.orthogonalize(z).any()
    for bad in (float("nan"), float("inf"), 1e30):
        u = torch.randn(40, 60, generator=_gen(5), device=DEV)
        u[3, 4] = bad
        assert bool(torch.isnan(ss.orthogonalize(u)).all()), bad
    # another matrix of the same call is not touched by it
    ok = torch.randn(40, 60, generator=_gen(6), device=DEV)
    u[3, 4] = float("nan")
    got = ss.orthogonalize([u, ok])
    assert bool(torch.isnan(got[0]).all())
    _check(got[1], _quintic(ok))


def test_inputs_outside_bands_and_misaligned():
    g = _gen(7)
    for shift in (0, 1, 3):
        buf = torch.full((131 * 67 + 200,), float("nan"), device=DEV).bfloat16()
        u = buf[64 + shift:64 + shift + 131 * 67].view(131, 67)
        u.copy_(torch.randn(131, 67, generator=g, device=DEV))
        out = torch.full((131 * 67 + 200,), 7.0, device=DEV)
        o = out[64 + shift:64 + shift + 131 * 67].view(131, 67)
        ss.orthogonalize(u, out=o)
        _check(o, _quintic(u), shift)
        assert bool((out[:64 + shift] == 7).all()) and bool((out[64 + shift + 131 * 67:] == 7).all())


# ------------------------------------------------------------------- the step

class _Plain:
    """The step in 64 bits."""

    def __init__(self, params, hps, groups):
        self.p = [p.double() for p in params]
        self.m = [torch.zeros_like(p) for p in self.p]
        self.hps, self.groups = hps, groups

    def step(self, grads, coef=1.0):
        for k, g in enumerate(grads):
            h = self.hps[self.groups[k]]
            g = g.double() * coef
            self.m[k] = h.momentum * self.m[k] + (1 - h.momentum) * g
            u = h.momentum * self.m[k] + (1 - h.momentum) * g if h.nesterov else self.m[k]
            rows, cols = u.shape
            s = (h.match_rms * math.sqrt(max(rows, cols)) if h.match_rms
                 else math.sqrt(max(1, rows / cols)))
            self.p[k] = self.p[k] * (1 - h.lr * h.weight_decay) - h.lr * s * _quintic(u)


def _scale(h, shape):
    return h.lr * (h.match_rms * math.sqrt(max(shape)) if h.match_rms
                   else math.sqrt(max(1, shape[0] / shape[1])))


STEP_SHAPES = [(64, 200), (200, 64), (129, 131), (1, 30), (30, 1), (256, 256)]


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("param_dt", ["bf16", "f16"])
def test_steps(dt, param_dt):
    g = _gen(11)
    params = [(torch.randn(*s, generator=g, device=DEV) * 0.05).to(DT[param_dt])
              for s in STEP_SHAPES]
    hps = [ss.Muon(lr=2e-3, weight_decay=0.1), ss.Muon(lr=1e-2, momentum=0.8, match_rms=0.0,
                                                       nesterov=False, weight_decay=0.0)]
    groups = [0, 0, 1, 1, 0, 0]
    opt = ss.TensorMuon(params, hps, groups=groups)
    plain = _Plain(params, hps, groups)
    coef = torch.tensor([0.25], device=DEV)
    for t in range(3):
        grads = [torch.randn(*s, generator=g, device=DEV).to(DT[dt]) for s in STEP_SHAPES]
        opt.step(grads, grad_coef=coef if t else None)
        plain.step(grads, 0.25 if t else 1.0)
        for k, s in enumerate(STEP_SHAPES):
            m, p = opt.view(opt.m, k), opt.view(opt.master, k)
            # each step's own roundings, three of 2^-24 of the larger term, on what was there
            assert float((m.double() - plain.m[k]).abs().max()) <= 6 * (t + 1) * 2.0 ** -24 * max(
                1.0, float(plain.m[k].abs().max())) * 6
            tol = (t + 1) * _scale(hps[groups[k]], s) * ABS + 4 * (t + 1) * 2.0 ** -24 * float(
                plain.p[k].norm())
            assert float((p.double() - plain.p[k]).norm()) <= tol, (t, s)
            assert torch.equal(params[k], p.to(DT[param_dt])), s
    # the gaps between the matrices stay zero
    held = torch.zeros(opt.flat, dtype=torch.bool, device=DEV)
    for o, n in zip(opt.offsets, opt.numels):
        held[o:o + n] = True
    assert not opt.master[~held].any() and not opt.m[~held].any()


def test_skip_word_and_lists():
    g = _gen(12)
    params = [torch.randn(70, 90, generator=g, device=DEV).bfloat16() for _ in range(3)]
    opt = ss.TensorMuon(params, ss.Muon())
    grads = ss.TensorList([torch.randn(70, 90, generator=g, device=DEV) for _ in params])
    opt.step(grads)
    before = [t.clone() for t in (opt.master, opt.m, *params)]
    skip = torch.ones(1, dtype=torch.int32, device=DEV)
    opt.step(grads, skip=skip)
    assert all(torch.equal(a, b) for a, b in zip(before, (opt.master, opt.m, *params)))
    skip.zero_()
    opt.step(grads, skip=skip)
    assert not torch.equal(before[0], opt.master)


def test_repeats_graphs_and_streams():
    g = _gen(13)
    shapes = [(300, 500), (500, 300), (128, 64)]
    start = [torch.randn(*s, generator=g, device=DEV).bfloat16() for s in shapes]
    grads = ss.TensorList([torch.randn(*s, generator=g, device=DEV) for s in shapes])

    def steps(how):
        params = [p.clone() for p in start]
        opt = ss.TensorMuon(params, ss.Muon(lr=0.01))
        opt.step(grads)
        if how == "graph":
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                opt.step(grads)
            graph.replay()
            graph.replay()
        elif how == "stream":
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            opt.step(grads, stream=s)
            opt.step(grads, stream=s)
            s.synchronize()
        else:
            opt.workspace.buf.fill_(255)         # any contents
            opt.step(grads)
            opt.step(grads)
        return opt.master.clone(), opt.m.clone(), params
    want = steps("eager")
    for how in ("eager", "graph", "stream"):
        got = steps(how)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), how
        assert all(torch.equal(p, q) for p, q in zip(got[2], want[2])), how


def test_large_square_and_wide():
    g = _gen(14)
    us = [torch.randn(1024, 1024, generator=g, device=DEV),
          torch.randn(1000, 4100, generator=g, device=DEV),
          torch.randn(4096, 512, generator=g, device=DEV)]
    for u, o in zip(us, ss.orthogonalize(us)):
        _check(o, _quintic(u), u.shape)


def test_waits_that_run_out_are_reported():
    u = torch.randn(600, 900, generator=_gen(15), device=DEV)
    want = ss.orthogonalize(u)
    torch.cuda.synchronize()
    before = ss.set_tma_wait_ns(1)
    try:
        ss.orthogonalize(u)
        torch.cuda.synchronize()
    finally:
        ss.set_tma_wait_ns(before)
    assert ss.device_status(clear=True) & 3
    assert ss.device_status() == 0
    assert torch.equal(ss.orthogonalize(u), want)


def test_a_list_as_output():
    g = _gen(5)
    us = [torch.randn(40, 30, device=DEV, generator=g), torch.randn(9, 70, device=DEV, generator=g)]
    want = ss.orthogonalize(us)
    outs = ss.TensorList([torch.empty_like(u) for u in us])
    assert ss.orthogonalize(us, out=outs) is outs
    for a, b in zip(outs.tensors, want):
        assert torch.equal(a, b)
