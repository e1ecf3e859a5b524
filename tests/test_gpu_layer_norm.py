"""Layer norm and its gradients on the GPU against plain 64-bit formulas.

Bounds, with u = 2^-24 and a sum of c terms taken by threads of at most
c / 512 + 32 terms each, five shuffles and sixteen warps, so at most
depth = c / 512 + 56 additions deep:
  mean        depth u mean|x|                                   (em)
  variance    (depth + 4) u var + em^2 (the first power of em drops out of a sum of
              differences from the mean), so rstd: half of it relative, and 3 u
  out         r |w| (em + |x - mean| (rel + 4 u)) + 2 u |b|, half a step of out
Backward from the given mean and rstd: xh is 3 u off; the two sums
(depth + 6) u of the sum of magnitudes; the rest a few u of each term; a
column's sum takes rows / 64 + 64 additions at most."""
import pytest
import torch

import sharded_optimizer_step_gb300 as ss

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ss.build()
    yield
    assert ss.device_status() == 0


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _matrix(x, dt, stride, shift, fill=float("nan")):
    rows, cols = x.shape
    buf = torch.full(((rows + 2) * stride + shift + 16,), fill, dtype=dt, device=DEV)
    view = buf[stride + shift:stride + shift + rows * stride].view(rows, stride)[:, :cols]
    view.copy_(x)
    return buf, view


def _untouched(buf, view, fill):
    held = torch.zeros(buf.shape, dtype=torch.bool, device=DEV)
    torch.as_strided(held, view.shape, view.stride(), view.storage_offset())[:] = True
    return bool((buf[~held] == fill).all())


def _half(dt, value, at_least=0.0):
    """Half a step of a result of that size, subnormal ones included."""
    return torch.finfo(dt).eps / 2 * value.abs() + torch.finfo(dt).tiny * torch.finfo(dt).eps / 2


def _depth(cols):
    return cols / 512 + 56


def _check(got, want, tol, what):
    bad = ~((got.double() - want).abs() <= tol * (1 + 1e-9))
    assert not bad.any(), (what, torch.nonzero(bad)[:4], (got.double() - want)[bad][:4], tol[bad][:4])


def _forward(x, w, b, eps, y):
    cols = x.shape[1]
    xd = x.double()
    mean = xd.mean(1, keepdim=True)
    xc = xd - mean
    var = (xc * xc).mean(1, keepdim=True)
    r = (var + eps) ** -0.5
    wd = w.double() if w is not None else torch.ones(cols, dtype=torch.float64, device=DEV)
    bd = b.double() if b is not None else torch.zeros(cols, dtype=torch.float64, device=DEV)
    want = xc * r * wd + bd
    em = _depth(cols) * U * xd.abs().mean(1, keepdim=True)
    rel = ((_depth(cols) + 4) * U * var + em * em) / (2 * (var + eps)) + 3 * U
    _check(y.mean, mean[:, 0], em[:, 0] + U * mean[:, 0].abs(), "mean")
    _check(y.rstd, r[:, 0], (r * rel)[:, 0], "rstd")
    tol = r * wd.abs() * (em + xc.abs() * (rel + 4 * U)) + 2 * U * bd.abs()
    _check(y.out, want, tol + _half(x.dtype, want.abs() + tol), "out")


def _backward(d, x, mean, r, w, g, old_w=None, old_b=None, w_dt=None):
    rows, cols = x.shape
    dd, xd = d.double(), x.double()
    wd = w.double() if w is not None else torch.ones(cols, dtype=torch.float64, device=DEV)
    m, r = mean.double()[:, None], r.double()[:, None]
    xh = (xd - m) * r
    gg = dd * wd
    c1, c2 = gg.mean(1, keepdim=True), (gg * xh).mean(1, keepdim=True)
    if g.d_x is not None:
        want = r * (gg - c1 - xh * c2)
        e1 = (_depth(cols) + 3) * U * gg.abs().mean(1, keepdim=True)
        e2 = (_depth(cols) + 7) * U * (gg * xh).abs().mean(1, keepdim=True)
        tol = r * (e1 + xh.abs() * e2 + 5 * U * (gg.abs() + c1.abs() + 2 * (xh * c2).abs()))
        _check(g.d_x, want, tol + _half(x.dtype, want.abs() + tol), "d_x")
    depth = rows / 64 + 64
    for got, terms, old in ((g.d_weight, dd * xh, old_w), (g.d_bias, dd, old_b)):
        if got is None:
            continue
        want = terms.sum(0) + (old.double() if old is not None else 0.0)
        tol = (depth + 5) * U * terms.abs().sum(0) + U * want.abs()
        _check(got, want, tol + _half(got.dtype, want.abs() + tol), "columns")


SHAPES = [  # rows, columns, stride, shift: registers, vectors with and without tails, wide
    (1, 1, 1, 0), (3, 768, 768, 0), (5, 7, 9, 1), (700, 64, 64, 0), (300, 1000, 1000, 0),
    (257, 2049, 2056, 0), (33, 4096, 4096, 0), (19, 5003, 5056, 0), (2, 8192, 8192, 0),
    (7, 8200, 8200, 0), (5, 16384, 16384, 0), (3, 20001, 20008, 0), (9, 5003, 5003, 0),
    (4, 9001, 9001, 0), (2000, 129, 136, 0), (65, 31, 31, 0)]


@pytest.mark.parametrize("rows,cols,stride,shift", SHAPES)
@pytest.mark.parametrize("dt,w_dt", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"),
                                     ("f16", "f32"), ("f32", "f32")])
def test_forward_and_backward(rows, cols, stride, shift, dt, w_dt):
    g = _gen(rows * 7 + cols)
    rand = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    _, x = _matrix(rand(rows, cols) * torch.exp(0.5 * rand(cols)) + 3 * rand(rows, 1), DT[dt],
                   stride, shift)
    _, d = _matrix(rand(rows, cols), DT[dt], stride, shift)
    w, b = (1 + 0.3 * rand(cols)).to(DT[w_dt]), rand(cols).to(DT[w_dt])
    out_buf, out = _matrix(torch.zeros(rows, cols, device=DEV), DT[dt], stride, shift, fill=7.0)
    y = ss.layer_norm(x, w, b, eps=1e-5, out=out)
    _forward(x, w, b, 1e-5, y)
    assert y.out is out and _untouched(out_buf, out, 7.0)
    dx_buf, d_x = _matrix(torch.zeros(rows, cols, device=DEV), DT[dt], stride, shift, fill=7.0)
    dw, db = torch.full_like(w, 5.0), torch.full_like(b, 5.0)
    got = ss.layer_norm_grad(d, x, y.mean, y.rstd, w, d_x=d_x, d_weight=dw, d_bias=db)
    _backward(d, x, y.mean, y.rstd, w, got)
    assert _untouched(dx_buf, d_x, 7.0)
    old_w, old_b = dw.clone(), db.clone()
    got = ss.layer_norm_grad(d, x, y.mean, y.rstd, w, d_weight=dw, d_bias=db, accumulate=True)
    assert got.d_x is None
    _backward(d, x, y.mean, y.rstd, w, got, old_w, old_b)


@pytest.mark.parametrize("rows,cols,out_stride,out_shift", [
    (37, 5003, 5003, 0), (19, 768, 769, 1), (1, 4097, 4097, 0), (70, 31, 31, 3), (5, 8191, 8191, 0),
    (3, 5, 5, 1), (1500, 2056, 2056, 0), (1300, 3001, 3001, 0), (1700, 4099, 4104, 0),
    (2, 8192, 8200, 0), (1, 3, 8, 0), (6, 8, 9, 0)])
@pytest.mark.parametrize("dt,w_dt", [("bf16", "f32"), ("f16", "f16"), ("f32", "f32")])
def test_results_in_other_rows_than_the_inputs(rows, cols, out_stride, out_shift, dt, w_dt):
    """Aligned inputs, results anywhere; many long rows; nothing past the last row's end."""
    g = _gen(rows + cols)
    rand = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    wide = (cols + 15) // 8 * 8

    def aligned(v):                             # the last row ends where its buffer does
        buf = torch.full(((rows - 1) * wide + cols,), float("nan"), dtype=DT[dt], device=DEV)
        view = torch.as_strided(buf, (rows, cols), (wide, 1))
        view.copy_(v)
        return view
    x, d = aligned(rand(rows, cols) + 2 * rand(rows, 1)), aligned(rand(rows, cols))
    w, b = (1 + 0.3 * rand(cols)).to(DT[w_dt]), rand(cols).to(DT[w_dt])
    empty = torch.zeros(rows, cols, device=DEV)
    out_buf, out = _matrix(empty, DT[dt], out_stride, out_shift, fill=7.0)
    y = ss.layer_norm(x, w, b, out=out)
    _forward(x, w, b, 1e-5, y)
    assert _untouched(out_buf, out, 7.0)
    dx_buf, d_x = _matrix(empty, DT[dt], out_stride, out_shift, fill=7.0)
    got = ss.layer_norm_grad(d, x, y.mean, y.rstd, w, d_x=d_x, d_weight=torch.empty_like(w),
                             d_bias=torch.empty_like(b))
    _backward(d, x, y.mean, y.rstd, w, got)
    assert _untouched(dx_buf, d_x, 7.0)
    _forward(x, None, None, 1e-5, ss.layer_norm(x, out=out))
    _backward(d, x, y.mean, y.rstd, None, ss.layer_norm_grad(d, x, y.mean, y.rstd, d_x=d_x))


@pytest.mark.parametrize("rows,cols,stride,shift", [
    # groups of 64, 96, 160, 192, 320, .. threads; rows that end behind the last whole vector a
    # group holds; single elements in groups of 96, 192, 320
    (300, 1600, 1600, 0), (41, 2560, 2560, 0), (23, 5120, 5128, 0), (700, 1090, 1096, 0),
    (9, 16391, 16392, 0), (5, 16387, 16392, 0), (6, 8199, 8200, 0), (7, 8195, 8200, 0),
    (400, 1027, 1032, 0), (130, 1300, 1301, 0), (50, 2500, 2501, 1), (50, 3900, 3901, 0),
    (40, 6200, 6200, 1), (3, 8193, 8193, 0)])
@pytest.mark.parametrize("dt,w_dt", [("bf16", "f32"), ("f16", "f16"), ("f32", "f32")])
def test_groups_of_any_number_of_warps(rows, cols, stride, shift, dt, w_dt):
    test_forward_and_backward(rows, cols, stride, shift, dt, w_dt)
    test_results_in_other_rows_than_the_inputs(rows, cols, cols + 1, 1, dt, w_dt)


@pytest.mark.parametrize("cols", [96, 5003, 20000])
def test_parts_left_out(cols):
    g = _gen(cols)
    x = torch.randn(11, cols, generator=g, device=DEV)
    d = torch.randn(11, cols, generator=g, device=DEV)
    y = ss.layer_norm(x)
    _forward(x, None, None, 1e-5, y)
    _backward(d, x, y.mean, y.rstd, None, ss.layer_norm_grad(d, x, y.mean, y.rstd))
    w = torch.rand(cols, generator=g, device=DEV)
    _forward(x, w, None, 0.5, ss.layer_norm(x, w, eps=0.5))
    _forward(x, None, w, 1e-5, ss.layer_norm(x, None, w))
    only = ss.layer_norm_grad(d, x, y.mean, y.rstd, w, d_bias=torch.empty_like(w))
    assert only.d_x is None and only.d_weight is None
    _backward(d, x, y.mean, y.rstd, w, only)
    only = ss.layer_norm_grad(d, x, y.mean, y.rstd, w, d_weight=torch.empty_like(w),
                              d_x=torch.empty_like(x))
    _backward(d, x, y.mean, y.rstd, w, only)


def test_three_dimensions_and_no_rows():
    x = torch.randn(3, 5, 64, device=DEV)
    y = ss.layer_norm(x)
    assert y.out.shape == x.shape and y.mean.shape == (15,)
    _forward(x.view(15, 64), None, None, 1e-5, y._replace(out=y.out.view(15, 64)))
    none = x[:0]
    y = ss.layer_norm(none)
    assert y.out.shape == (0, 5, 64) and y.mean.numel() == 0
    dw, db = torch.full((64,), 3.0, device=DEV), torch.full((64,), 3.0, device=DEV)
    ss.layer_norm_grad(none, none, y.mean, y.rstd, d_weight=dw, d_bias=db, accumulate=True)
    assert bool((dw == 3.0).all())
    ss.layer_norm_grad(none, none, y.mean, y.rstd, d_weight=dw, d_bias=db)
    assert not dw.any() and not db.any()


def test_constant_rows_far_from_zero_and_not_finite_ones():
    x = torch.full((4, 1000), 1000.0, device=DEV)
    x[1] += torch.arange(1000, device=DEV) % 2 * 0.125      # variance 2^-8, mean 1000.0625: exact
    x[2, 17] = float("nan")
    x[3, 999] = float("inf")
    y = ss.layer_norm(x, eps=1e-5)
    assert not y.out[0].any() and abs(float(y.rstd[0]) - 1e-5 ** -0.5) < 1e-3
    assert abs(float(y.rstd[1]) - (2.0 ** -8 + 1e-5) ** -0.5) < 1e-4
    assert bool(torch.isnan(y.out[2:]).all())
    d = torch.ones_like(x)
    dw, db = torch.empty(1000, device=DEV), torch.empty(1000, device=DEV)
    g = ss.layer_norm_grad(d, x, y.mean, y.rstd, d_x=torch.empty_like(x), d_weight=dw, d_bias=db)
    assert bool(torch.isfinite(g.d_x[:2]).all()) and bool((db == 4.0).all())


def test_gradient_matches_differences():
    # of sum(out * d) in double, from the formula's own derivative at h = 1e-4
    g = _gen(3)
    x = torch.randn(4, 24, generator=g, device=DEV)
    d = torch.randn(4, 24, generator=g, device=DEV)
    w, b = torch.rand(24, generator=g, device=DEV) + 0.5, torch.randn(24, generator=g, device=DEV)
    y = ss.layer_norm(x, w, b)
    got = ss.layer_norm_grad(d, x, y.mean, y.rstd, w, d_x=torch.empty_like(x),
                             d_weight=torch.empty_like(w), d_bias=torch.empty_like(b))

    def loss(x, w, b):
        xc = x - x.mean(1, keepdim=True)
        return float(((xc * (xc.square().mean(1, keepdim=True) + 1e-5) ** -0.5 * w + b)
                      * d.double()).sum())
    args = [t.double() for t in (x, w, b)]
    for k, grad in enumerate((got.d_x, got.d_weight, got.d_bias)):
        for at in ((0,), (5,), (23,)) if k else ((0, 0), (3, 7)):
            ends = []
            for h in (1e-4, -1e-4):
                moved = [t.clone() for t in args]
                moved[k][at] += h
                ends.append(loss(*moved))
            # the third derivative's share is below 1e-6, the gradient's rounding 1e-6
            assert abs((ends[0] - ends[1]) / 2e-4 - float(grad[at])) < 1e-5


def test_repeats_streams_and_graphs():
    g = _gen(8)
    x = torch.randn(3000, 768, generator=g, device=DEV).bfloat16()
    d = torch.randn(3000, 768, generator=g, device=DEV).bfloat16()
    w, b = torch.rand(768, generator=g, device=DEV), torch.rand(768, generator=g, device=DEV)

    def both(ws, stream=None, bufs=None):
        out, d_x, dw, db = bufs or [torch.empty_like(t) for t in (x, x, w, b)]
        y = ss.layer_norm(x, w, b, out=out, stream=stream)
        ss.layer_norm_grad(d, x, y.mean, y.rstd, w, d_x=d_x, d_weight=dw, d_bias=db,
                           workspace=ws, stream=stream)
        return out, d_x, dw, db
    ws = ss.LayerNormWorkspace(DEV)
    want = both(ws)
    ws.buf.fill_(255)
    assert all(torch.equal(p, q) for p, q in zip(both(ws), want))
    s = torch.cuda.Stream()
    bufs = [torch.empty_like(t) for t in (x, x, w, b)]
    s.wait_stream(torch.cuda.current_stream())
    got = both(None, stream=s, bufs=bufs)
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both(ws)
    for t in got:
        t.zero_()
    graph.replay()
    assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_offsets_past_32_bits():
    rows, cols = 600_000, 4096
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device=DEV)
    x[-1, ::2], x[-1, 1::2] = 2.0, -2.0
    y = ss.layer_norm(x, eps=0.0 + 1e-5)
    assert bool((y.out[-1, ::2] == 1.0).all()) and bool((y.out[-1, 1::2] == -1.0).all())
    assert not y.out[-2].any()
    dw = torch.empty(cols, dtype=torch.float32, device=DEV)
    ss.layer_norm_grad(y.out, x, y.mean, y.rstd, d_weight=dw)
    assert bool(((dw - 1.0).abs() < 1e-5).all())
