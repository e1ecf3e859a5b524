"""The token embedding and its gradient on the GPU against plain 64-bit sums.

The lookup is one fp32 product and one rounding: the bits of torch's.  A row of
the gradient is a sum of k terms in fp32, k - 1 additions, then the product with
the scale and, accumulating, one more addition: an element is off by at most
(k + 1) 2^-24 scale sum |d| + 2^-24 |old + sum|, and half a step of its type."""
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


def _band(rows, cols, dtype, stride=None, shift=0, fill=float("nan")):
    """A matrix inside a band of `fill`, its rows `stride` apart, `shift` elements in."""
    stride = stride or cols
    buf = torch.full(((rows + 2) * stride + shift + 64,), fill, dtype=dtype, device=DEV)
    view = buf[stride + shift:stride + shift + rows * stride]
    return buf, view.view(rows, stride)[:, :cols]


def _outside(buf, view):
    """What of a band lies outside its matrix."""
    held = torch.zeros(buf.shape, dtype=torch.bool, device=DEV)
    torch.as_strided(held, view.shape, view.stride(), view.storage_offset())[:] = True
    return buf[~held]


SHAPES = [(1, 1, 1, 1, 0), (3, 768, 100, 768, 0), (5, 7, 3, 9, 1), (129, 64, 50, 72, 0),
          (1000, 2056, 40, 2056, 0), (33, 4097, 300, 4104, 0), (64, 24, 5000, 24, 3)]


@pytest.mark.parametrize("n,dim,vocab,stride,shift", SHAPES)
@pytest.mark.parametrize("dt", DT)
def test_lookup(n, dim, vocab, stride, shift, dt):
    g = _gen(n + dim)
    _, table = _band(vocab, dim, DT[dt], stride, shift)
    table.copy_(torch.randn(vocab, dim, generator=g, device=DEV))
    table[0, 0] = float("inf")
    ids = torch.randint(-2, vocab + 2, (n,), generator=g, device=DEV)
    buf, out = _band(n, dim, DT[dt], stride, shift, fill=7.0)
    for kind in (torch.int64, torch.int32):
        out.fill_(3.0)
        got = ss.embedding(table, ids.to(kind), scale=0.7, out=out)
        assert got is out
        live = (ids >= 0) & (ids < vocab)
        rows = table[ids.clamp(0, vocab - 1)].float() * 0.7
        want = torch.where(live[:, None], rows, 0.0).to(DT[dt])
        assert torch.equal(out.nan_to_num(9.0), want.nan_to_num(9.0))
        assert bool((_outside(buf, out) == 7.0).all())


def test_lookup_shapes_and_empty():
    table = torch.randn(11, 8, device=DEV)
    ids = torch.tensor([[1, 2, 3], [10, 0, -1]], device=DEV)
    out = ss.embedding(table, ids)
    assert out.shape == (2, 3, 8) and torch.equal(out[0], table[1:4])
    assert not out[1, 2].any()
    assert ss.embedding(table, ids[:0]).shape == (0, 3, 8)


def _want(d, ids, vocab, scale, old):
    live = (ids >= 0) & (ids < vocab)
    at = torch.where(live, ids, vocab)
    total = torch.zeros(vocab + 1, d.shape[1], dtype=torch.float64, device=DEV)
    size, count = torch.zeros_like(total), torch.zeros(vocab + 1, device=DEV)
    value = torch.where(live[:, None], d.double(), 0.0)
    total.index_add_(0, at, value)
    size.index_add_(0, at, value.abs())
    count.index_add_(0, at, torch.ones_like(at, dtype=torch.float32))
    return scale * total[:vocab] + old, abs(scale) * size[:vocab], count[:vocab, None]


GRADS = [  # tokens, columns, vocabulary, ids
    (1, 8, 1, "uniform"), (1, 5, 40, "uniform"), (7, 16, 3, "uniform"), (8, 768, 50, "one"),
    (9, 768, 50, "one"), (500, 64, 5000, "uniform"), (2500, 136, 700, "skewed"),
    (4096, 768, 1000, "skewed"), (3001, 2056, 90, "skewed"), (1000, 4099, 33, "uniform"),
    (30000, 24, 400_000, "skewed"), (70001, 8, 17, "one"), (300, 32, 200, "none")]


def _tokens(kind, n, vocab, g):
    if kind == "one":
        return torch.full((n,), vocab - 1, device=DEV)
    if kind == "none":
        return torch.full((n,), -1, device=DEV)
    u = torch.rand(n, generator=g, device=DEV)
    ids = ((u ** 4 if kind == "skewed" else u) * vocab).long().clamp(0, vocab - 1)
    ids[torch.rand(n, generator=g, device=DEV) < 0.1] = -1 if n % 2 else vocab
    return ids


@pytest.mark.parametrize("n,dim,vocab,kind", GRADS)
@pytest.mark.parametrize("dt,grad_dt", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"),
                                        ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("accumulate", [False, True])
def test_gradient(n, dim, vocab, kind, dt, grad_dt, accumulate):
    g = _gen(n + dim)
    ids = _tokens(kind, n, vocab, g)
    stride, shift = (dim, 0) if n % 2 == 0 else (dim + 8, 0) if dim % 8 == 0 else (dim + 3, 1)
    _, d = _band(n, dim, DT[dt], stride, shift)
    d.copy_(torch.randn(n, dim, generator=g, device=DEV))
    d[(ids < 0) | (ids >= vocab)] = float("nan")               # not read
    buf, grad = _band(vocab, dim, DT[grad_dt], stride, shift, fill=7.0)
    if accumulate:
        grad.copy_(torch.randn(vocab, dim, generator=g, device=DEV))
    before = grad.clone()
    old = grad.double() if accumulate else torch.zeros(vocab, dim, dtype=torch.float64, device=DEV)
    want, size, count = _want(torch.where(torch.isnan(d), 0.0, d), ids, vocab, 0.37, old)
    assert ss.embedding_grad(d, ids.to(torch.int32 if n % 3 == 0 else torch.int64), grad,
                             scale=0.37, accumulate=accumulate) is grad
    # the scale itself is 0.37 to within 2^-24
    tol = (count + 2) * U * size + U * want.abs() + torch.finfo(DT[grad_dt]).eps / 2 * (
        want.abs() + (count + 3) * U * size)
    bad = ~((grad.double() - want).abs() <= tol * (1 + 1e-9) + 1e-300)
    if grad_dt == "f16":                                       # subnormals: half of 2^-24
        bad &= (grad.double() - want).abs() > tol + 2.0 ** -25
    assert not bad.any(), torch.nonzero(bad)[:4]
    absent = (count == 0).expand_as(grad)
    assert torch.equal(grad[absent], before[absent] if accumulate else torch.zeros_like(grad[absent]))
    assert bool((_outside(buf, grad) == 7.0).all())


@pytest.mark.parametrize("n,dim,vocab,kind", [
    (40, 2047, 300, "uniform"), (41, 1031, 90, "uniform"), (2, 1025, 40, "none"),
    (3, 1026, 60, "uniform"), (12, 1028, 50, "one"), (7, 1036, 64, "skewed")])
@pytest.mark.parametrize("dt,grad_dt", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
def test_absent_rows_that_start_anywhere(n, dim, vocab, kind, dt, grad_dt):
    """Zeros by vectors within rows of more than 1024 columns at any alignment."""
    test_gradient(n, dim, vocab, kind, dt, grad_dt, False)


def test_gradient_repeats_to_the_bit_and_needs_no_clean_workspace():
    g = _gen(5)
    n, dim, vocab = 5000, 520, 300
    ids = _tokens("skewed", n, vocab, g)
    d = torch.randn(n, dim, generator=g, device=DEV)
    ws, grads = ss.EmbeddingWorkspace(DEV), []
    for k in range(4):
        grads.append(ss.embedding_grad(d, ids, torch.full((vocab, dim), float(k), device=DEV),
                                       workspace=ws))
        ws.buf.fill_(255 - k)
    assert all(torch.equal(x, grads[0]) for x in grads[1:])


def test_gradient_of_many_ids_and_none():
    # more ids than the sorting blocks' ranges times the SMs, few of them used
    vocab = 700_001
    ids = torch.tensor([0, vocab - 1, 350_000, vocab - 1, 2047, 2048, 350_000], device=DEV)
    d = torch.arange(7 * 4, device=DEV).float().view(7, 4)
    grad = torch.ones(vocab, 4, device=DEV)
    ss.embedding_grad(d, ids, grad)
    want = torch.zeros(vocab, 4, device=DEV)
    want.index_add_(0, ids, d)                                 # small whole numbers: exact
    assert torch.equal(grad, want)
    grad.fill_(2.0)
    ss.embedding_grad(d[:0], ids[:0], grad, accumulate=True)
    assert bool((grad == 2.0).all())
    ss.embedding_grad(d[:0], ids[:0], grad)
    assert not grad.any()


def test_offsets_past_32_bits():
    # rows of the table, of the output and of the gradient beyond 2^32 bytes
    vocab, dim = 600_000, 4096
    table = torch.zeros(vocab, dim, dtype=torch.bfloat16, device=DEV)
    ids = torch.tensor([vocab - 1, 5, vocab - 2, vocab - 1], device=DEV)
    table[vocab - 1], table[vocab - 2] = 3.0, 5.0
    out = ss.embedding(table, ids, scale=2.0)
    assert [float(r[0]) for r in out] == [6.0, 0.0, 10.0, 6.0] and bool((out[3] == 6.0).all())
    ss.embedding_grad(out, ids, table)
    assert float(table[vocab - 1, dim - 1]) == 12.0 and float(table[vocab - 2, 0]) == 10.0
    assert float(table.double().sum()) == dim * 22.0


def test_gradient_matches_differences():
    # <d, embedding(table + h e)> - <d, embedding(table - h e)> over 2 h, exact in powers of two
    table = torch.randint(-8, 8, (9, 8), device=DEV).float()
    ids = torch.tensor([3, 3, 0, 8, -1, 3], device=DEV)
    d = torch.randint(-8, 8, (6, 8), device=DEV).float()
    grad = ss.embedding_grad(d, ids, torch.empty_like(table), scale=0.5)
    for v, c in ((3, 0), (0, 7), (8, 2), (5, 1)):
        diff = []
        for h in (0.5, -0.5):
            moved = table.clone()
            moved[v, c] += h
            diff.append(float((ss.embedding(moved, ids, scale=0.5) * d).sum()))
        assert diff[0] - diff[1] == float(grad[v, c])


@pytest.mark.parametrize("own_stream", [False, True])
def test_graph_and_stream(own_stream):
    g = _gen(9)
    table = torch.randn(300, 768, generator=g, device=DEV).bfloat16()
    ids = torch.randint(0, 300, (2000,), generator=g, device=DEV)
    d = torch.randn(2000, 768, generator=g, device=DEV).bfloat16()
    want_out = ss.embedding(table, ids, scale=3.0)
    want = ss.embedding_grad(d, ids, torch.zeros(300, 768, device=DEV), accumulate=True)
    if own_stream:
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        grad = torch.zeros(300, 768, device=DEV)
        s.wait_stream(torch.cuda.current_stream())
        out = ss.embedding(table, ids, scale=3.0, stream=s)
        ss.embedding_grad(d, ids, grad, accumulate=True, stream=s)
        s.synchronize()
        assert torch.equal(out, want_out) and torch.equal(grad, want)
        return
    ws, grad, out = ss.EmbeddingWorkspace(DEV), torch.zeros(300, 768, device=DEV), want_out * 0
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ss.embedding(table, ids, scale=3.0, out=out)
        ss.embedding_grad(d, ids, grad, accumulate=True, workspace=ws)
    # a larger call afterwards takes another buffer; the graph's stays
    ss.embedding_grad(d.repeat(20, 1), ids.repeat(20), torch.empty(300, 768, device=DEV),
                      workspace=ws)
    graph.replay()
    assert torch.equal(out, want_out) and torch.equal(grad, want)
    graph.replay()
    assert not torch.equal(grad, want)                          # added once more
