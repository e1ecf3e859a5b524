"""The policy and preference losses on the GPU against the 64-bit oracle.

Tolerances, derived from the arithmetic: with d = x_y - max x and
a = d - log S, both differences and log S round to 2^-24 of their size, and
the sum S of V exponentials carries at most V / 128 + 64 roundings along any
path of its tree, each exponential 2^-21 (the exponent's rounding and the
base-2 exponential); so |error of a| <= T = 2^-23 (|d| + |a| + 1) +
(V / 128 + 64) 2^-24 + 2^-21.  The slope moves by its sensitivity to a times
T, p by p T, and the gradient is rounded once to its type."""
import numpy as np
import pytest
import torch

import sharded_optimizer_step_gb300 as ss
from oracle import token_loss as OL

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = {"bf16": 2.0 ** -8, "f16": 2.0 ** -10, "f32": 2.0 ** -23}
SUB = {"bf16": 2.0 ** -133, "f16": 2.0 ** -24, "f32": 2.0 ** -140}


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ss.build()
    yield
    assert ss.device_status() == 0


def _inputs(n, v, dt, seed=0, stride=None, shift=0, masked=0.0, spread=2.0):
    """Logits in a poisoned buffer: NaN before, between and after the rows."""
    r = np.random.default_rng(seed)
    stride = stride or v
    buf = torch.full((shift + n * stride + 64,), float("nan"), dtype=DT[dt], device=DEV)
    x = buf[shift:shift + n * stride].view(n, stride)[:, :v]
    x.copy_(torch.from_numpy(r.normal(size=(n, v)) * spread).to(DT[dt]))
    ids = r.integers(0, v, n)
    host = x.double().cpu().numpy()
    host[np.arange(n), ids] += 3.0
    x.copy_(torch.from_numpy(host).to(DT[dt]))
    host = x.double().cpu().numpy()
    lp = OL.log_softmax(host)[np.arange(n), ids]
    old = lp + r.normal(size=n) * 0.3
    for edge in (0.8, 1.2):
        old = np.where(np.abs(np.exp(lp - old) - edge) < 1e-3, old + 5e-3, old)
    w = np.where(r.random(n) < masked, 0.0, r.choice([1.0, 0.5, 2.0], n))
    f = lambda a: np.asarray(a, np.float32)  # noqa: E731
    return dict(buf=buf, x=x, host=host, ids=ids, old=f(old), adv=f(r.normal(size=n)),
                ref=f(lp + r.normal(size=n) * 0.2), w=f(w))


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def _lp_tol(host, ids, logps, v):
    d = np.abs(host[np.arange(len(ids)), ids] - host.max(axis=1))
    return 2.0 ** -23 * (d + np.abs(logps) + 1) + (v / 128 + 64) * 2.0 ** -24 + 2.0 ** -21


def _grad_buffer(n, v, dt, stride=None, shift=0):
    stride = stride or v
    buf = torch.full((shift + n * stride + 64,), 7.0, dtype=DT[dt], device=DEV)
    return buf, buf[shift:shift + n * stride].view(n, stride)[:, :v]


def _check_grad(got, want, sens, tol, dt):
    got = got.double().cpu().numpy()
    bound = EPS[dt] * np.abs(want) + (4 * sens * (tol + 2.0 ** -21))[:, None] + SUB[dt]
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], want[bad][:4])


def _check_untouched(buf, n, v, stride, shift):
    keep = torch.ones(buf.numel(), dtype=torch.bool, device=DEV)
    keep[shift:shift + n * stride].view(n, stride)[:, :v] = False
    assert (buf[keep] == 7.0).all()


def _run_policy(c, dt, kl=0.05, ids_dtype=np.int64, weights=True, grad=None, **kw):
    return ss.policy_loss(c["x"], _dev(c["ids"].astype(ids_dtype)), _dev(c["old"]),
                          _dev(c["adv"]), ref_logps=_dev(c["ref"]) if kl else None, kl_coef=kl,
                          weights=_dev(c["w"]) if weights else None, grad=grad, **kw)


def _check_policy(c, out, dt, kl, weights=True, norm=None, scale=1.0, rows=None):
    n, v = c["host"].shape
    w = c["w"].astype(np.float64) if weights else np.ones(n)
    stats, logps, grad = OL.policy(c["host"], c["ids"], c["old"], c["adv"], ref=c["ref"],
                                   weights=w, kl=kl, norm=norm)
    tol = _lp_tol(c["host"], c["ids"], logps, v)
    live = w != 0
    got = out.logps.double().cpu().numpy()
    assert (np.abs(got - logps)[live] <= tol[live]).all()
    assert (got[~live] == 0).all()
    total = w.sum() if norm is None else norm
    k = np.abs(w) / total if live.any() else w
    u = np.exp(np.where(live, logps, 0) - c["old"])
    sens = k * (np.abs(u * c["adv"]) + kl * (np.exp(c["ref"] - np.where(live, logps, 0)) + 1))
    bound = 4 * (sens * (tol + 2.0 ** -21))[live].sum() + 2.0 ** -21 * np.abs(stats).max()
    # each term of the statistics: the policy term, kl (relative to 1 / kl_coef), the count
    got = out.stats.double().cpu().numpy()
    assert abs(got[0] - stats[0]) <= bound and abs(got[1] - stats[1]) <= bound
    assert abs(got[2] - stats[2]) <= (bound / kl if kl else 0.0)
    assert abs(got[3] - stats[3]) <= 1e-6
    if out.grad is not None:
        _check_grad(out.grad, grad * scale, sens * scale, tol, dt)
    return stats


SHAPES = [(1, 1), (3, 2), (2, 7), (5, 8), (1, 9), (4, 31), (7, 257), (3, 1000), (33, 4099),
          (400, 515), (2, 32000), (5, 50257)]


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("n,v", SHAPES)
def test_policy_forward_and_backward(n, v, dt):
    c = _inputs(n, v, dt, seed=n * v, masked=0.3 if n > 3 else 0.0)
    buf, g = _grad_buffer(n, v, dt)
    out = _run_policy(c, dt, grad=g)
    _check_policy(c, out, dt, 0.05)
    _check_untouched(buf, n, v, v, 0)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("stride,shift,gstride,gshift", [
    (1013, 0, 1013, 0), (1024, 0, 1001, 0), (1000, 1, 1000, 1), (1000, 3, 1000, 0),
    (1007, 5, 1013, 2), (1000, 8, 1000, 8), (1002, 0, 1002, 4)])
def test_policy_any_stride_and_alignment(stride, shift, gstride, gshift, dt):
    n, v = 9, 1000
    c = _inputs(n, v, dt, seed=stride + shift, stride=stride, shift=shift, masked=0.2)
    buf, g = _grad_buffer(n, v, dt, gstride, gshift)
    _check_policy(c, _run_policy(c, dt, kl=0.0, grad=g), dt, 0.0)
    _check_untouched(buf, n, v, gstride, gshift)


@pytest.mark.parametrize("v,dt", [(120001, "bf16"), (120001, "f32"), (300007, "f16")])
def test_policy_wide_vocabularies(v, dt):
    c = _inputs(3, v, dt, seed=9)
    _, g = _grad_buffer(3, v, dt)
    _check_policy(c, _run_policy(c, dt, grad=g), dt, 0.05)


@pytest.mark.parametrize("v,dt", [(50257, "f32"), (50257, "bf16"), (32000, "f32")])
def test_many_wide_rows_per_block(v, dt):
    """Several rows per block at widths where one or two rows fill the block's
    shared memory, so that a slot is used again by another team's row."""
    n = 640
    c = _inputs(n, v, dt, seed=v, stride=v + 47, masked=0.2)
    _, g = _grad_buffer(n, v, dt, v + 47)
    _check_policy(c, _run_policy(c, dt, grad=g), dt, 0.05)
    lens = [200, 100, 160, 180]
    _check_pref(c, lens, _run_pref(c, lens, g), dt)


@pytest.mark.parametrize("v,dt,shift", [(128256, "bf16", 0), (60001, "f32", 0),
                                        (128256, "f16", 1), (230001, "bf16", 0)])
def test_many_rows_longer_than_shared_memory(v, dt, shift):
    """Rows that do not fit an SM's shared memory, several per block: the losses
    take a forward and a backward pass, whose teams skip rows of more chunks than
    there are slots.  Also with the gradient at another offset than the logits."""
    n = 400
    c = _inputs(n, v, dt, seed=v, masked=0.15)
    _, g = _grad_buffer(n, v, dt, v, shift)
    _check_policy(c, _run_policy(c, dt, grad=g), dt, 0.05)
    lens = [100, 50, 60, 190]
    _check_pref(c, lens, _run_pref(c, lens, g), dt)


@pytest.mark.parametrize("shift", [0, 1])
def test_more_rows_than_one_launch_takes(shift):
    """Above 1024 rows per SM a call goes in several launches, which carry the sums
    on; a sequence may begin in one launch and end in another."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    n, v, dt = 1024 * sms + 4321, 37, "bf16"
    c = _inputs(n, v, dt, seed=21, masked=0.3)
    buf, g = _grad_buffer(n, v, dt, v, shift)
    _check_policy(c, _run_policy(c, dt, grad=g), dt, 0.05)
    _check_untouched(buf, n, v, v, shift)
    _check_policy(c, _run_policy(c, dt), dt, 0.05)
    lens = [70_000, 20_000, 50_001, n - 140_001]
    _check_pref(c, lens, _run_pref(c, lens, g), dt)
    _check_untouched(buf, n, v, v, shift)


def test_policy_forms():
    """int32 ids, no weights, a given norm, scales, forward only, in place."""
    n, v, dt = 12, 777, "bf16"
    c = _inputs(n, v, dt, seed=4, masked=0.25)
    _, g = _grad_buffer(n, v, dt)
    _check_policy(c, _run_policy(c, dt, ids_dtype=np.int32, grad=g), dt, 0.05)
    _check_policy(c, _run_policy(c, dt, weights=False, grad=g), dt, 0.05, weights=False)
    scale = torch.tensor([64.0], device=DEV)
    _check_policy(c, _run_policy(c, dt, norm=40.0, grad=g, grad_scale=0.25, loss_scale=scale), dt,
                  0.05, norm=40.0, scale=16.0)
    fwd = _run_policy(c, dt)
    assert fwd.grad is None
    _check_policy(c, fwd, dt, 0.05)
    both = _run_policy(c, dt, grad=g)
    _check_policy(c, both, dt, 0.05)
    again = _run_policy(c, dt, grad=c["x"])
    assert torch.equal(again.grad, g) and torch.equal(again.logps, both.logps)
    assert torch.equal(again.stats, both.stats)


@pytest.mark.parametrize("n", [1, 7, 700])
def test_policy_all_tokens_masked(n):
    c = _inputs(n, 300, "bf16", seed=1)
    c["w"][:] = 0
    c["x"].fill_(float("nan"))
    c["ids"][:] = 1 << 40
    _, g = _grad_buffer(n, 300, "bf16")
    out = _run_policy(c, "bf16", grad=g)
    assert not out.stats.any() and not out.logps.any() and not out.grad.any()


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_special_logits(dt):
    """-inf and the type's lowest value in masked places, rows of one value,
    large values, ids outside the vocabulary, NaN rows: a row that should be
    finite is right, one that should not is NaN and leaves the others alone."""
    n, v = 8, 515
    c = _inputs(n, v, dt, seed=2)
    low = torch.finfo(DT[dt]).min
    x = c["x"]
    keep = torch.arange(v, device=DEV) % 3 == 0
    c["ids"] = c["ids"] // 3 * 3
    x[0, ~keep] = float("-inf")
    x[1, ~keep] = low
    x[2] = low                       # a row of the lowest value: uniform
    x[3] = torch.finfo(DT[dt]).max   # and of the largest
    x[4] = 0.0
    x[4, c["ids"][4]] = torch.finfo(DT[dt]).max
    x[5, :] = float("-inf")
    x[5, c["ids"][5]] = 1.5          # a certain token
    c["host"] = x.double().cpu().numpy()
    lp = OL.log_softmax(c["host"])[np.arange(n), c["ids"]]
    c["old"] = (lp + 0.05).astype(np.float32)
    c["ref"] = (lp - 0.1).astype(np.float32)
    _, g = _grad_buffer(n, v, dt)
    _check_policy(c, _run_policy(c, dt, grad=g), dt, 0.05)
    assert g[0, ~keep].abs().max() == 0 and g[1, ~keep].abs().max() == 0
    # rows that cannot be finite
    x[6, 7] = float("nan")
    x[7] = float("-inf")
    ids = _dev(c["ids"])
    ids[0] = v
    ids[1] = -1
    good = g.clone()
    w = torch.ones(n, device=DEV)
    out = ss.policy_loss(x, ids, _dev(c["old"]), _dev(c["adv"]), weights=w, norm=float(n),
                         ref_logps=_dev(c["ref"]), kl_coef=0.05, grad=g)
    bad = torch.tensor([1, 1, 0, 0, 0, 0, 1, 1], dtype=torch.bool, device=DEV)
    assert torch.equal(torch.isnan(out.logps), bad)
    assert torch.isnan(out.stats[0])
    assert torch.isnan(g[bad]).all() and not torch.isnan(g[~bad]).any()
    # the rows left alone: the same up to the divisor (sum of w against n)
    k = float(n / c["w"].sum())
    for i in range(2, 6):
        want = good[i].double() / (float(c["w"][i]) * k)
        assert (g[i].double() - want).abs().max() <= 4 * EPS[dt] * want.abs().max() + SUB[dt]


def test_policy_is_deterministic_and_streams():
    c = _inputs(700, 4099, "bf16", seed=6, masked=0.2)
    _, g1 = _grad_buffer(700, 4099, "bf16")
    _, g2 = _grad_buffer(700, 4099, "bf16")
    a = _run_policy(c, "bf16", grad=g1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ws = ss.LossWorkspace(DEV)
    with torch.cuda.stream(s):
        b = _run_policy(c, "bf16", grad=g2, workspace=ws)
        first = b.stats.clone(), b.logps.clone(), b.grad.clone()
        b = _run_policy(c, "bf16", grad=g2, workspace=ws)    # the workspace is ready again
    s.synchronize()
    for x, y, z in zip((a.stats, a.logps, a.grad), (b.stats, b.logps, b.grad), first):
        assert torch.equal(x, y) and torch.equal(x, z)


def _run_pref(c, lens, grad=None, **kw):
    return ss.preference_loss(c["x"], _dev(c["ids"]), lens, _dev(c["ref"]), weights=_dev(c["w"]),
                              grad=grad, **kw)


def _check_pref(c, lens, out, dt, beta=0.1, smoothing=0.0, norm=None, scale=1.0):
    n, v = c["host"].shape
    stats, ratios, logps, grad = OL.preference(c["host"], c["ids"], lens, c["ref"], beta,
                                               smoothing, c["w"], norm)
    w = np.abs(c["w"].astype(np.float64))
    tol = _lp_tol(c["host"], c["ids"], logps, v)
    live = w != 0
    assert (np.abs(out.logps.double().cpu().numpy() - logps)[live] <= tol[live]).all()
    seq = np.repeat(np.arange(len(lens)), lens)
    rtol = np.bincount(seq, np.where(live, w * (tol + 2.0 ** -22 * np.abs(logps - c["ref"])), 0),
                       len(lens)) + 2.0 ** -23 * np.abs(ratios)
    assert (np.abs(out.log_ratios.double().cpu().numpy() - ratios) <= rtol).all()
    htol = beta * (rtol[0::2] + rtol[1::2]) + 2.0 ** -22
    total = len(lens) // 2 if norm is None else norm
    got = out.stats.double().cpu().numpy()
    assert abs(got[0] - stats[0]) <= htol.sum() / total + 2.0 ** -21 * abs(stats[0])
    assert abs(got[1] - stats[1]) <= htol.sum() / total + 2.0 ** -22 * abs(stats[1])
    assert abs(got[2] - stats[2]) <= 1e-6
    if out.grad is not None:
        sens = beta * w / total * scale
        _check_grad(out.grad, grad * scale, sens, tol + np.repeat(htol, 2)[seq], dt)


LENS = [[1, 1], [3, 5], [0, 4], [2, 0, 1, 7], [40, 33, 1, 2, 0, 0, 17, 90], [130, 260, 64, 31]]


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("v", [5, 515, 4099])
def test_preference_forward_and_backward(lens, v, dt):
    n = sum(lens)
    c = _inputs(n, v, dt, seed=n + v, masked=0.3 if n > 8 else 0.0)
    buf, g = _grad_buffer(n, v, dt)
    _check_pref(c, lens, _run_pref(c, lens, g), dt)
    _check_untouched(buf, n, v, v, 0)


@pytest.mark.parametrize("v,dt", [(32000, "bf16"), (50257, "f32"), (120001, "f32")])
def test_preference_wide_rows(v, dt):
    lens = [2, 3, 4, 1]
    c = _inputs(10, v, dt, seed=v, masked=0.2)
    _, g = _grad_buffer(10, v, dt)
    _check_pref(c, lens, _run_pref(c, lens, g), dt)


@pytest.mark.parametrize("stride,shift,gstride,gshift", [
    (1013, 0, 1013, 0), (1024, 0, 1001, 0), (1000, 1, 1000, 1), (1007, 5, 1013, 2)])
def test_preference_any_stride_and_alignment(stride, shift, gstride, gshift):
    lens, v, dt = [3, 4, 2, 2], 1000, "bf16"
    c = _inputs(11, v, dt, seed=stride, stride=stride, shift=shift, masked=0.2)
    buf, g = _grad_buffer(11, v, dt, gstride, gshift)
    _check_pref(c, lens, _run_pref(c, lens, g), dt)
    _check_untouched(buf, 11, v, gstride, gshift)


def test_preference_forms():
    lens, dt = [20, 31, 7, 9], "bf16"
    c = _inputs(67, 515, dt, seed=3, masked=0.2)
    _, g = _grad_buffer(67, 515, dt)
    scale = torch.tensor([128.0], device=DEV)
    out = _run_pref(c, lens, g, beta=0.5, label_smoothing=0.1, norm=16, grad_scale=0.5,
                    loss_scale=scale)
    _check_pref(c, lens, out, dt, 0.5, 0.1, 16, 64.0)
    fwd = _run_pref(c, lens)
    _check_pref(c, lens, fwd, dt)
    both = _run_pref(c, lens, g)
    assert torch.equal(fwd.stats, both.stats) and torch.equal(fwd.log_ratios, both.log_ratios)
    keep = g.clone()
    again = _run_pref(c, lens, c["x"])
    assert torch.equal(again.grad, keep) and torch.equal(again.log_ratios, both.log_ratios)


@pytest.mark.parametrize("spread,boost", [(1.5, 0.0), (1.5, 5.0), (3.0, 0.0)])
@pytest.mark.parametrize("v,dt", [(32000, "bf16"), (4099, "f32")])
def test_log_ratios_gather_no_common_error(v, dt, spread, boost):
    """Sequences of one token against the exact log probabilities as references:
    each log ratio is the token's own error, at most a few 1e-7 with either sign,
    and their mean stays below 1.5e-8 (a one-sided relative error of 2^-24, 6e-8,
    of the exponentials or of log2 e would show as 2e-8 to 1.2e-7)."""
    n = 4096
    g = torch.Generator(device=DEV).manual_seed(v + int(10 * spread + boost))
    x = (torch.randn(n, v, device=DEV, generator=g) * spread).to(DT[dt])
    ids = torch.randint(0, v, (n,), device=DEV, generator=g)
    rows = torch.arange(n, device=DEV)
    x[rows, ids] = (x[rows, ids].float() + boost).to(DT[dt])
    exact = torch.cat([x[i:i + 512].double().gather(1, ids[i:i + 512, None])[:, 0] -
                       torch.logsumexp(x[i:i + 512].double(), 1) for i in range(0, n, 512)])
    out = ss.preference_loss(x, ids, [1] * n, exact.float())
    error = out.log_ratios.double() + exact.float().double() - exact
    assert error.abs().max() < 2e-6 and abs(float(error.mean())) < 1.5e-8


def test_preference_many_pairs_and_all_masked():
    """More pairs than one launch's table holds; then every token masked."""
    r = np.random.default_rng(8)
    lens = [int(x) for x in r.integers(0, 4, 2 * 1300)]
    n = sum(lens)
    c = _inputs(n, 33, "f32", seed=5, masked=0.2)
    _, g = _grad_buffer(n, 33, "f32")
    _check_pref(c, lens, _run_pref(c, lens, g), "f32")
    c["w"][:] = 0
    c["x"].fill_(float("nan"))
    out = _run_pref(c, lens, g)
    assert abs(float(out.stats[0]) - np.log(2)) < 1e-6 and not out.grad.any()
    assert not out.log_ratios.any() and not out.logps.any()


def test_preference_is_deterministic():
    lens = [100, 120, 80, 90, 200, 150]
    c = _inputs(sum(lens), 4099, "bf16", seed=6, masked=0.2)
    _, g = _grad_buffer(sum(lens), 4099, "bf16")
    ws = ss.LossWorkspace(DEV)
    first = None
    for _ in range(4):
        o = _run_pref(c, lens, g, workspace=ws)
        now = [t.clone() for t in (o.stats, o.log_ratios, o.logps, o.grad)]
        first = first or now
        assert all(torch.equal(a, b) for a, b in zip(first, now))


def test_no_tokens():
    x = torch.empty(0, 100, dtype=torch.bfloat16, device=DEV)
    e, i = torch.empty(0, device=DEV), torch.empty(0, dtype=torch.int64, device=DEV)
    before = ss.launch_count()
    assert not ss.policy_loss(x, i, e, e, grad=x).stats.any()
    assert not ss.preference_loss(x, i, [0, 0], e, grad=x).log_ratios.any()
    assert ss.launch_count() == before


def test_offsets_past_2_31_elements():
    """70000 rows of 32000 (2.2e9 elements), in place; rows at both ends and
    around the 2^31st element against the oracle."""
    n, v = 70000, 32000
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GB")
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.empty(n, v, dtype=torch.bfloat16, device=DEV)
    for a in range(0, n, 5000):
        x[a:a + 5000].normal_(0, 2, generator=g)
    ids = torch.randint(0, v, (n,), generator=g, device=DEV)
    adv = torch.randn(n, generator=g, device=DEV)
    rows = np.array([0, 1, 67107, 67108, 67109, n - 2, n - 1])
    host, pick = x[rows].double().cpu().numpy(), ids[rows].cpu().numpy()
    lp = OL.log_softmax(host)[np.arange(len(rows)), pick]
    old = torch.full((n,), -12.0, device=DEV)
    old[rows] = torch.from_numpy(lp.astype(np.float32) + 0.05).to(DEV)
    out = ss.policy_loss(x, ids, old, adv, grad=x)
    c = dict(host=host, ids=pick, old=old[rows].cpu().numpy(), adv=adv[rows].cpu().numpy(),
             ref=np.zeros(len(rows), np.float32), w=np.ones(len(rows)))
    _, logps, grad = OL.policy(host, pick, c["old"], c["adv"], norm=n)
    tol = _lp_tol(host, pick, logps, v)
    assert (np.abs(out.logps[rows].double().cpu().numpy() - logps) <= tol).all()
    sens = np.abs(np.exp(logps - c["old"]) * c["adv"]) / n
    _check_grad(x[rows], grad, sens, tol, "bf16")
