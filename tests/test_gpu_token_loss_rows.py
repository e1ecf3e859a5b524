"""The token losses on rows that are not one heap of noise: ids far below the
row's largest logit with small slopes, confident rows, rows whose mass is one
other token; and calls without a token.  Against 64 bits."""
import math

import numpy as np
import pytest
import torch

import sharded_optimizer_step_gb300 as ss
from oracle import token_loss as OL

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = {"bf16": 2.0 ** -8, "f16": 2.0 ** -10, "f32": 2.0 ** -23}


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ss.build()
    yield
    assert ss.device_status() == 0


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


# ------------------------------------------------ gradients of unlikely ids

GAPS = [30.0, 45.0, 60.0, 70.0, 76.0, 80.0, 82.5]
SLOPES = [1e-2, 1e-4, 1e-6, 1e-7, 1e-8, 1e-9, 1e-10]


def _unlikely(v, dt):
    """A row for every gap between the largest logit and the id's and every
    weight; the references are the row's own log probabilities."""
    r = np.random.default_rng(v)
    n = len(GAPS) * len(SLOPES)
    x = r.normal(size=(n, v)) * 2
    rows, ids = np.arange(n), r.integers(0, v, n)
    top = (ids + 1 + r.integers(0, v - 1, n)) % v
    gap = np.repeat(GAPS, len(SLOPES))
    x[rows, top], x[rows, ids] = gap / 2, -gap / 2
    x = torch.from_numpy(x).to(DT[dt])
    host = x.double().numpy()
    lp = OL.log_softmax(host)[rows, ids].astype(np.float32)
    return x.to(DEV), host, ids, lp, np.tile(np.float32(SLOPES), len(GAPS))


def _check_relative(got, want, host, ids, lp, dt):
    """Every element to its own size: c moves by the log probability's error
    T = 2^-23 (|d| + |a| + 1), the element's exponential and the row's sum by
    their arguments' roundings, 2^-24 |t| log 2 each with |t| log 2 <= |a| + 1,
    and the result is rounded once; what is below 2^-125 may be flushed."""
    d = np.abs(host[np.arange(len(ids)), ids] - host.max(axis=1))
    rel = 4 * 2.0 ** -23 * (d + np.abs(lp.astype(np.float64)) + 1) + 2.0 ** -20
    bound = np.abs(want) * (EPS[dt] + rel[:, None]) + 2.0 ** -125
    got = got.double().cpu().numpy()
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (bad.any(axis=1).nonzero()[0], np.argwhere(bad)[:4], got[bad][:4],
                           want[bad][:4])


@pytest.mark.parametrize("shift", [0, 1], ids=["staged", "other_offsets"])
@pytest.mark.parametrize("v,dt", [(2003, "bf16"), (2003, "f32"), (16411, "bf16"),
                                  (120001, "bf16"), (60001, "f32")])
def test_gradients_of_unlikely_ids(v, dt, shift):
    x, host, ids, lp, w = _unlikely(v, dt)
    n = len(ids)
    g = torch.zeros(n * v + shift, dtype=DT[dt], device=DEV)[shift:].view(n, v)
    adv = np.where(np.arange(n) % 2, 1.0, -1.0).astype(np.float32)
    ss.policy_loss(x, _dev(ids), _dev(lp), _dev(adv), weights=_dev(w), norm=1.0, grad=g)
    _check_relative(g, OL.policy(host, ids, lp, adv, weights=w, norm=1.0)[2], host, ids, lp, dt)
    lens = [20, 9, 0, 4, 7, n - 40]
    ss.preference_loss(x, _dev(ids), lens, _dev(lp), beta=0.5, weights=_dev(w), norm=1.0, grad=g)
    want = OL.preference(host, ids, lens, lp, 0.5, 0.0, w, 1.0)[3]
    _check_relative(g, want, host, ids, lp, dt)


# ------------------------------------------------------ log probabilities

def _token_errors(x, ids):
    """Each token's log ratio against its exact log probability, 64 bits."""
    n = x.shape[0]
    exact = torch.cat([x[i:i + 512].double().gather(1, ids[i:i + 512, None])[:, 0] -
                       torch.logsumexp(x[i:i + 512].double(), 1) for i in range(0, n, 512)])
    out = ss.preference_loss(x, ids, [1] * n, exact.float())
    return out.log_ratios.double() + exact.float().double() - exact


@pytest.mark.parametrize("v,dt", [(4099, "bf16"), (4099, "f32"), (4096, "f16")])
@pytest.mark.parametrize("kind", ["confident", "other_5", "other_12", "other_20", "other_50"])
def test_log_ratios_of_peaked_rows_gather_no_common_error(kind, v, dt):
    """Rows whose mass is the id's (probability 0.9 to 1) or one other token's, 5
    to 50 above: the mean error over the rows whose dominant token lies at one
    place of a 16-byte vector stays at the level of rounding.  The argument t of
    the dominant exponential, |t| in [2^k, 2^(k+1)), rounds by up to 2^(k-24) either
    way, which moves the result by log 2 / sqrt(3) of that (rms); what else rounds
    is below 2^-25.  Equal arguments round alike, so a class counts as many draws
    as it has different ones; allowed are four standard deviations of its mean, and
    1.5e-8 for what is one-sided."""
    n, vec = 16384, 16 // (4 if dt == "f32" else 2)
    g = torch.Generator(device=DEV).manual_seed(v + len(kind))
    draw = lambda: torch.rand(n, device=DEV, generator=g)  # noqa: E731
    x = torch.randn(n, v, device=DEV, generator=g)
    rows = torch.arange(n, device=DEV)
    top = torch.randint(0, v, (n,), device=DEV, generator=g)
    if kind == "confident":
        ids = top
        x[rows, top] = math.log(v) + 0.5 + 2.2 + 4 * draw()      # p from 0.9 to 0.998
    else:
        gap = float(kind.split("_")[1])
        ids = (top + 1 + torch.randint(0, v - 1, (n,), device=DEV, generator=g)) % v
        x -= 24.0 + gap / 2
        x[rows, top] = gap / 2 + 4 + 4 * draw()
        x[rows, ids] = -gap / 2 + 4 - 3 * draw()
    x = x.to(DT[dt])
    error = _token_errors(x, ids)
    xt, ref = x[rows, top].double(), torch.round(x[rows, ids].double() / math.log(2))
    t = (xt / math.log(2) - ref).abs().clamp(min=0.5)
    var = torch.exp2(2 * (torch.floor(torch.log2(t)) - 24)) * math.log(2) ** 2 / 3 + 2.0 ** -50
    place = (rows * v + top) % vec
    for k in range(vec):
        e = error[place == k]
        draws = len(torch.unique(t[place == k]))
        assert len(e) > n / vec / 2
        limit = 1.5e-8 + 4 * math.sqrt(float(var[place == k].mean()) / draws)
        assert abs(float(e.mean())) < limit, (k, float(e.mean()), limit)


# ----------------------------------------------------- calls without a token

@pytest.mark.parametrize("weights", [False, True])
def test_pairs_without_a_token_have_the_loss_of_a_zero_margin(weights):
    x = torch.empty(0, 100, dtype=torch.bfloat16, device=DEV)
    e, i = torch.empty(0, device=DEV), torch.empty(0, dtype=torch.int64, device=DEV)
    kw = dict(weights=e) if weights else {}
    for lens in ([0, 0], [0, 0, 0, 0, 0, 0]):
        for ls, norm in ((0.0, None), (0.2, None), (0.1, 7.0)):
            want = OL.preference(np.zeros((0, 100)), np.zeros(0, int), lens, np.zeros(0), 0.3, ls,
                                 None, norm)[0]
            for grad in (None, x):
                out = ss.preference_loss(x, i, lens, e, beta=0.3, label_smoothing=ls, norm=norm,
                                         grad=grad, **kw)
                assert np.abs(out.stats.cpu().numpy() - want).max() <= 2.0 ** -23 * want.max()
                assert out.log_ratios.shape == (len(lens),) and not out.log_ratios.any()
    out = ss.preference_loss(x, i, [], e, **kw)
    assert not out.stats.any() and out.log_ratios.numel() == 0
    out = ss.policy_loss(x, i, e, e, grad=x, **kw)
    assert not out.stats.any() and out.logps.numel() == 0
