"""The token losses on rows that are not one heap of noise: ids far below the
row's largest logit with small slopes; and calls without a token.  Against 64
bits."""
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
