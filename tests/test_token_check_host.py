"""The tight check of the token losses (tests/_token_check.py), on the CPU: it agrees
with the oracle, accepts the oracle's gradient rounded to its type, and does not
accept planted mistakes at the widths that take many chunks."""
import numpy as np
import pytest
import torch

import _token_check as TC
from oracle import token_loss as OL

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _case(n, v, dt, seed):
    r = np.random.default_rng(seed)
    x = r.normal(size=(n, v)) * 2
    ids, rows = r.integers(0, v, n), np.arange(n)
    x[rows, ids] += np.choose(rows % 3, [3.0, 14.0, 0.0])
    x[rows, (ids + 1) % v] += np.choose(rows % 3, [0.0, 0.0, 18.0])
    x = torch.from_numpy(x).to(DT[dt])
    host = x.double().numpy()
    lp = OL.log_softmax(host)[rows, ids]
    f = lambda q: np.float32(q).astype(np.float64)  # noqa: E731
    return x, host, ids, dict(old=f(lp + r.choice([-0.1, 0.05, 0.4, -0.5], n)),
                              adv=f(r.normal(size=n)), ref=f(lp + r.normal(size=n) * 0.2),
                              w=np.where(rows % 5 == 4, 0.0, r.choice([1.0, 0.5], n)))


@pytest.mark.parametrize("kl", [0.0, 0.05])
def test_the_check_agrees_with_the_oracle(kl):
    x, host, ids, s = _case(40, 300, "bf16", 1)
    y = torch.from_numpy(ids)
    q = {k: torch.from_numpy(v) for k, v in s.items()}
    a, t = TC.row_facts(x, y)
    want = OL.policy(host, ids, s["old"], s["adv"], s["ref"], s["w"], kl=kl)
    stats, errors, c, slack = TC.policy(a, t, q["old"], q["adv"], q["ref"], q["w"], kl,
                                        float(s["w"].sum()))
    assert np.allclose(stats, want[0], rtol=0, atol=1e-13)
    live = s["w"] != 0
    assert np.allclose(a[live], want[1][live], rtol=0, atol=1e-12)
    got = c[:, None] * (torch.nn.functional.one_hot(y, 300) - torch.softmax(x.double(), 1))
    assert np.abs(got.numpy() - want[2]).max() < 1e-15
    lens = [7, 5, 0, 8, 12, 8]
    want = OL.preference(host, ids, lens, s["ref"], 0.3, 0.1, s["w"])
    stats, _, r, _, c, _ = TC.preference(a, t, lens, q["ref"], q["w"], 0.3, 0.1, 3.0)
    assert np.allclose(stats, want[0], atol=1e-12) and np.allclose(r, want[1], atol=1e-12)
    got = c[:, None] * (torch.nn.functional.one_hot(y, 300) - torch.softmax(x.double(), 1))
    assert np.abs(got.numpy() - want[3]).max() < 1e-15


def _chunks(g, dt):
    return 16384 // g.element_size()


MISTAKES = {
    "zeros": lambda g, e: g * 0,
    "rows reversed": lambda g, e: g.flip(1),
    "rows swapped": lambda g, e: g.roll(1, 0),
    "a chunk from another row": lambda g, e: torch.cat([g[:, :e], g.roll(1, 0)[:, e:2 * e],
                                                        g[:, 2 * e:]], 1),
    "two chunks swapped": lambda g, e: torch.cat([g[:, e:2 * e], g[:, :e], g[:, 2 * e:]], 1),
    "a chunk of zeros": lambda g, e: torch.cat([g[:, :e], 0 * g[:, e:2 * e], g[:, 2 * e:]], 1),
    "one vector late": lambda g, e: g.roll(8, 1),
    "one per cent more": lambda g, e: g.double() * 1.01,
    "the last element": lambda g, e: torch.cat([g[:, :-1], g[:, -1:] * 0], 1),
}


@pytest.mark.parametrize("v,dt", [(32000, "bf16"), (50257, "bf16"), (50257, "f32"),
                                  (128256, "bf16"), (32000, "f32"), (50257, "f16")])
def test_planted_mistakes_are_seen(v, dt):
    n = 6
    x, host, ids, s = _case(n, v, dt, v)
    y, q = torch.from_numpy(ids), {k: torch.from_numpy(k2) for k, k2 in s.items()}
    a, t = TC.row_facts(x, y)
    # unclipped rows of one slope: weights of 1, a loss scale that fp16 holds
    c = torch.full((n,), 64.0 if dt == "f16" else 1e-3, dtype=torch.float64)
    slack = c * (t + 2.0 ** -20)
    want = (c[:, None] * (torch.nn.functional.one_hot(y, v) - torch.softmax(x.double(), 1)))
    good = want.to(DT[dt])
    assert not TC.gradient_misses(good, x, y, c, slack, t).any()
    e = _chunks(good, dt)
    for name, plant in MISTAKES.items():
        if dt == "f16" and name == "the last element":
            continue                              # it may be below fp16's smallest step
        bad = plant(good, e).to(DT[dt])
        misses = TC.gradient_misses(bad, x, y, c, slack, t)
        assert (misses > 0).all(), (name, misses)
        if name == "zeros" and dt != "f16":
            assert (misses > 0.99 * v).all(), misses
