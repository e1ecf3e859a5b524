"""The oracle of the tuning operators against things other than itself:
finite differences of the losses, torch's log softmax and clipping, the code
tables by brute force, and the mean-gradient identity over micro-batches."""
import numpy as np
import pytest
import torch

from oracle import tensors as OT
from oracle import token_loss as OL


def _case(seed, n=6, v=11):
    r = np.random.default_rng(seed)
    x = r.normal(size=(n, v)) * 2
    ids = r.integers(0, v, n)
    lp = OL.log_softmax(x)[np.arange(n), ids]
    return r, x, ids, lp


@pytest.mark.parametrize("kl", [0.0, 0.07])
def test_policy_gradient_against_differences(kl):
    r, x, ids, lp = _case(1)
    old = lp + r.normal(size=len(ids)) * 0.4
    adv, ref = r.normal(size=len(ids)), lp + r.normal(size=len(ids)) * 0.2
    w = np.array([1, 0, 2, 1, 0.5, 1.0])
    args = dict(ref=ref, weights=w, clip_low=0.2, clip_high=0.3, kl=kl)
    u = np.exp(lp - old)
    assert np.abs(u - 0.8).min() > 1e-3 and np.abs(u - 1.3).min() > 1e-3
    stats, logps, grad = OL.policy(x, ids, old, adv, **args)
    eps = 1e-5
    for i in range(x.shape[0]):
        for j in range(x.shape[1]):
            up, dn = x.copy(), x.copy()
            up[i, j] += eps
            dn[i, j] -= eps
            d = (OL.policy(up, ids, old, adv, **args)[0][0]
                 - OL.policy(dn, ids, old, adv, **args)[0][0]) / (2 * eps)
            assert abs(d - grad[i, j]) < 1e-8
    assert not grad[1].any() and logps[1] == 0


def test_policy_against_torch():
    r, x, ids, lp = _case(2, 64, 37)
    old, adv = lp + r.normal(size=64) * 0.4, r.normal(size=64)
    ref = lp + r.normal(size=64) * 0.2
    t = torch.tensor(x, requires_grad=True)
    a = torch.log_softmax(t, 1)[torch.arange(64), torch.tensor(ids)]
    u = torch.exp(a - torch.tensor(old))
    A, d = torch.tensor(adv), torch.tensor(ref) - a
    pg = -torch.minimum(u * A, u.clamp(0.8, 1.2) * A)
    loss = (pg + 0.05 * (torch.exp(d) - d - 1)).mean()
    loss.backward()
    stats, logps, grad = OL.policy(x, ids, old, adv, ref=ref, kl=0.05)
    assert abs(stats[0] - float(loss)) < 1e-12
    assert np.abs(grad - t.grad.numpy()).max() < 1e-12
    assert np.abs(logps - a.detach().numpy()).max() < 1e-12


@pytest.mark.parametrize("smoothing", [0.0, 0.2])
def test_preference_gradient_against_differences(smoothing):
    r, x, ids, lp = _case(3, 9, 7)
    lens = [3, 2, 0, 4]
    w = np.array([1, 1, 0, 1, 0.5, 1, 1, 0, 1.0])
    ref = lp + r.normal(size=9) * 0.3
    args = dict(beta=0.7, smoothing=smoothing, weights=w)
    stats, ratios, logps, grad = OL.preference(x, ids, lens, ref, **args)
    eps = 1e-5
    for i in range(9):
        for j in range(7):
            up, dn = x.copy(), x.copy()
            up[i, j] += eps
            dn[i, j] -= eps
            d = (OL.preference(up, ids, lens, ref, **args)[0][0]
                 - OL.preference(dn, ids, lens, ref, **args)[0][0]) / (2 * eps)
            assert abs(d - grad[i, j]) < 1e-8
    assert ratios[2] == 0 and not grad[2].any()


def test_micro_batches_with_the_global_norm_add_up_to_one_batch():
    r, x, ids, lp = _case(4, 8, 5)
    old, adv = lp + r.normal(size=8) * 0.3, r.normal(size=8)
    whole = OL.policy(x, ids, old, adv)
    parts = [OL.policy(x[s], ids[s], old[s], adv[s], norm=8) for s in (slice(0, 3), slice(3, 8))]
    assert np.abs(sum(p[0] for p in parts) - whole[0]).max() < 1e-12
    assert np.abs(np.concatenate([p[2] for p in parts]) - whole[2]).max() < 1e-12


def test_e4m3_codes_are_torchs():
    x = np.random.default_rng(0).normal(size=1 << 16).astype(np.float32) * 60
    x = np.clip(x, -448, 448)
    want = torch.tensor(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    k = OT._nearest(np.abs(x), OT.e4m3_values()[:127], True)
    assert np.array_equal(np.where(np.signbit(x), k + 128, k), want)


def test_codes_are_the_nearest_by_brute_force():
    r = np.random.default_rng(5)
    m = (r.normal(size=1000) * np.exp(r.normal(size=1000) * 3)).astype(np.float32)
    for encode, decode, values, x in (
            (OT.encode_m, OT.decode_m, OT.e4m3_values(), m),
            (OT.encode_r, OT.decode_r, OT.root_values(), np.abs(m))):
        code, scale = encode(x)
        each = np.repeat(scale, OT.BLOCK)[:1000].astype(np.float64)
        values = values[np.isfinite(values)]
        best = np.abs(values[None, :] * each[:, None] - x[:, None]).min(axis=1)
        got = np.abs(decode(code, scale).astype(np.float64) - x)
        # the root never rounds a non-zero value to zero
        floor = 1.0625 * 2.0 ** -15 * each if encode is OT.encode_r else 0.0
        assert (got <= np.maximum(best, floor) * (1 + 1e-5) + each * 1e-5).all()
    code, scale = OT.encode_r(np.abs(m))
    assert (code[np.abs(m) > 0] > 0).all()


def test_largest_element_survives_and_tiny_blocks_are_zero():
    x = np.zeros(600, np.float32)
    x[3], x[300], x[599] = 3.0, -1e-20, 1e-31
    code, scale = OT.encode_m(x)
    y = OT.decode_m(code, scale)
    assert abs(y[3] - 3) < 1e-6 and abs(y[300] + 1e-20) < 1e-26 and y[599] == 0
    assert scale[2] == 0
    code, scale = OT.encode_r(np.array([1.0, np.nan, 2.0], np.float32))
    assert np.isnan(scale[0])


def test_adamw8_follows_adamw32_within_the_codes_step():
    """From zero moments, one step: the parameters are those of exact moments
    (they are formed before rounding), the moments within a code's step."""
    r = np.random.default_rng(6)
    from oracle.numerics import AdamWConfig, adamw
    hp = AdamWConfig()
    g = r.normal(size=700).astype(np.float32) * 1e-3
    p = r.normal(size=700).astype(np.float32)
    z = np.zeros(700, np.float32)
    b = np.zeros(3, np.float32)
    c = np.zeros(700, np.uint8)
    p8, mc, ms, vc, vs = OT.adamw8(g, p, c, b, c, b, hp, 1)
    p32, m32, v32 = adamw(p, z, z, g, hp, 1)[:3]
    assert np.array_equal(p8, p32)
    top = np.repeat(ms, 256)[:700] * 448
    assert (np.abs(OT.decode_m(mc, ms) - m32) <= np.maximum(np.abs(m32) / 16, top * 2 ** -18)).all()
    root = OT.decode_r(vc, vs)
    assert (np.abs(root - np.sqrt(v32)) <= np.sqrt(v32) / 31.9 + np.repeat(vs, 256)[:700] * 2 ** -14).all()
