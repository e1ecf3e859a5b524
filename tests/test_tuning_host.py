"""Refusals of the tuning operators' entry points, without a GPU: every call
here is rejected (or has nothing to do) before anything is launched, so the
device addresses are made up and never followed."""
import ctypes

import pytest

import sharded_optimizer_step_gb300 as ss
from sharded_optimizer_step_gb300 import _capi

A = 1 << 40
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def built():
    ss.build()


def _tokens(**kw):
    f = dict(logits=A, row_stride=100, dtype=0, id_bytes=8, ids=A + (1 << 30), n_tokens=8,
             vocab=100, weights=None, ref_logps=A + (2 << 30), logps=A + (3 << 30),
             grad=A + (4 << 30), grad_stride=100, grad_scale=1.0, norm=0.0, loss_scale=None,
             stats=A + (5 << 30), workspace=A + (6 << 30), workspace_bytes=1 << 20)
    f.update(kw)
    return _capi.TokenLoss(**f)


def _policy(args, old=A + (7 << 30), adv=A + (8 << 30), lo=0.2, hi=0.2, kl=0.0):
    return _capi.lib().token_policy_loss(ctypes.byref(args), old, adv, lo, hi, kl, None)


def _pref(args, lens=(2, 2, 4, 0), beta=0.1, ls=0.0, ratios=A + (9 << 30), pairs=None):
    return _capi.lib().token_preference_loss(
        ctypes.byref(args), _capi.i64_array(lens), len(lens) // 2 if pairs is None else pairs,
        beta, ls, ratios, None)


BAD_TOKENS = [
    dict(dtype=7), dict(id_bytes=2), dict(n_tokens=-1), dict(vocab=0), dict(vocab=1 << 31),
    dict(row_stride=99), dict(grad_stride=99), dict(row_stride=1 << 60), dict(logits=None),
    dict(ids=None), dict(logps=None), dict(stats=None), dict(workspace=None),
    dict(logits=A + 1), dict(grad=A + (4 << 30) + 1), dict(ids=A + (1 << 30) + 4),
    dict(weights=A + (10 << 30) + 2), dict(workspace=A + (6 << 30) + 4), dict(workspace_bytes=64),
    dict(grad_scale=INF), dict(grad_scale=NAN), dict(norm=-1.0), dict(norm=INF), dict(norm=NAN),
    dict(loss_scale=A + (10 << 30) + 1),
    dict(grad=A, grad_stride=104),                  # in place with another stride
    dict(grad=A + 200),                             # partly over the logits
    dict(logps=A + (5 << 30)),                      # logps over stats
    dict(weights=A + (3 << 30)),                    # weights over logps
    dict(stats=A + 100),                            # stats inside the logits
]


@pytest.mark.parametrize("bad", BAD_TOKENS, ids=[str(b)[:40] for b in BAD_TOKENS])
def test_both_losses_refuse(bad):
    assert _policy(_tokens(**bad)) == _capi.ERR_INVALID
    assert _capi.lib().shardstep_last_error()
    assert _pref(_tokens(**bad)) == _capi.ERR_INVALID


def test_widest_vocabulary():
    """A row's byte offsets are 32-bit in the kernels; the check comes first."""
    wide = dict(vocab=(1 << 28) + 1, row_stride=(1 << 28) + 1, grad=None, n_tokens=1)
    assert _policy(_tokens(**wide)) == _capi.ERR_INVALID
    assert b"vocab" in _capi.lib().shardstep_last_error()
    assert _pref(_tokens(**wide), lens=(1, 0)) == _capi.ERR_INVALID
    assert b"vocab" in _capi.lib().shardstep_last_error()


def test_policy_refuses():
    t = _tokens()
    assert _capi.lib().token_policy_loss(None, A, A, 0.2, 0.2, 0.0, None) == _capi.ERR_INVALID
    for kw in (dict(old=None), dict(adv=None), dict(old=A + (7 << 30) + 1), dict(lo=-0.1),
               dict(lo=1.5), dict(hi=-1.0), dict(hi=INF), dict(kl=-1.0), dict(kl=NAN),
               dict(old=A + (3 << 30))):
        assert _policy(t, **kw) == _capi.ERR_INVALID, kw
    assert _policy(_tokens(ref_logps=None), kl=0.1) == _capi.ERR_INVALID
    assert _policy(_tokens(n_tokens=0, logits=None, ids=None)) == _capi.OK


def test_preference_refuses():
    t = _tokens()
    assert _capi.lib().token_preference_loss(None, None, 0, 0.1, 0.0, A, None) == \
        _capi.ERR_INVALID
    for kw in (dict(lens=(2, 2, 4, 1)), dict(lens=(9, -1, 0, 0)), dict(pairs=-1),
               dict(beta=INF), dict(ls=0.6), dict(ls=-0.1), dict(ls=NAN), dict(ratios=None),
               dict(ratios=A + (9 << 30) + 2), dict(ratios=A + (3 << 30))):
        assert _pref(t, **kw) == _capi.ERR_INVALID, kw
    assert _pref(_tokens(ref_logps=None)) == _capi.ERR_INVALID
    assert _pref(_tokens(n_tokens=0), lens=(0, 0)) == _capi.OK
    need = _capi.lib().token_loss_workspace_bytes(8, 2)
    assert _pref(_tokens(workspace_bytes=need - 1)) == _capi.ERR_INVALID
    assert "workspace" in _capi.lib().shardstep_last_error().decode()
    assert _capi.lib().token_loss_workspace_bytes(-1, 0) == -1
    assert _capi.lib().token_loss_workspace_bytes(0, -1) == -1


def _list(n=2, numel=1000, grad_step=1 << 20, bits=8, **kw):
    ts = (_capi.Tensor * n)()
    for i in range(n):
        b = A + (i << 24)
        ts[i] = _capi.Tensor(b + (1 << 32), b + (2 << 32), b + (3 << 32), b + (4 << 32),
                             b + (5 << 32), b + (6 << 32), numel, 0, 0)
    for k, v in kw.items():
        setattr(ts[0], k, v)
    return [A + i * grad_step for i in range(n)], ts


def _step(grads, ts, gd=0, pd=0, bits=8, groups=1, step=1, coef=None, skip=None):
    hp = (_capi.AdamWHP * 16)(*[ss.AdamW().at_step(step)] * 16)
    return _capi.lib().tensors_adamw_step(_capi.ptr_array(grads), ts, len(ts), gd, pd, bits, hp,
                                          groups, coef, skip, None)


def test_tensors_adamw_step_refuses():
    g, ts = _list()
    for kw in (dict(gd=9), dict(pd=1), dict(bits=16), dict(groups=0), dict(step=0),
               dict(coef=A + 1), dict(skip=A + 2)):
        assert _step(g, ts, **kw) == _capi.ERR_INVALID, kw
    assert _step(g, ts, groups=9) == _capi.ERR_CAPACITY
    for kw in (dict(numel=-1), dict(group=1), dict(group=-1), dict(master=None), dict(m=None),
               dict(v=None), dict(m_scale=None), dict(v_scale=None), dict(master=A + 2),
               dict(param=A + 1), dict(m_scale=A + 1), dict(numel=1 << 41)):
        g2, t2 = _list(**kw)
        assert _step(g2, t2) == _capi.ERR_INVALID, kw
    assert _step([0, g[1]], ts) == _capi.ERR_INVALID            # NULL gradient
    assert _step([g[0] + 1, g[1]], ts) == _capi.ERR_INVALID     # misaligned gradient
    assert _step([ts[0].master, g[1]], ts) == _capi.ERR_INVALID  # gradient over an output
    g2, t2 = _list(v=A + (2 << 32) + 999)                       # v over m's last code
    assert _step(g2, t2) == _capi.ERR_INVALID
    assert "overlap" in _capi.lib().shardstep_last_error().decode()
    L = _capi.lib()
    assert L.tensors_adamw_step(None, ts, 2, 0, 0, 8, (_capi.AdamWHP * 1)(ss.AdamW().at_step(1)),
                                1, None, None, None) == _capi.ERR_INVALID
    assert L.tensors_adamw_step(None, None, 0, 0, 0, 8, None, 1, None, None, None) == \
        _capi.ERR_INVALID                                       # hp NULL
    for states in (None, _capi.ptr_array([0]), _capi.ptr_array([A + 4])):
        assert L.tensors_state_adamw_step(_capi.ptr_array(g), ts, 2, 0, 0, 8, states, 1, None,
                                          None, None) == _capi.ERR_INVALID


def test_step_words_may_not_lie_in_its_outputs():
    """The factor, the skip word and the step states are read by every block while
    others write."""
    g, ts = _list()
    inside = ts[0].master + 8
    for kw in (dict(coef=inside), dict(skip=inside)):
        assert _step(g, ts, **kw) == _capi.ERR_INVALID, kw
        assert "overlap" in _capi.lib().shardstep_last_error().decode()
    assert _capi.lib().tensors_state_adamw_step(
        _capi.ptr_array(g), ts, 2, 0, 0, 8, _capi.ptr_array([inside]), 1, None, None,
        None) == _capi.ERR_INVALID
    assert "overlap" in _capi.lib().shardstep_last_error().decode()


def test_empty_lists_are_nothing_to_do():
    assert _step([], (_capi.Tensor * 0)()) == _capi.OK
    ts = (_capi.Tensor * 3)()                                   # numel 0, NULL arrays
    assert _step([0, 0, 0], ts) == _capi.OK
    assert _capi.lib().tensors_moments_decode(None, None, None, None, 0, None, None, None) == 0


def test_moments_and_norm_refuse():
    L = _capi.lib()
    a = [A + (i << 30) for i in range(6)]
    for f in (L.tensors_moments_decode,):
        assert f(a[0], a[1], a[2], a[3], -1, a[4], a[5], None) == _capi.ERR_INVALID
        assert f(a[0], None, a[2], a[3], 8, a[4], a[5], None) == _capi.ERR_INVALID
        assert f(a[0], a[1], a[2], a[3], 8, a[4], a[4] + 28, None) == _capi.ERR_INVALID
        assert f(a[0], a[1], a[2], a[3], 8, a[0], a[5], None) == _capi.ERR_INVALID
        assert f(a[0], a[1] + 1, a[2], a[3], 8, a[4], a[5], None) == _capi.ERR_INVALID
    assert L.tensors_moments_encode(a[4], a[5], 8, a[0], a[1], a[0] + 4, a[3], None) == \
        _capi.ERR_INVALID

    def norm(g=(A, A + 4096), n=(8, 8), dt=0, mx=1.0, scale=None, out=a[1], found=None, ws=a[2]):
        return L.tensors_grad_norm(_capi.ptr_array(g), _capi.i64_array(n), len(n), dt, mx, scale,
                                   out, found, ws, None)
    for kw in (dict(dt=5), dict(mx=0.0), dict(mx=NAN), dict(mx=-1.0), dict(out=None),
               dict(ws=None), dict(ws=a[2] + 4), dict(out=a[1] + 2), dict(n=(8, -1)),
               dict(g=(A, 0)), dict(g=(A, A + 4097)), dict(scale=A + (7 << 30) + 1),
               dict(found=a[3] + 1), dict(out=A + 8), dict(found=a[1] + 4), dict(found=a[2] + 64),
               dict(n=(8, 1 << 41))):
        assert norm(**kw) == _capi.ERR_INVALID, kw


def test_python_wrappers_refuse_on_the_host():
    import torch
    x, ids = torch.zeros(2, 4), torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError):
        ss.policy_loss(x, ids, ids, ids)                        # not CUDA
    with pytest.raises(ValueError):
        ss.TensorList([x])
    with pytest.raises(ValueError):
        ss.TensorAdamW([], ss.AdamW())
    with pytest.raises(ValueError):
        ss.TensorAdamW([x], ss.AdamW(), state_bits=16)
    with pytest.raises(ValueError):
        ss.grad_norm_clip([], 1.0)
