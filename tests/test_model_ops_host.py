"""Refusals of the embedding, layer norm and matrix entry points, without a GPU:
every call here is rejected (or has nothing to do) before anything is launched,
so the device addresses are made up and never followed."""
import ctypes

import pytest
import torch

import sharded_optimizer_step_gb300 as ss
from sharded_optimizer_step_gb300 import _capi

A = 1 << 40
G = 1 << 30
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def built():
    ss.build()


def _name(bad):
    return ",".join(k + "=" + (repr(v) if not isinstance(v, (ctypes.Structure, list)) else "bad")
                    for k, v in bad.items())


def _call(name, defaults, **kw):
    f = dict(defaults)
    assert not set(kw) - set(f), kw
    f.update(kw)
    return getattr(_capi.lib(), name)(*f.values())


LOOKUP = dict(table=A, table_stride=64, dtype=0, vocab=100, dim=64, ids=A + G, id_bytes=8, n=10,
              scale=1.0, out=A + 2 * G, out_stride=64, stream=None)


@pytest.mark.parametrize("bad", [
    dict(table=None), dict(ids=None), dict(out=None), dict(dtype=5), dict(id_bytes=2), dict(n=-1),
    dict(n=1 << 31), dict(vocab=0), dict(vocab=1 << 31), dict(dim=0), dict(dim=(1 << 23) + 1),
    dict(table_stride=63), dict(out_stride=63), dict(table_stride=1 << 60), dict(scale=INF),
    dict(scale=NAN), dict(table=A + 1), dict(out=A + 2 * G + 1), dict(ids=A + G + 4),
    dict(out=A), dict(out=A + 64 * 100 * 2 - 2), dict(out=A + G + 40),
], ids=str)
def test_lookup_refuses(bad):
    assert _call("token_embedding", LOOKUP, **bad) == _capi.ERR_INVALID
    assert _capi.lib().shardstep_last_error()


def test_lookup_without_tokens():
    assert _call("token_embedding", LOOKUP, n=0, ids=None, out=None) == _capi.OK


GRAD = dict(d_out=A, d_out_stride=64, dtype=0, ids=A + G, id_bytes=4, n=10, scale=1.0,
            grad=A + 2 * G, grad_stride=64, grad_dtype=1, vocab=100, dim=64, accumulate=0,
            workspace=A + 3 * G, workspace_bytes=1 << 20, stream=None)


@pytest.mark.parametrize("bad", [
    dict(d_out=None), dict(ids=None), dict(grad=None), dict(workspace=None), dict(dtype=-1),
    dict(grad_dtype=3), dict(id_bytes=1), dict(n=-1), dict(vocab=0), dict(dim=0),
    dict(d_out_stride=60), dict(grad_stride=63), dict(scale=NAN), dict(d_out=A + 1),
    dict(grad=A + 2 * G + 2), dict(ids=A + G + 2), dict(workspace=A + 3 * G + 8),
    dict(workspace_bytes=1000), dict(grad=A), dict(workspace=A), dict(grad=A + 3 * G + 64),
    dict(grad=A + G),
], ids=str)
def test_embedding_grad_refuses(bad):
    assert _call("token_embedding_grad", GRAD, **bad) == _capi.ERR_INVALID
    assert _capi.lib().shardstep_last_error()


def test_embedding_grad_workspace():
    need = _capi.lib().token_embedding_grad_workspace_bytes
    assert need(-1, 10, 8) == need(10, 0, 8) == need(10, 10, 0) == need(1 << 31, 1, 1) == -1
    for n, vocab, dim in ((0, 1, 1), (10, 100, 64), (16384, 32000, 4096), (1 << 20, 50257, 768)):
        # the sorted list, each id's place, two pieces per chunk of 8 to 512 tokens
        assert need(n, vocab, dim) >= 8 * n + 4 * (vocab + 1) + 8 * dim * (n // 512)
        assert need(n, vocab, dim) <= 8 * n + 4 * vocab + 64 + 8 * dim * (n // 8 + 1)
    assert _call("token_embedding_grad", GRAD, n=0, accumulate=1) == _capi.OK


NORM = dict(x=A, x_stride=64, dtype=0, rows=10, cols=64, weight=A + G, bias=A + 2 * G,
            weight_dtype=1, eps=1e-5, out=A + 3 * G, out_stride=64, mean=A + 4 * G,
            rstd=A + 5 * G, stream=None)


@pytest.mark.parametrize("bad", [
    dict(x=None), dict(out=None), dict(mean=None), dict(rstd=None), dict(dtype=9),
    dict(weight_dtype=2), dict(rows=-1), dict(cols=0), dict(cols=(1 << 24) + 1),
    dict(x_stride=63), dict(out_stride=1), dict(eps=-1.0), dict(eps=NAN), dict(eps=INF),
    dict(x=A + 1), dict(weight=A + G + 2), dict(mean=A + 4 * G + 1), dict(out=A),
    dict(mean=A + 5 * G), dict(out=A + G), dict(rstd=A + 100),
], ids=str)
def test_layer_norm_refuses(bad):
    assert _call("rows_layer_norm", NORM, **bad) == _capi.ERR_INVALID
    assert _capi.lib().shardstep_last_error()


NORM_GRAD = dict(d_out=A, d_out_stride=64, x=A + G, x_stride=64, dtype=0, rows=10, cols=64,
                 mean=A + 2 * G, rstd=A + 3 * G, weight=A + 4 * G, weight_dtype=0,
                 d_x=A + 5 * G, d_x_stride=64, d_weight=A + 6 * G, d_bias=A + 7 * G,
                 accumulate=0, workspace=A + 8 * G, workspace_bytes=1 << 20, stream=None)


@pytest.mark.parametrize("bad", [
    dict(d_out=None), dict(x=None), dict(mean=None), dict(rstd=None), dict(workspace=None),
    dict(dtype=3), dict(weight_dtype=2), dict(rows=-1), dict(cols=0), dict(d_out_stride=2),
    dict(x_stride=63), dict(d_x_stride=63), dict(d_out=A + 1), dict(x=A + G + 1),
    dict(d_x=A + 5 * G + 1), dict(d_weight=A + 6 * G + 1), dict(rstd=A + 3 * G + 2),
    dict(workspace=A + 8 * G + 4), dict(workspace_bytes=1000), dict(d_x=A), dict(d_x=A + G),
    dict(d_weight=A + 7 * G), dict(d_bias=A + 2 * G), dict(d_weight=A + 8 * G),
    dict(d_weight=A + 4 * G),
], ids=str)
def test_layer_norm_grad_refuses(bad):
    assert _call("rows_layer_norm_grad", NORM_GRAD, **bad) == _capi.ERR_INVALID
    assert _capi.lib().shardstep_last_error()


def test_layer_norm_with_nothing_to_do():
    assert _call("rows_layer_norm", NORM, rows=0, x=None, out=None) == _capi.OK
    nothing = dict(d_x=None, d_weight=None, d_bias=None, workspace=None, workspace_bytes=0)
    assert _call("rows_layer_norm_grad", NORM_GRAD, **nothing) == _capi.OK
    assert _call("rows_layer_norm_grad", NORM_GRAD, rows=0, accumulate=1) == _capi.OK
    assert _capi.lib().rows_layer_norm_workspace_bytes(0) == -1
    assert _capi.lib().rows_layer_norm_workspace_bytes(64) >= 8 * 64 * 152


# --------------------------------------------------------------- matrices

USUAL = _capi.Quintic(*ss.QUINTIC, 1e-7, 5, 0)
OUT_OF_RANGE = [
    _capi.Quintic(*ss.QUINTIC, 1e-7, 0, 0), _capi.Quintic(*ss.QUINTIC, 1e-7, 65, 0),
    _capi.Quintic(*ss.QUINTIC, -1.0, 5, 0), _capi.Quintic(*ss.QUINTIC, NAN, 5, 0),
    _capi.Quintic(NAN, -1.0, 1.0, 1e-7, 5, 0), _capi.Quintic(1.5, INF, 0.0, 1e-7, 5, 0),
    _capi.Quintic(4.0, -1.0, 0.0, 1e-7, 5, 0),       # grows past what halves hold
    _capi.Quintic(1.0, -8.0, 7.0, 1e-7, 1, 0),       # b does
    _capi.Quintic(1.0, 1.0, 2.0, 1e-7, 1, 0),        # a + b + c does
    _capi.Quintic(1.39, 0.0, 0.0, 1e-7, 3, 0),       # in its second round
]


def _orthogonalize(n=2, rows=(10, 20), cols=(30, 5), ins=(A, A + G), outs=(A + 2 * G, A + 3 * G),
                   in_dtype=0, out_dtype=1, quintic=USUAL, ws=A + 4 * G, ws_bytes=1 << 30):
    return _capi.lib().matrices_orthogonalize(
        _capi.ptr_array(ins) if ins else None, _capi.ptr_array(outs) if outs else None,
        _capi.i64_array(rows) if rows else None, _capi.i64_array(cols) if cols else None, n,
        in_dtype, out_dtype, ctypes.byref(quintic) if quintic else None, ws, ws_bytes, None)


@pytest.mark.parametrize("bad", [
    dict(n=-1), dict(rows=None), dict(cols=None), dict(ins=None), dict(outs=None),
    dict(rows=(-1, 5)), dict(cols=((1 << 20) + 1, 5)), dict(ins=(None, A)), dict(outs=(A, None)),
    dict(ins=(A + 1, A + G)), dict(outs=(A + 2 * G + 2, A + 3 * G)), dict(in_dtype=4),
    dict(out_dtype=-1), dict(quintic=None), dict(ws=None), dict(ws=A + 4 * G + 8),
    dict(ws_bytes=1000), dict(outs=(A, A + 3 * G)), dict(outs=(A + 2 * G, A + 2 * G)),
    dict(ws=A), dict(outs=(A + 2 * G, A + 4 * G)),
] + [dict(quintic=q) for q in OUT_OF_RANGE], ids=_name)
def test_orthogonalize_refuses(bad):
    assert _orthogonalize(**bad) == _capi.ERR_INVALID
    assert _capi.lib().shardstep_last_error()


def test_matrices_workspace():
    need = lambda r, c: _capi.lib().matrices_workspace_bytes(  # noqa: E731
        _capi.i64_array(r), _capi.i64_array(c), len(r))
    assert need([-1], [3]) == need([3], [(1 << 20) + 1]) == -1 and need([], []) == 0
    assert need([0, 7], [9, 0]) == 0
    one = need([1], [1])
    assert one == 32 * 256 * 256 + 2176 and need([128], [100]) == need([100], [128]) == one
    assert need([600], [700]) == 32 * 768 * 768 + 2176
    assert need([200] * 3, [300] * 3) == 3 * need([200], [300])
    assert need([5] * 200, [5] * 200) == 64 * one          # a group at a time
    assert need([8192] * 9, [8192] * 9) == need([8192], [8192])
    assert _orthogonalize(n=0, ws=None, ws_bytes=0) == _capi.OK
    assert _orthogonalize(rows=(0, 3), cols=(4, 0), ins=(None, None), outs=(None, None), ws=None,
                          ws_bytes=0) == _capi.OK


def _muon(mats=None, n=1, grad_dtype=0, param_dtype=0, hp=None, groups=None, quintic=USUAL,
          coef=None, skip=None, ws=A + 4 * G, ws_bytes=1 << 30, **kw):
    m = dict(grad=A, master=A + G, m=A + 2 * G, param=A + 3 * G, rows=20, cols=30, group=0,
             pad_=0)
    m.update(kw)
    hp = hp or [_capi.MuonHP(1e-3, 0.95, 0.1, 0.2, 1, 0)]
    return _capi.lib().tensors_muon_step(
        (_capi.Matrix * 1)(_capi.Matrix(**m)) if mats is None else mats, n, grad_dtype,
        param_dtype, (_capi.MuonHP * len(hp))(*hp), len(hp) if groups is None else groups,
        ctypes.byref(quintic) if quintic else None, coef, skip, ws, ws_bytes, None)


@pytest.mark.parametrize("bad", [
    dict(n=-1), dict(grad_dtype=3), dict(param_dtype=1), dict(groups=0), dict(quintic=None),
    dict(coef=A + 9 * G + 1), dict(skip=A + 9 * G + 2), dict(ws=None), dict(ws=A + 4 * G + 4),
    dict(ws_bytes=5000), dict(grad=None), dict(master=None), dict(m=None), dict(rows=-1),
    dict(cols=1 << 21), dict(group=1), dict(group=-1), dict(grad=A + 1), dict(master=A + G + 2),
    dict(m=A + 2 * G + 1), dict(param=A + 3 * G + 1), dict(m=A + G), dict(grad=A + G),
    dict(param=A + G + 16), dict(coef=A + G), dict(skip=A + 2 * G + 8), dict(ws=A + 3 * G),
] + [dict(hp=[_capi.MuonHP(*v, 1, 0)]) for v in (
    (NAN, 0.9, 0.1, 0.2), (1e-3, 1.0, 0.1, 0.2), (1e-3, -0.1, 0.1, 0.2), (1e-3, NAN, 0.1, 0.2),
    (1e-3, 0.9, INF, 0.2), (1e-3, 0.9, 0.1, -1.0), (1e-3, 0.9, 0.1, INF))] + [
    dict(quintic=q) for q in OUT_OF_RANGE], ids=_name)
def test_muon_refuses(bad):
    assert _muon(**bad) == _capi.ERR_INVALID
    assert _capi.lib().shardstep_last_error()


def test_muon_capacity_and_nothing_to_do():
    nine = [_capi.MuonHP(1e-3, 0.95, 0.1, 0.2, 1, 0)] * 9
    assert _muon(hp=nine) == _capi.ERR_CAPACITY
    assert _muon(n=0, ws=None, ws_bytes=0) == _capi.OK
    assert _muon(rows=0, grad=None, master=None, m=None, param=None, ws=None,
                 ws_bytes=0) == _capi.OK


# ------------------------------------------------- the wrappers' own checks

class _Claimed(torch.Tensor):
    is_cuda = True


def _claim(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(_Claimed)


@pytest.fixture
def wrappers(monkeypatch):
    """Tensors that claim to be on a GPU, no stream, and a library that must not be
    reached."""
    import contextlib

    class Never:
        def __getattr__(self, name):
            if name.endswith("workspace_bytes"):
                return lambda *a: 64
            raise AssertionError(f"{name} was reached")
    monkeypatch.setattr(_capi, "lib", lambda: Never())
    monkeypatch.setattr(ss, "_here", lambda device, stream: contextlib.nullcontext())
    monkeypatch.setattr(ss, "_elsewhere", lambda device, stream: False)
    monkeypatch.setattr(ss._Scratch, "at_least", lambda self, nbytes: (4096, nbytes))


def test_wrappers_refuse(wrappers):
    ids = _claim(6, dtype=torch.int64)
    table, out = _claim(9, 8), _claim(6, 8)
    x, mean, w = _claim(5, 8), _claim(5), _claim(8)
    half = torch.bfloat16
    bad = [
        lambda: ss.embedding(_claim(9), ids), lambda: ss.embedding(_claim(0, 8), ids),
        lambda: ss.embedding(torch.zeros(9, 8), ids),
        lambda: ss.embedding(table, _claim(6)), lambda: ss.embedding(table, ids[::2]),
        lambda: ss.embedding(table, ids, out=_claim(5, 8)),
        lambda: ss.embedding(table, ids, out=_claim(6, 7)),
        lambda: ss.embedding(table, ids, out=_claim(6, 8, dtype=half)),
        lambda: ss.embedding(table, ids, out=_claim(8, 6).t()),
        lambda: ss.embedding(_claim(1, 8).expand(9, 8), ids),
        lambda: ss.embedding_grad(out, ids, _claim(9)),
        lambda: ss.embedding_grad(_claim(5, 8), ids, table),
        lambda: ss.embedding_grad(_claim(6, 7), ids, table),
        lambda: ss.embedding_grad(_claim(1, 8).expand(6, 8), ids, table),
        lambda: ss.embedding_grad(out, ids, _claim(1, 8).expand(9, 8)),
        lambda: ss.layer_norm(x, _claim(7)), lambda: ss.layer_norm(x, _claim(8, dtype=half)),
        lambda: ss.layer_norm(_claim(5, 8, dtype=half), w, _claim(8, dtype=half)),
        lambda: ss.layer_norm(x, torch.zeros(8)), lambda: ss.layer_norm(x, out=_claim(5, 9)),
        lambda: ss.layer_norm(x, out=_claim(5, 8, dtype=half)), lambda: ss.layer_norm(_claim(5, 0)),
        lambda: ss.layer_norm(_claim(8, 5).t()),
        lambda: ss.layer_norm_grad(_claim(5, 7), x, mean, mean),
        lambda: ss.layer_norm_grad(_claim(5, 8, dtype=half), x, mean, mean),
        lambda: ss.layer_norm_grad(x, x, _claim(4), mean),
        lambda: ss.layer_norm_grad(x, x, mean, _claim(5, dtype=half)),
        lambda: ss.layer_norm_grad(x, x, mean, mean, d_x=_claim(5, 9)),
        lambda: ss.layer_norm_grad(_claim(5, 8, dtype=half), _claim(5, 8, dtype=half), mean, mean,
                                   w, d_weight=_claim(8, dtype=half)),
        lambda: ss.orthogonalize(_claim(4)), lambda: ss.orthogonalize(_claim(4, 5).t()),
        lambda: ss.orthogonalize(torch.zeros(4, 5)),
        lambda: ss.orthogonalize([_claim(4, 5), _claim(4, 5, dtype=half)]),
        lambda: ss.orthogonalize(_claim(4, 5), out=_claim(5, 4)),
        lambda: ss.orthogonalize([_claim(4, 5)] * 2, out=[_claim(4, 5)]),
        lambda: ss.orthogonalize([_claim(4, 5)] * 2, out=[_claim(4, 5), _claim(4, 5, dtype=half)]),
        lambda: ss.TensorMuon([], ss.Muon()), lambda: ss.TensorMuon([_claim(4, 5)], ss.Muon()),
        lambda: ss.TensorMuon([_claim(20, dtype=half)], ss.Muon()),
        lambda: ss.TensorMuon([_claim(4, 5, dtype=half)], []),
        lambda: ss.TensorMuon([_claim(4, 5, dtype=half)], [ss.Muon()] * 9),
        lambda: ss.TensorMuon([_claim(4, 5, dtype=half)], ss.Muon(), groups=[1]),
        lambda: ss.TensorMuon([_claim(4, 5, dtype=half)], ss.Muon(), groups=[0, 0]),
    ]
    for k, call in enumerate(bad):
        with pytest.raises((ValueError, TypeError)):
            call()
            pytest.fail(f"case {k} was taken")


def test_muon_list_checks(wrappers):
    params = [_claim(4, 6, dtype=torch.bfloat16) for _ in range(2)]
    opt = ss.TensorMuon(params, [ss.Muon(), ss.Muon()])
    opt.master, opt.m = (t.as_subclass(_Claimed) for t in (opt.master, opt.m))
    grads = [_claim(4, 6) for _ in range(2)]
    lst = ss.TensorList(grads)
    opt._call(lst)
    opt._call(lst)
    with pytest.raises(ValueError):
        opt._call(grads[:1])
    with pytest.raises(ValueError):
        opt._call([_claim(4, 6), _claim(4, 7)])
    with pytest.raises(ValueError):
        opt.step(lst, skip=torch.zeros(1, dtype=torch.int64))
    with pytest.raises(ValueError):
        opt.step(lst, grad_coef=torch.zeros(1))
    grads[0].data = torch.zeros(5, 6)
    with pytest.raises(ValueError):
        opt._call(lst)
    grads[0].data = torch.zeros(4, 6)
    params[1].data = torch.zeros(6, 4, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        opt._call(grads)
    params[1].data = torch.zeros(4, 6, dtype=torch.float16)
    with pytest.raises(ValueError):
        opt._call(grads)
    params[1].data = torch.zeros(4, 6, dtype=torch.bfloat16)
    opt.groups[1] = 1
    opt._call(grads)
    assert [r.group for r in opt._table] == [0, 1]
    opt.groups[1] = 2
    with pytest.raises(ValueError):
        opt._call(grads)
    opt.groups[1] = 0
    opt.m = opt.m[:5]
    with pytest.raises(ValueError):
        opt._call(grads)


def test_muon_refuses_gradients_of_another_shape(wrappers):
    """As many elements are not enough: the update sees rows and columns."""
    opt = ss.TensorMuon([_claim(4, 6, dtype=torch.bfloat16)], ss.Muon())
    opt.master, opt.m = (t.as_subclass(_Claimed) for t in (opt.master, opt.m))
    opt._call([_claim(4, 6)])
    opt._call([_claim(24)])                       # a bucket's piece
    for shape in ((6, 4), (2, 12), (1, 4, 6)):
        with pytest.raises(ValueError):
            opt._call([_claim(*shape)])
        with pytest.raises(ValueError):
            opt._call(ss.TensorList([_claim(*shape)]))
