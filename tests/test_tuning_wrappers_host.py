"""Checks of the tuning operators' Python wrappers on tensors that only claim to
be on a GPU: what is refused here is refused before the library is called, which
no case below reaches."""
import pytest
import torch

import sharded_optimizer_step_gb300 as ss
from sharded_optimizer_step_gb300 import _capi


class _Claimed(torch.Tensor):
    is_cuda = True


def _claim(t):
    return t.as_subclass(_Claimed)


@pytest.fixture(autouse=True)
def no_library(monkeypatch):
    """Nothing here may get as far as a call into the library."""
    class Never:
        def __getattr__(self, name):
            raise AssertionError(f"{name} was reached")
    monkeypatch.setattr(_capi, "lib", lambda: Never())
    monkeypatch.setattr(ss, "_LOSS_HEAD", [64])


def _losses(x, grad=None):
    n = x.shape[0]
    ids, f = _claim(torch.zeros(n, dtype=torch.int64)), _claim(torch.zeros(n))
    yield lambda: ss.policy_loss(x, ids, f, f, grad=grad, stream=0)
    yield lambda: ss.preference_loss(x, ids, [n, 0], f, grad=grad, stream=0)


@pytest.fixture
def no_stream(monkeypatch):
    import contextlib
    monkeypatch.setattr(ss, "_on", lambda stream, device: contextlib.nullcontext())


@pytest.mark.parametrize("v", [1, 2, 5])
def test_rows_that_share_memory_are_refused(v, no_stream):
    """Rows that are one row seen many times (an expanded tensor) have no storage
    for the rows that the kernels would step over, whatever the vocabulary."""
    one, rows = _claim(torch.zeros(1, v)), _claim(torch.zeros(6, v))
    for call in _losses(one.expand(6, v)):
        with pytest.raises(ValueError, match="rows"):
            call()
    for call in _losses(rows, grad=one.expand(6, v)):
        with pytest.raises(ValueError, match="rows"):
            call()


def test_rows_apart_are_taken(no_stream):
    """The same calls with rows of their own get as far as the library."""
    for x in (torch.zeros(6, 1), torch.zeros(1, 6).t(), torch.zeros(6, 9)[:, 2:3],
              torch.zeros(6, 9)[:, :4], torch.zeros(2, 3)[:1].expand(1, 3)):
        for call in _losses(_claim(x), grad=_claim(torch.zeros(x.shape))):
            with pytest.raises(AssertionError, match="was reached"):
                call()


# ------------------------------------------------------ lists of tensors

def _kept(bits=8, n=3):
    """An optimizer and a list as a program keeps them, after a first call."""
    params = [_claim(torch.zeros(4, 6, dtype=torch.bfloat16)) for _ in range(n)]
    grads = [_claim(torch.zeros(4, 6, dtype=torch.bfloat16)) for _ in range(n)]
    opt = ss.TensorAdamW(params, [ss.AdamW(), ss.AdamW(lr=1e-4)], state_bits=bits)
    for name in ("master", "m", "v") + (("m_scale", "v_scale") if bits == 8 else ()):
        setattr(opt, name, _claim(getattr(opt, name)))
    lst = ss.TensorList(grads)
    opt._call(lst)
    return opt, params, lst, grads


CHANGES = {
    "shorter": lambda t: t[:2],
    "another type of the same size": lambda t: t.view(torch.float16),
    "a wider type": lambda t: t.view(torch.float32),
    "transposed": lambda t: t.t(),
}


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("change", list(CHANGES))
def test_a_parameter_changed_at_its_address_is_refused(change, bits):
    opt, params, lst, _ = _kept(bits)
    at = params[1].data_ptr()
    params[1].data = CHANGES[change](params[1].data)
    assert params[1].data_ptr() == at
    for grads in (lst, lst.tensors):
        with pytest.raises(ValueError):
            opt.step(grads)
    assert opt.t == 0


@pytest.mark.parametrize("change", list(CHANGES))
def test_a_gradient_changed_at_its_address_is_refused(change):
    opt, _, lst, grads = _kept()
    grads[1].data = CHANGES[change](grads[1].data)
    with pytest.raises(ValueError):
        opt.step(lst)
    if change == "shorter":        # the others are the same bytes, the norm's type is the list's
        with pytest.raises(ValueError):
            ss.grad_norm_clip(lst, 1.0)


@pytest.mark.parametrize("name,change", [("master", lambda t: t[:-1]), ("m", lambda t: t[:-256]),
                                         ("v", lambda t: t.view(torch.int8)),
                                         ("m_scale", lambda t: t[:1]),
                                         ("v_scale", lambda t: t.view(torch.int32))])
def test_a_state_buffer_changed_at_its_address_is_refused(name, change):
    opt, _, lst, _ = _kept()
    setattr(opt, name, change(getattr(opt, name)))
    with pytest.raises(ValueError):
        opt.step(lst)


def test_groups_given_later_are_taken_and_checked():
    opt, _, lst, _ = _kept()
    opt.groups = [0, 1, 1]
    opt._call(lst)
    assert [row.group for row in opt._table] == [0, 1, 1]
    opt.groups[0] = 1
    opt._call(lst)
    assert [row.group for row in opt._table] == [1, 1, 1]
    for bad in ([0, 1], [0, 1, 2], [0, -1, 0]):
        opt.groups = bad
        with pytest.raises(ValueError):
            opt.step(lst)


def test_an_unchanged_list_reaches_the_library():
    opt, _, lst, _ = _kept()
    for _ in range(2):
        with pytest.raises(AssertionError, match="tensors_adamw_step was reached"):
            opt.step(lst)
