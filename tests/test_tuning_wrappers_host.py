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
