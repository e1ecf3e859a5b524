"""Optimizers over parameters that require gradients: their master copies are no part of
the parameters' graph (which would hold the leaves' accumulation nodes, made on the
stream of that moment, for as long as the optimizer lives).  No GPU: tensors that claim
to be on one."""
import contextlib

import pytest
import torch

import sharded_optimizer_step_gb300 as ss
from sharded_optimizer_step_gb300 import _capi


class _Claimed(torch.Tensor):
    is_cuda = True


@pytest.fixture(autouse=True)
def _no_gpu(monkeypatch):
    class Never:
        def __getattr__(self, name):
            if name.endswith("workspace_bytes"):
                return lambda *a: 64
            raise AssertionError(f"{name} was reached")
    monkeypatch.setattr(_capi, "lib", lambda: Never())
    monkeypatch.setattr(ss, "_here", lambda device, stream: contextlib.nullcontext())


@pytest.mark.parametrize("make", [
    lambda p: ss.TensorMuon(p, ss.Muon()), lambda p: ss.TensorAdamW(p, ss.AdamW()),
    lambda p: ss.TensorAdamW(p, ss.AdamW(), state_bits=8)])
def test_masters_hold_no_graph(make):
    params = [torch.randn(4, 6).bfloat16().as_subclass(_Claimed).requires_grad_()
              for _ in range(2)]
    opt = make(params)
    assert not opt.master.requires_grad and opt.master.grad_fn is None
    for k, p in enumerate(params):
        assert p.is_leaf and p.requires_grad
        assert torch.equal(opt.view(opt.master, k), p.detach().float())
