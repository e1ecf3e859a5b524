"""What is on another device than the tensors is refused before anything is allocated or
launched: a caller's workspace, whether it holds a buffer yet or not, and the words,
buffers and parameters of a step.  No GPU: tensors that claim to be on one, and a library
that must not be reached."""
import contextlib

import pytest
import torch

import sharded_optimizer_step_gb300 as ss
from sharded_optimizer_step_gb300 import _capi

KINDS = (ss.EmbeddingWorkspace, ss.LayerNormWorkspace, ss.MatrixWorkspace)


class _Buffer:
    def __init__(self, device, nbytes):
        self.device, self.nbytes = torch.device(device), nbytes

    def numel(self):
        return self.nbytes


class _OnGpu(torch.Tensor):
    is_cuda = True
    device = torch.device("cuda:0")


def _claim(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(_OnGpu)


@pytest.fixture(autouse=True)
def _no_gpu(monkeypatch):
    class Never:
        def __getattr__(self, name):
            if name.endswith("workspace_bytes"):
                return lambda *a: 64
            raise AssertionError(f"{name} was reached")

    def at_least(self, nbytes):
        made.append(torch.device(self.device))
        return 4096, nbytes
    made = []
    ss._load_torch()
    monkeypatch.setattr(_capi, "lib", lambda: Never())
    monkeypatch.setattr(ss, "_here", lambda device, stream: contextlib.nullcontext())
    monkeypatch.setattr(ss, "_elsewhere", lambda device, stream: False)
    monkeypatch.setattr(ss._Scratch, "at_least", at_least)
    return made


@pytest.mark.parametrize("kind", KINDS)
def test_only_the_tensors_device(kind, _no_gpu):
    dev = torch.device("cuda:1")
    for where in ("cuda:0", "cpu", torch.device("cuda", 2), 0):
        with pytest.raises(ValueError):
            ss._scratch(kind(where), kind, dev, 64)
        held = kind("cuda")
        held.buf = _Buffer(torch.device(where), 1 << 20)
        with pytest.raises(ValueError):
            ss._scratch(held, kind, dev, 64)
    assert not _no_gpu                                     # nothing was allocated
    for where in ("cuda", "cuda:1", dev, 1):
        assert ss._scratch(kind(where), kind, dev, 64)[:2] == (4096, 64)
    held = kind("cuda")                                    # made while cuda:1 was current
    held.buf = _Buffer(dev, 1 << 20)
    assert ss._scratch(held, kind, dev, 64)[2] is held
    assert ss._scratch(None, kind, dev, 64)[2].device == dev


def test_every_call_that_takes_one():
    x, mean = _claim(5, 8), _claim(5)
    ids = _claim(5, dtype=torch.int64)
    calls = [
        lambda: ss.embedding_grad(x, ids, _claim(9, 8), workspace=ss.EmbeddingWorkspace("cuda:1")),
        lambda: ss.layer_norm_grad(x, x, mean, mean, d_weight=_claim(8),
                                   workspace=ss.LayerNormWorkspace("cuda:1")),
        lambda: ss.orthogonalize(x, out=_claim(5, 8), workspace=ss.MatrixWorkspace("cuda:1")),
    ]
    for call in calls:
        with pytest.raises(ValueError, match="another device"):
            call()


class _OnAnother(torch.Tensor):
    is_cuda = True
    device = torch.device("cuda:1")


def _other(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(_OnAnother)


@pytest.fixture
def muon(monkeypatch):
    made = torch.zeros                                     # the state, where the parameters are
    monkeypatch.setattr(torch, "zeros", lambda *a, device=None, **k: made(*a, **k).as_subclass(
        _OnGpu) if device is not None else made(*a, **k))
    opt = ss.TensorMuon([_claim(4, 6, dtype=torch.bfloat16) for _ in range(2)], ss.Muon())
    monkeypatch.undo()
    return opt


def test_a_steps_words_and_buffers(muon, monkeypatch):
    class Never:
        def __getattr__(self, name):
            raise AssertionError(f"{name} was reached")
    monkeypatch.setattr(_capi, "lib", lambda: Never())
    monkeypatch.setattr(ss, "_here", lambda device, stream: contextlib.nullcontext())
    monkeypatch.setattr(ss._Scratch, "at_least", lambda self, nbytes: (4096, nbytes))
    grads = [_claim(4, 6) for _ in range(2)]
    with pytest.raises(AssertionError, match="was reached"):
        muon.step(grads, grad_coef=_claim(1), skip=_claim(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="different devices"):
        muon.step(grads, grad_coef=_other(1))
    with pytest.raises(ValueError, match="different devices"):
        muon.step(grads, skip=_other(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        muon.step([_other(4, 6) for _ in range(2)])
    for what in ("m", "params"):
        was = getattr(muon, what)
        setattr(muon, what, _other(muon.flat) if what == "m" else
                [was[0], _other(4, 6, dtype=torch.bfloat16)])
        with pytest.raises(ValueError, match="different devices"):
            muon.step(grads)
        setattr(muon, what, was)


@pytest.mark.parametrize("held", [False, True])
def test_losses_and_the_norm(held, monkeypatch):
    monkeypatch.setattr(ss, "_LOSS_HEAD", [64])
    monkeypatch.setattr(ss, "_on", lambda stream, device: contextlib.nullcontext())
    monkeypatch.setattr(ss.LossWorkspace, "at_least", lambda self, n, pairs: (4096, 64, None))
    x, f, ids = _claim(6, 9), _claim(6), _claim(6, dtype=torch.int64)
    plain = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **k: plain(*a, **k))

    def spaces(where):
        loss, norm = ss.LossWorkspace(where), object.__new__(ss.NormWorkspace)
        norm.buf = torch.zeros(8)
        norm.buf = (_other if torch.device(where).index == 1 else _claim)(8)
        if held:
            loss.buf = _Buffer(where, 1 << 20)
        return loss, norm

    def calls(loss, norm):
        yield lambda: ss.policy_loss(x, ids, f, f, workspace=loss, stream=0)
        yield lambda: ss.preference_loss(x, ids, [6, 0], f, workspace=loss, stream=0)
        yield lambda: ss.grad_norm_clip([x], 1.0, out=_claim(2), workspace=norm, stream=0)
    for call in calls(*spaces("cuda:1")):
        with pytest.raises(ValueError, match="another device"):
            call()
    for call in calls(*spaces("cuda:0")):
        with pytest.raises(AssertionError, match="was reached"):
            call()
