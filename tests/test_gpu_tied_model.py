"""Embedding, layer norm, policy loss, their gradients, the norm and both steps
together, as examples/tied_model_tuning.py runs them: the gradients against
torch's autograd in float64, steps that repeat to the bit, a step captured in a
graph, and two programs beside each other on two streams."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import sharded_optimizer_step_gb300 as ss
from oracle import model_ops as OM

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ss.build()
    spec = importlib.util.spec_from_file_location(
        "tied_model_tuning", os.path.join(ROOT, "examples", "tied_model_tuning.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    yield m
    assert ss.device_status() == 0


def test_gradients_against_autograd(example):
    """In fp32: sums of up to 700 terms (the vocabulary) and 96 tokens in fp32, a chain
    of seven operations, so an element is off by a few 700 2^-24 = 4e-5 of the terms'
    sizes at the worst; in norm, with signs at random, sqrt(700) 2^-24 an operation,
    1e-5 for all."""
    gen = torch.Generator(device=DEV).manual_seed(3)
    p = example.parameters(700, 40, gen, dtype=torch.float32, device=DEV)
    p["norm_w"].add_(torch.randn(40, generator=gen, device=DEV) * 0.2)
    p["norm_b"].add_(torch.randn(40, generator=gen, device=DEV) * 0.2)
    n = 96
    prev = torch.randint(0, 700, (n,), generator=gen, device=DEV)
    prev[5], prev[50:60] = -1, 17
    ids = torch.randint(0, 700, (n,), generator=gen, device=DEV)
    adv = torch.randn(n, generator=gen, device=DEV)
    w = (torch.rand(n, generator=gen, device=DEV) > 0.2).float()
    logits, kept = example.forward(p, prev)
    old = torch.log_softmax(logits, 1).gather(1, ids[:, None])[:, 0].contiguous()
    out = ss.policy_loss(logits, ids, old, adv, weights=w, grad=logits)
    grads = {k: torch.empty_like(v) for k, v in p.items()}
    spaces = (ss.LayerNormWorkspace(DEV), ss.EmbeddingWorkspace(DEV))
    example.backward(p, prev, kept, logits, grads, spaces)

    q = {k: v.double().requires_grad_() for k, v in p.items()}
    live = (prev >= 0).double()[:, None]
    h = q["table"][prev.clamp(min=0)] * live * 40 ** 0.5
    y = torch.nn.functional.layer_norm(h, (40,), q["norm_w"], q["norm_b"], 1e-5)
    r = h + torch.tanh(y @ q["up"].T) @ q["down"].T
    lp = torch.log_softmax(r @ q["table"].T, 1).gather(1, ids[:, None])[:, 0]
    u = torch.exp(lp - old.double())
    loss = -(w * torch.minimum(u * adv, u.clamp(0.8, 1.2) * adv)).sum() / w.sum()
    loss.backward()
    assert abs(float(out.stats[0]) - float(loss.detach())) < 1e-5
    for k in example.NAMES:
        want = q[k].grad
        assert float((grads[k].double() - want).norm()) < 1e-5 * float(want.norm()), k
    # once more, added to the vectors' and the table's gradients
    before = {k: grads[k].clone() for k in example.NAMES}
    example.backward(p, prev, kept, logits, grads, spaces, accumulate=True)
    for k in example.NAMES:
        assert float((grads[k] - 2 * before[k]).norm()) < 1e-5 * float(before[k].norm()), k


def test_steps_repeat_to_the_bit(example):
    first = example.tune(steps=4)
    assert all(np.isfinite(v).all() for v in first)
    assert first == example.tune(steps=4)


def test_operators_against_the_oracle():
    r = np.random.default_rng(7)
    table, ids = r.normal(size=(50, 24)).astype(np.float32), r.integers(-2, 52, 200)
    d = r.normal(size=(200, 24)).astype(np.float32)
    t, i, g = (torch.from_numpy(v).to(DEV) for v in (table, ids, d))
    near = lambda a, b, tol: np.abs(a.cpu().double().numpy() - b).max() <= tol  # noqa: E731
    # one product; sums of at most some ten terms below 5; rows of 24
    assert near(ss.embedding(t, i, scale=1.5), OM.embedding(table, ids, 1.5), 8 * 2.0 ** -24)
    assert near(ss.embedding_grad(g, i, torch.empty(50, 24, device=DEV), scale=1.5),
                OM.embedding_grad(d, ids, 50, 1.5), 50 * 15 * 2.0 ** -24)
    w, b = (r.normal(size=24).astype(np.float32) for _ in range(2))
    y = ss.layer_norm(g, *(torch.from_numpy(v).to(DEV) for v in (w, b)))
    out, mean, rstd = OM.layer_norm(d, w, b)
    assert near(y.out, out, 1e-5) and near(y.mean, mean, 1e-6) and near(y.rstd, rstd, 1e-5)
    p = r.normal(size=(40, 70)).astype(np.float32)
    params = [torch.from_numpy(p).to(DEV).bfloat16()]
    start = params[0].float().cpu().double().numpy()
    opt = ss.TensorMuon(params, ss.Muon(lr=0.01, weight_decay=0.1))
    u = r.normal(size=(40, 70)).astype(np.float32)
    opt.step([torch.from_numpy(u).to(DEV)])
    want, m = OM.muon_step(start, np.zeros((40, 70)), u, 0.01, 0.95, 0.1, 0.2)
    # the update's elements are off by 1e-4 of 0.01 * 0.2 sqrt(70) at most, p by 3 2^-24
    assert near(opt.view(opt.master, 0), want, 2e-6 + 3 * 4 * 2.0 ** -24)
    assert near(opt.view(opt.m, 0), m, 2.0 ** -23)


def _program(stream, shapes, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    params = [torch.randn(*s, generator=g, device=DEV).bfloat16() for s in shapes]
    grads = [torch.randn(*s, generator=g, device=DEV) for s in shapes]
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        opt = ss.TensorMuon(params, ss.Muon(lr=0.01))
        lst = ss.TensorList(grads)
    return opt, lst, stream


def test_two_steps_at_once():
    """Each of the two wants all SMs for blocks that wait for one another: whichever
    comes first runs, the other follows, and both are right."""
    shapes = [[(600, 900), (300, 2000)], [(1100, 700), (64, 64), (700, 1500)]]
    alone = []
    for k, s in enumerate(shapes):
        opt, lst, _ = _program(torch.cuda.current_stream(), s, k)
        for _ in range(6):
            opt.step(lst)
        torch.cuda.synchronize()
        alone.append(opt.master.clone())
    both = [_program(torch.cuda.Stream(), s, k) for k, s in enumerate(shapes)]
    for _ in range(6):
        for opt, lst, stream in both:
            with torch.cuda.stream(stream):
                opt.step(lst)
    torch.cuda.synchronize()
    assert all(torch.equal(b[0].master, a) for b, a in zip(both, alone))
    assert ss.device_status() == 0


def test_a_step_in_a_graph(example):
    """Loss to steps captured once and replayed twice: the same bits as eager calls."""
    def program():
        gen = torch.Generator(device=DEV).manual_seed(11)
        p = example.parameters(500, 64, gen, device=DEV)
        grads = {k: torch.zeros_like(v) for k, v in p.items()}
        muon = ss.TensorMuon([p["up"], p["down"]], ss.Muon(lr=2e-3))
        adamw = ss.TensorAdamW([p[k] for k in example.NAMES[:3]], ss.AdamW(lr=1e-3))
        adamw.device_step_state()
        lists = [ss.TensorList([grads[k] for k in names])
                 for names in (example.NAMES, ("up", "down"), example.NAMES[:3])]
        loss_ws, norm_ws = ss.LossWorkspace(DEV), ss.NormWorkspace(DEV)
        spaces = (ss.LayerNormWorkspace(DEV), ss.EmbeddingWorkspace(DEV))
        prev = torch.randint(0, 500, (128,), generator=gen, device=DEV)
        ids = torch.randint(0, 500, (128,), generator=gen, device=DEV)
        adv, old = torch.randn(128, generator=gen, device=DEV), torch.full((128,), -6.0, device=DEV)

        def step():
            logits, kept = example.forward(p, prev)
            ss.policy_loss(logits, ids, old, adv, grad=logits, workspace=loss_ws)
            example.backward(p, prev, kept, logits, grads, spaces)
            clip = ss.grad_norm_clip(lists[0], 1.0, workspace=norm_ws)
            muon.step(lists[1], grad_coef=clip[1:])
            adamw.step(lists[2], grad_coef=clip[1:])
        return step, p
    eager, p = program()
    for _ in range(3):
        eager()
    captured, q = program()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        captured()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p[k], q[k]) for k in p)


def test_layer_norm_waits_that_run_out_are_reported():
    g = torch.Generator(device=DEV).manual_seed(2)
    x = torch.randn(5000, 2048, generator=g, device=DEV).bfloat16()
    d = torch.randn(5000, 2048, generator=g, device=DEV).bfloat16()
    y = ss.layer_norm(x)
    want = ss.layer_norm_grad(d, x, y.mean, y.rstd).d_x
    torch.cuda.synchronize()
    before, st = ss.set_tma_wait_ns(1), 0
    try:
        for _ in range(20):
            ss.layer_norm_grad(d, x, y.mean, y.rstd)
            torch.cuda.synchronize()
            st |= ss.device_status(clear=True)
            if st & 3:
                break
    finally:
        ss.set_tma_wait_ns(before)
    assert st & 3 and not st & 4
    assert torch.equal(ss.layer_norm_grad(d, x, y.mean, y.rstd).d_x, want)
    torch.cuda.synchronize()
    assert ss.device_status() == 0
