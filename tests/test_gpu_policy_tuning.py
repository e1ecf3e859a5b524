"""The tuning operators together, as examples/policy_tuning.py runs them: the
rewarded tokens become likelier, with 8-bit moments as with 32-bit ones, and
two runs from one seed agree.

Also the staged losses' wait limit: a wait that is made to run out sets the
status word and the launch ends."""
import importlib.util
import os

import pytest
import torch

import sharded_optimizer_step_gb300 as ss

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def tune():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ss.build()
    spec = importlib.util.spec_from_file_location(
        "policy_tuning", os.path.join(ROOT, "examples", "policy_tuning.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m.tune


@pytest.mark.parametrize("bits", [8, 32])
def test_rewarded_tokens_become_likelier(tune, bits):
    rewards, losses = tune(steps=15, state_bits=bits)
    assert abs(rewards[0] - 1 / 7) < 0.05         # a policy that knows nothing yet
    assert rewards[-1] > 0.5
    assert all(x == x for x in losses)


def test_the_loop_is_deterministic(tune):
    assert tune(steps=3) == tune(steps=3)


def test_a_wait_that_runs_out_is_reported():
    """With a limit of 1 ns the waits for the first copies run out before they
    can land (at the clock's next tick: so several launches are tried): the
    launch ends, the status word says so, and after the limit is back the
    operator is right again."""
    n = 3000
    x = torch.randn(n, 32000, device="cuda").bfloat16()
    ids = torch.randint(0, 32000, (n,), device="cuda")
    z = torch.full((n,), -10.0, device="cuda")
    g = torch.empty_like(x)
    want = ss.policy_loss(x, ids, z, z, grad=g).logps.clone()
    assert ss.device_status(clear=True) == 0
    prev = ss.set_tma_wait_ns(1)
    try:
        for kw in ({"grad": g}, {}):
            st = 0
            for _ in range(20):
                ss.policy_loss(x, ids, z, z, **kw)
                torch.cuda.synchronize()
                st |= ss.device_status(clear=True)
                if st & 3:
                    break
            assert st & 3 and not st & 4
    finally:
        ss.set_tma_wait_ns(prev)
    assert torch.equal(ss.policy_loss(x, ids, z, z, grad=g).logps, want)
    torch.cuda.synchronize()
    assert ss.device_status() == 0


@pytest.mark.parametrize("form", ["stream", "handle"])
def test_a_stream_of_its_own_while_the_current_one_is_busy(form):
    """Calls given `stream` allocate, fill and zero on it: nothing that they need is
    left to the current stream, which is busy."""
    n, v = 300, 1000
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(n, v, device="cuda", generator=g).bfloat16()
    ids = torch.randint(0, v, (n,), device="cuda", generator=g)
    z = torch.full((n,), -7.0, device="cuda")
    adv = torch.randn(n, device="cuda", generator=g)
    w = (torch.rand(n, device="cuda", generator=g) < 0.7).float()
    params = [torch.randn(k, device="cuda", generator=g).bfloat16() for k in (5000, 300)]
    grads = [torch.randn(k, device="cuda", generator=g).bfloat16() for k in (5000, 300)]

    def run(stream, side):
        d1, d2 = torch.empty_like(x), torch.empty_like(x)
        p = [q.clone() for q in params]
        torch.cuda.synchronize()
        if stream is not None:
            torch.cuda._sleep(int(2e8))          # about 0.1 s of the current stream
        a = ss.policy_loss(x, ids, z, adv, weights=w, grad=d1, stream=stream)
        b = ss.preference_loss(x, ids, [100, 50, 70, 80], z, weights=w, grad=d2, stream=stream)
        c = ss.grad_norm_clip(grads, 1.0, stream=stream)
        opt = ss.TensorAdamW(p, ss.AdamW(), state_bits=8, stream=stream)
        opt.step(grads, grad_coef=c[1:], stream=stream)
        m = opt.moments(stream=stream)
        with torch.cuda.stream(side):
            out = [t.cpu() for t in (a.stats, a.logps, d1, b.stats, b.log_ratios, d2, c, *m, *p)]
        torch.cuda.synchronize()
        return out

    want = run(None, torch.cuda.current_stream())
    side = torch.cuda.Stream()
    # memory that is not zero where a workspace may land
    junk = [torch.full((k,), -1, dtype=torch.int64, device="cuda") for k in (1 << 12, 1 << 14, 1 << 16)]
    torch.cuda.synchronize()
    del junk
    got = run(side if form == "stream" else side.cuda_stream, side)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
