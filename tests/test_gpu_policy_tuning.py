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
