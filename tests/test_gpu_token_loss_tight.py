"""The token losses on wide rows, several to a block, each log probability and each
gradient element held to its own size in 64 bits (tests/_token_check.py, which
test_token_check_host.py tries planted mistakes on).  Rows are noise, confident, or
hold their mass at another token, in turn; a fifth is masked."""
import pytest
import torch

import _token_check as TC
import sharded_optimizer_step_gb300 as ss

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ss.build()
    yield
    assert ss.device_status() == 0


def _case(n, v, dt, seed, stride=None):
    g = torch.Generator(device=DEV).manual_seed(seed)
    buf = torch.full((n, stride or v), float("nan"), dtype=DT[dt], device=DEV)
    x, rows = buf[:, :v], torch.arange(n, device=DEV)
    for i in range(0, n, 256):
        j = min(n, i + 256)
        x[i:j] = (torch.randn(j - i, v, device=DEV, generator=g) * 2).to(DT[dt])
    ids = torch.randint(0, v, (n,), device=DEV, generator=g)
    x[rows, ids] += torch.tensor([3.0, 14.0, 0.0], device=DEV)[rows % 3].to(DT[dt])
    other = (ids + 1 + torch.randint(0, v - 1, (n,), device=DEV, generator=g)) % v
    x[rows, other] += torch.tensor([0.0, 0.0, 18.0], device=DEV)[rows % 3].to(DT[dt])
    a, t = TC.row_facts(x, ids)
    near = lambda s: (a + s * torch.randn(n, device=DEV, generator=g)).float()  # noqa: E731
    old = near(0.25)
    # off the clip's two edges
    for edge in (0.8, 1.2):
        old = torch.where((torch.exp(a - old) - edge).abs() < 1e-3, old - 5e-3, old)
    w = torch.tensor([1.0, 0.5, 2.0, 1.0, 0.0], device=DEV)[(rows * 7) % 5]
    return dict(x=x, ids=ids, a=a, t=t, old=old.float(), ref=near(0.2), w=w,
                adv=torch.randn(n, device=DEV, generator=g))


def _check(c, out, stats, errors, slope, slack, live):
    t, a = c["t"], c["a"]
    off = (out.logps.double() - a).abs()
    assert (off <= t + 2.0 ** -24 * a.abs())[live].all(), float((off / t)[live].max())
    assert not out.logps[~live].any()
    got = out.stats.double()
    assert ((got - stats).abs() <= errors + 1e-12).all(), (got, stats, errors)
    if out.grad is not None:
        misses = TC.gradient_misses(out.grad[live], c["given"][live], c["ids"][live], slope[live],
                                    slack[live], t[live])
        assert not misses.any(), (live.nonzero()[misses.nonzero()[:4, 0], 0], misses.max())
        assert not out.grad[~live].any()


def _policy(c, grad, kl=0.05, scale=256.0):
    word = torch.tensor([scale], device=DEV)
    out = ss.policy_loss(c["x"], c["ids"], c["old"], c["adv"], ref_logps=c["ref"], kl_coef=kl,
                         weights=c["w"], grad=grad, loss_scale=word)
    d = lambda k: c[k].double()  # noqa: E731
    facts = TC.policy(c["a"], c["t"], d("old"), d("adv"), d("ref"), d("w"), kl,
                      float(c["w"].double().sum()), scale)
    _check(c, out, *facts, c["w"] != 0)
    return out


def _preference(c, lens, grad, beta=0.2, smoothing=0.1, scale=256.0):
    word = torch.tensor([scale], device=DEV)
    out = ss.preference_loss(c["x"], c["ids"], lens, c["ref"], beta=beta, weights=c["w"],
                             label_smoothing=smoothing, grad=grad, loss_scale=word)
    stats, errors, r, roff, slope, slack = TC.preference(
        c["a"], c["t"], lens, c["ref"].double(), c["w"].double(), beta, smoothing, len(lens) / 2,
        scale)
    assert ((out.log_ratios.double() - r).abs() <= roff).all()
    _check(c, out._replace(stats=out.stats[:3]), stats, errors, slope, slack, c["w"] != 0)
    return out


def _lens(n):
    cut = [n // 5, n // 7, 0, n // 3, n // 11]
    return cut + [n - sum(cut)]


@pytest.mark.parametrize("shift", [0, 3], ids=["staged", "other_offsets"])
@pytest.mark.parametrize("n,v,dt,stride", [
    (640, 50257, "bf16", None), (640, 50257, "f32", 50304), (640, 32000, "f16", None),
    (500, 32000, "f32", None), (400, 128256, "bf16", None), (330, 60001, "f32", None),
    (310, 128256, "f16", 128257), (5, 300007, "f16", None), (1300, 4099, "bf16", None),
    (1000, 515, "f32", 517), (3, 32000, "bf16", None)])
def test_wide_rows(n, v, dt, stride, shift):
    c = _case(n, v, dt, n + v, stride)
    c["given"] = c["x"]
    g = torch.full((n * (stride or v) + 8,), 7.0, dtype=DT[dt], device=DEV)
    g = g[shift:shift + n * (stride or v)].view(n, stride or v)[:, :v]
    _policy(c, g)
    _preference(c, _lens(n), g)
    if shift == 0:
        _policy(c, None)
        _preference(c, _lens(n), None)
        c["given"] = c["x"].clone()          # in place
        _policy(c, c["x"])
        c["x"].copy_(c["given"])
        _preference(c, _lens(n), c["x"])


def test_rows_past_2_31_elements():
    """70000 rows of 32000 in place: rows at both ends and on either side of the 2^31st
    element, each element of their gradients."""
    n, v = 70000, 32000
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GB")
    g = torch.Generator(device=DEV).manual_seed(5)
    x = torch.empty(n, v, dtype=torch.bfloat16, device=DEV)
    for a in range(0, n, 5000):
        x[a:a + 5000].normal_(0, 2, generator=g)
    ids = torch.randint(0, v, (n,), generator=g, device=DEV)
    adv = torch.randn(n, generator=g, device=DEV)
    pick = torch.tensor([0, 1, 151, 152, 33333, 67107, 67108, 67109, n - 2, n - 1], device=DEV)
    given = x[pick].clone()
    a, t = TC.row_facts(given, ids[pick])
    old = torch.full((n,), -12.0, device=DEV)
    old[pick] = (a + 0.05).float()
    out = ss.policy_loss(x, ids, old, adv, grad=x)
    one = torch.ones(len(pick), dtype=torch.float64, device=DEV)
    _, _, c, slack = TC.policy(a, t, old[pick].double(), adv[pick].double(), old[pick].double(), one,
                               0.0, float(n))
    off = (out.logps[pick].double() - a).abs()
    assert (off <= t + 2.0 ** -24 * a.abs()).all()
    assert not TC.gradient_misses(x[pick], given, ids[pick], c, slack, t).any()
