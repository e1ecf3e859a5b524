"""AdamW over a list of tensors (32- and 8-bit moments) and the gradient norm
on the GPU against the oracle.  The step is elementwise fp32 with one rounding
per operation and codes fixed by it, so state and codes match bit for bit; the
norm is held to its rounding (2^-24 per addition of a thread's chain, joined
in double)."""
import numpy as np
import pytest
import torch

import oracle
import sharded_optimizer_step_gb300 as ss
from oracle import tensors as OT
from oracle.numerics import AdamWConfig

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


def _same(got, want, what=""):
    got = got.cpu().numpy() if torch.is_tensor(got) else got
    assert got.dtype == want.dtype and got.shape == want.shape, what
    same = (got == want) | ((got != got) & (want != want))
    assert same.all(), (what, np.argwhere(~same)[:5], got[~same][:5], want[~same][:5])


LISTS = {
    "one": [1], "small": [3, 0, 255, 256, 257, 1, 511],
    "mixed": [768, 100_003, 0, 2048, 2047, 2049, 4096 * 7 + 5, 8],
    "many": [(i * 37) % 900 + 1 for i in range(450)],
}


def _make(numels, dt, seed, shift=0):
    r = np.random.default_rng(seed)
    params = [torch.from_numpy(r.normal(size=n).astype(np.float32) * 0.02).to(DEV)
              .to(torch.bfloat16) for n in numels]
    grads = []
    for n in numels:
        b = torch.full((n + 64,), float("nan"), dtype=DT[dt], device=DEV)
        g = b[shift:shift + n]
        g.copy_(torch.from_numpy(r.normal(size=n) * np.exp(r.normal(size=n)) * 1e-3))
        grads.append(g)
    return params, grads


class _Oracle:
    def __init__(self, params, bits, hps, groups):
        self.p = [p.float().cpu().numpy().ravel() for p in params]
        self.bits, self.hps, self.groups = bits, hps, groups
        z, b = np.zeros, OT.BLOCK
        self.s = [([z(len(p), np.uint8), z(-(-len(p) // b), np.float32),
                    z(len(p), np.uint8), z(-(-len(p) // b), np.float32)] if bits == 8 else
                   [z(len(p), np.float32), z(len(p), np.float32)]) for p in self.p]

    def step(self, grads, t, coef=None):
        for i, g in enumerate(grads):
            g = g.float().cpu().numpy().ravel()
            if coef is not None:
                g = g * np.float32(coef)
            if not len(g):
                continue
            hp = self.hps[self.groups[i]]
            if self.bits == 8:
                self.p[i], *self.s[i] = OT.adamw8(g, self.p[i], *self.s[i], hp, t)
            else:
                self.p[i], *self.s[i] = oracle.adamw(self.p[i], *self.s[i], g, hp, t)[:3]


def _check(opt, o):
    for i, p in enumerate(opt.params):
        a, n = opt.offsets[i], opt.numels[i]
        _same(opt.master[a:a + n], o.p[i], f"master {i}")
        _same(p.view(torch.int16).cpu().numpy().view(np.uint16).ravel(),
              oracle.f32_to_bf16(o.p[i]), f"param {i}")
        if opt.bits8:
            b = slice(a // 256, a // 256 + -(-n // 256))
            for got, want, what in zip((opt.m[a:a + n], opt.m_scale[b], opt.v[a:a + n],
                                        opt.v_scale[b]), o.s[i], ("m", "m_scale", "v", "v_scale")):
                _same(got, want, f"{what} {i}")
        else:
            _same(opt.m[a:a + n], o.s[i][0], f"m {i}")
            _same(opt.v[a:a + n], o.s[i][1], f"v {i}")
        # the gap up to the next tensor's start stays zero
        end = opt.offsets[i + 1] if i + 1 < len(opt.params) else opt.flat
        assert not opt.master[a + n:end].any() and not opt.m[a + n:end].any()


def _opt(params, bits, hps=None, groups=None):
    opt = ss.TensorAdamW(params, hps or ss.AdamW(), groups=groups, state_bits=bits)
    opt.bits8 = bits == 8
    return opt


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("name", list(LISTS))
def test_steps_match_the_oracle(name, dt, bits):
    params, grads = _make(LISTS[name], dt, 1)
    opt, o = _opt(params, bits), _Oracle(params, bits, [AdamWConfig()], [0] * len(params))
    coef = torch.tensor([0.37], device=DEV)
    for t in range(1, 4):
        for g in grads:
            g.mul_(0.7)
        opt.step(grads, grad_coef=coef if t != 2 else None)
        o.step(grads, t, 0.37 if t != 2 else None)
    _check(opt, o)


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("shift", [1, 3, 8])
def test_unaligned_gradients(shift, bits):
    params, grads = _make(LISTS["mixed"], "bf16", 2, shift)
    opt, o = _opt(params, bits), _Oracle(params, bits, [AdamWConfig()], [0] * len(params))
    for t in (1, 2):
        opt.step(ss.TensorList(grads))
        o.step(grads, t)
    _check(opt, o)


@pytest.mark.parametrize("bits", [8, 32])
def test_unaligned_state_through_the_c_abi(bits):
    """Master, moments and the 16-bit copy at odd element offsets."""
    import ctypes
    from sharded_optimizer_step_gb300 import _capi
    n = 5000
    r = np.random.default_rng(3)
    g = torch.from_numpy(r.normal(size=n).astype(np.float32)).to(DEV)
    es = torch.uint8 if bits == 8 else torch.float32
    master, m, v = (torch.zeros(n + 8, dtype=d, device=DEV)[1:n + 1]
                    for d in (torch.float32, es, es))
    out = torch.zeros(n + 8, dtype=torch.float16, device=DEV)[3:n + 3]
    ms, vs = (torch.zeros(20, device=DEV) for _ in range(2))
    tab = (_capi.Tensor * 1)(_capi.Tensor(master.data_ptr(), m.data_ptr(), v.data_ptr(),
                                          ms.data_ptr(), vs.data_ptr(), out.data_ptr(), n, 0, 0))
    hp = ss.AdamW().at_step(1)
    _capi.check("step", _capi.lib().tensors_adamw_step(
        _capi.ptr_array([g.data_ptr()]), tab, 1, _capi.DTYPE_F32, _capi.DTYPE_F16, bits,
        ctypes.byref(hp), 1, None, None, None))
    torch.cuda.synchronize()
    o = _Oracle([torch.zeros(n)], bits, [AdamWConfig()], [0])
    o.step([g], 1)
    _same(master, o.p[0])
    _same(m, o.s[0][0])
    _same(v, o.s[0][2 if bits == 8 else 1])
    assert torch.equal(out, torch.from_numpy(o.p[0]).to(DEV).half())


@pytest.mark.parametrize("bits", [8, 32])
def test_32_bit_step_is_the_flat_step_and_groups(bits):
    params, grads = _make(LISTS["mixed"], "bf16", 4)
    groups = [i % 2 for i in range(len(params))]
    hps = [ss.AdamW(), ss.AdamW(lr=3e-4, beta1=0.8, weight_decay=0.0)]
    cfg = [AdamWConfig(), AdamWConfig(lr=3e-4, beta1=0.8, weight_decay=0.0)]
    opt, o = _opt(params, bits, hps, groups), _Oracle(params, bits, cfg, groups)
    for t in (1, 2):
        opt.step(grads)
        o.step(grads, t)
    _check(opt, o)
    if bits == 32:
        p2, g2 = _make([100_003], "bf16", 5)
        flat = [torch.zeros(100_003, device=DEV) for _ in range(3)]
        flat[0].copy_(p2[0])
        cast = torch.empty_like(p2[0])
        lst = _opt(p2, 32)
        for t in (1, 2):
            ss.fsdp_rs_avg_adamw_cast([g2[0].clone()], *flat, cast, ss.AdamW(), t)
            lst.step(g2)
        n = 100_003
        for a, b in zip(flat, (lst.master, lst.m, lst.v)):
            assert torch.equal(a, b[:n])
        assert torch.equal(cast, p2[0])


@pytest.mark.parametrize("bits", [8, 32])
def test_skip_word_and_device_step_state(bits):
    params, grads = _make(LISTS["mixed"], "f16", 6)
    opt, o = _opt(params, bits), _Oracle(params, bits, [AdamWConfig()], [0] * len(params))
    skip = torch.ones(1, dtype=torch.int32, device=DEV)
    opt.step(grads, skip=skip)
    _check(opt, o)
    opt.t = 0
    (state,) = opt.device_step_state()
    opt.step(grads, skip=skip)
    assert state.step() == 0
    skip.zero_()
    for t in (1, 2):
        opt.step(grads, skip=skip)
        o.step(grads, t)
    assert state.step() == 2
    _check(opt, o)


def test_non_finite_gradients_are_not_lost():
    """Without a skip word an inf or NaN reaches its element (32 bits) or its
    block (8 bits), and nothing else."""
    for bits in (8, 32):
        params, grads = _make([700], "f32", 7)
        grads[0][300] = float("nan")
        grads[0][600] = float("inf")
        opt, o = _opt(params, bits), _Oracle(params, bits, [AdamWConfig()], [0])
        opt.step(grads)
        o.step(grads, 1)
        m, v = opt.moments()
        assert torch.isfinite(m[:256]).all() and torch.isfinite(v[:256]).all()
        assert not torch.isfinite(m[300]) and not torch.isfinite(v[600])
        _same(opt.master[:700], o.p[0])
        if bits == 8:
            assert not torch.isfinite(m[256:700]).any()
            _same(opt.m_scale, o.s[0][1])


def test_eight_bit_state_special_values():
    """Zero gradients from a zero state, tiny and huge blocks, decay."""
    params, _ = _make([256 * 6], "f32", 8)
    g = torch.zeros(256 * 6, device=DEV)
    g[256:512] = 1e-34
    g[512:768] = torch.logspace(-12, 0, 256, device=DEV)
    g[768:1024] = 1e18
    g[1024] = 1.0
    g[1025:1280] = 1e-9
    opt, o = _opt(params, 8), _Oracle(params, 8, [AdamWConfig()], [0])
    for t in range(1, 6):
        opt.step([g])
        o.step([g], t)
        g.mul_(0.5)
    _check(opt, o)
    m, v = opt.moments()
    assert not m[:256].any() and not v[:256].any() and (v[512:768] > 0).all()


@pytest.mark.parametrize("hp", [dict(), dict(lr=0.0), dict(eps=0.0), dict(eps=2.0),
                                dict(beta1=0.0, beta2=0.0), dict(beta2=0.99999), dict(lr=1e12)],
                         ids=lambda h: "-".join(h) or "default")
def test_eight_bit_step_over_all_magnitudes(hp):
    """Blocks whose gradients have magnitudes from 2^-75 to 2^60, most of one size
    and some of many, with zeros of both signs among gradients and parameters: the
    step's roots and quotients are the IEEE ones on either side of every bound of
    the paired arithmetic."""
    r = np.random.default_rng(13)
    e = np.arange(-75, 61)
    n = 256 * len(e)
    x = np.exp2(np.repeat(e, 256) + r.uniform(-1, 1, n)) * r.choice([-1.0, 1.0], n)
    spread = np.repeat(np.arange(len(e)) % 4 == 3, 256)
    x = np.where(spread, x * np.exp2(r.integers(-30, 31, n)), x).astype(np.float32)
    x[r.integers(0, n, 20)] = 0.0
    x[r.integers(0, n, 20)] = -0.0
    params, _ = _make([n], "f32", 14)
    params[0][::97] = 0.0
    params[0][::89] = -0.0
    cfg = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.1)
    cfg.update(hp)
    opt = _opt(params, 8, ss.AdamW(**cfg))
    o = _Oracle(params, 8, [AdamWConfig(**cfg)], [0])
    sound = np.ones(n, bool)
    for t in range(1, 4):
        g = torch.from_numpy(x * np.float32(0.9 ** t)).to(DEV)
        opt.step([g])
        o.step([g], t)
        scales = opt.m_scale.cpu().numpy(), opt.v_scale.cpu().numpy()
        for got, want in zip(scales, o.s[0][1::2]):
            _same(np.isfinite(got), np.isfinite(want))
        # a block whose squares overflow keeps a non-finite scale and nothing else
        # that is fixed
        sound &= np.repeat(np.isfinite(scales[0]) & np.isfinite(scales[1]), 256)
        _same(opt.master[:n].cpu().numpy()[sound], o.p[0][sound], "master")
        _same(np.signbit(opt.master[:n].cpu().numpy()[sound]), np.signbit(o.p[0][sound]))
        for got, want, what in ((opt.m, o.s[0][0], "m"), (opt.v, o.s[0][2], "v")):
            _same(got[:n].cpu().numpy()[sound], want[sound], what)
        for got, want, what in zip(scales, o.s[0][1::2], ("m_scale", "v_scale")):
            _same(got[sound[::256]], want[sound[::256]], what)
    assert sound.mean() > 0.9


@pytest.mark.parametrize("n", [1, 7, 256, 1000, 256 * 300 + 9])
def test_moment_codes_both_ways(n):
    r = np.random.default_rng(n)
    m = (r.normal(size=n) * np.exp(r.normal(size=n) * 4)).astype(np.float32)
    v = np.square(m * np.float32(0.3)).astype(np.float32)
    blocks = -(-n // 256)
    for off in (0, 1):
        dm, dv = (torch.zeros(n + 8, dtype=torch.uint8, device=DEV)[off:off + n]
                  for _ in range(2))
        ms, vs = (torch.zeros(blocks, device=DEV) for _ in range(2))
        src = [torch.zeros(n + 4, device=DEV)[off:off + n] for _ in range(2)]
        src[0].copy_(torch.from_numpy(m))
        src[1].copy_(torch.from_numpy(v))
        ss.moments_encode(*src, dm, ms, dv, vs)
        (mc, msc), (rc, rsc) = OT.encode_m(m), OT.encode_r(np.sqrt(v))
        for got, want in ((dm, mc), (ms, msc), (dv, rc), (vs, rsc)):
            _same(got, want)
        out = [torch.zeros(n + 4, device=DEV)[off:off + n] for _ in range(2)]
        ss.moments_decode(dm, ms, dv, vs, out=out)
        _same(out[0], OT.decode_m(mc, msc))
        root = OT.decode_r(rc, rsc)
        _same(out[1], root * root)


def test_all_codes_decode_and_encode_back():
    code = torch.arange(256, dtype=torch.uint8, device=DEV)
    one = torch.ones(1, device=DEV)
    m, v = ss.moments_decode(code, one, code, one)
    _same(m, OT.e4m3_values().astype(np.float32))
    _same(v, np.square(OT.root_values().astype(np.float32)))


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("name", list(LISTS) + ["long", "above_one_launch"])
def test_norm_matches_the_oracle(name, dt):
    numels = {"long": [9_000_001, 5], "above_one_launch": [(i * 13) % 50 for i in range(2500)]}
    numels = numels.get(name) or LISTS[name]
    for shift in (0, 3):
        _, grads = _make(numels, dt, 9, shift)
        want = OT.grad_norm([g.double().cpu().numpy() for g in grads], 0.05, 8.0)
        scale = torch.tensor([8.0], device=DEV)
        found = torch.zeros(1, dtype=torch.int32, device=DEV)
        ws = ss.NormWorkspace(DEV)
        out = [ss.grad_norm_clip(grads, 0.05, loss_scale=scale, found_inf=found, workspace=ws)
               for _ in range(3)]
        assert torch.equal(out[0], out[1]) and torch.equal(out[0], out[2])
        got = out[0].double().cpu().numpy()
        # a thread's chain: at most its share of the elements, 8 sums side by side
        chain = sum(numels) / (152 * 256 * 8) + 64
        assert abs(got[0] / want[0] - 1) <= chain * 2.0 ** -24 + 2.0 ** -23
        assert abs(got[1] / want[1] - 1) <= chain * 2.0 ** -24 + 2.0 ** -21
        assert found.item() == 0


def test_norm_edges():
    z = torch.zeros(1000, device=DEV)
    out = ss.grad_norm_clip([z], 1.0)
    assert out.tolist() == [0.0, 1.0]
    assert ss.grad_norm_clip([], 1.0, out=torch.ones(2, device=DEV)).tolist() == [0.0, 1.0]
    e = torch.empty(0, device=DEV)
    assert ss.grad_norm_clip([e, e], 1.0).tolist() == [0.0, 1.0]
    assert ss.grad_norm_clip([z + 2], float("inf")).tolist()[1] == 1.0
    for bad in (float("nan"), float("inf"), 1e30):
        found = torch.zeros(1, dtype=torch.int32, device=DEV)
        z2 = z.clone()
        z2[999] = bad
        out = ss.grad_norm_clip([z, z2], 1.0, found_inf=found)
        assert found.item() == 1 and not torch.isfinite(out[0])


def test_wrappers_refuse():
    params, grads = _make([8, 16], "bf16", 1)
    opt = _opt(params, 8)
    with pytest.raises(ValueError):
        opt.step(grads[:1])
    with pytest.raises(ValueError):
        opt.step([grads[0], grads[0]])
    with pytest.raises(ValueError):
        ss.TensorList([grads[0], grads[1].float()])
    with pytest.raises(ValueError):
        ss.TensorAdamW([params[0].float()], ss.AdamW())
    with pytest.raises(ValueError):
        ss.TensorAdamW(params, [ss.AdamW()] * 9)
    with pytest.raises(ValueError):
        ss.TensorAdamW(params, ss.AdamW(), groups=[0, 1])
    lst = ss.TensorList(grads)
    grads[0].set_(torch.zeros(8, dtype=torch.bfloat16, device=DEV))
    with pytest.raises(ValueError):
        opt.step(lst)
    assert opt.t == 0


def test_loss_to_update_in_one_graph():
    """Loss, norm and update captured once, replayed, against eager calls."""
    def job():
        torch.manual_seed(0)
        n, h, v = 24, 16, 515
        x = torch.randn(n, h, device=DEV, dtype=torch.bfloat16)
        w = (torch.randn(v, h, device=DEV) * 0.1).bfloat16()
        ids = torch.randint(0, v, (n,), device=DEV)
        old = torch.full((n,), -6.2, device=DEV)
        adv = torch.randn(n, device=DEV)
        opt = ss.TensorAdamW([w], ss.AdamW(lr=1e-2), state_bits=8)
        opt.device_step_state()
        lw, nw = ss.LossWorkspace(DEV), ss.NormWorkspace(DEV)
        sc = ss.GradScaler(init_scale=1024.0, device=DEV)
        g = torch.empty(n, v, device=DEV, dtype=torch.bfloat16)
        gw = torch.empty(v, h, device=DEV, dtype=torch.bfloat16)
        loss = torch.zeros(4, device=DEV)

        def step():
            out = ss.policy_loss(x @ w.T, ids, old, adv, grad=g, loss_scale=sc.scale,
                                 workspace=lw)
            loss.copy_(out.stats)
            torch.mm(g.T, x, out=gw)
            c = ss.grad_norm_clip([gw], 0.5, loss_scale=sc.scale, found_inf=sc.found_inf,
                                  workspace=nw)
            opt.step([gw], grad_coef=c[1:], skip=sc.found_inf)
            sc.update()
        return opt, step, loss
    opt, step, loss = job()
    for _ in range(5):
        step()
    torch.cuda.synchronize()
    opt2, step2, loss2 = job()
    step2()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step2()
    for _ in range(4):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(loss, loss2) and torch.equal(opt.master, opt2.master)
    assert torch.equal(opt.m, opt2.m) and torch.equal(opt.v_scale, opt2.v_scale)
