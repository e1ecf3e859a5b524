"""Cases of the tuning operators: the clipped policy loss and the preference
loss over the vocabulary's logits with their gradients, the global gradient
norm with its clipping factor, and the AdamW step over a list of tensors with
its moments in 32 or in 8 bits.

``own = False`` computes them in plain torch operations in 32 bits;
``own = True`` through sharded_optimizer_step_gb300.

Formulas (x the logits of one token, y its id, w its weight):
  log probability  a = (x_y - max x) - log(sum exp(x - max x))
  policy loss      u = exp(a - old), pg = -min(u A, clip(u, 1 - cl, 1 + ch) A),
                   d = ref - a, kl = exp(d) - 1 - d,
                   loss = sum w (pg + k kl) / W, W = sum w
  preference loss  r = sum over a sequence of w (a - ref), h = beta (r_chosen -
                   r_rejected), loss = mean over pairs of
                   (1 - ls) softplus(-h) + ls softplus(h)
  both: d loss / d x = c (1[y] - softmax(x)), c = d loss / d a
  norm             n = sqrt(sum g^2) / s, factor = min(1, max / (n + 1e-6)) / s
  AdamW            g = grad * factor; p -= lr wd p; m = b1 m + (1 - b1) g;
                   v = b2 v + (1 - b2) g^2;
                   p -= (lr / bc1) m / (sqrt(v) / sqrt(bc2) + eps)
  8-bit moments    in blocks of 256 elements of a tensor: m as an e4m3 float
                   times max|m| / 448; sqrt(v) as an unsigned float of 4
                   exponent and 4 mantissa bits (no subnormals, largest 1.9375,
                   nearest, ties up, non-zero values at least code 1) times
                   max sqrt(v) / 1.9375
"""
import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
BLOCK = 256                 # elements that share a scale of the 8-bit moments
E4M3_MAX = 448.0
ROOT_MAX = 1.9375           # largest value of the unsigned 4 + 4 bit float
TINY = 2.0 ** -100          # a block below this is stored as zeros
HP = {"lr": 1e-3, "beta1": 0.9, "beta2": 0.999, "eps": 1e-8, "weight_decay": 0.01}
STEP = 100                  # mid-training: the bias corrections are not at their limits


# ------------------------------------------------------------------- cases

def listed():
    return [
        # the last few tokens of a stream: latency is all there is
        {"name": "policy_3x32000", "op": "policy", "tokens": 3, "vocab": 32000, "stride": 32000,
         "dtype": "bf16", "masked": 0.0, "kl": 0.0, "backward": True},
        # a micro-batch of responses behind masked prompts, Llama vocabulary
        {"name": "policy_4096x32000", "op": "policy", "tokens": 4096, "vocab": 32000,
         "stride": 32000, "dtype": "bf16", "masked": 0.3, "kl": 0.05, "backward": True},
        # a large micro-batch on GPT-2's odd vocabulary: rows start at any 2-byte address
        {"name": "policy_8192x50257", "op": "policy", "tokens": 8192, "vocab": 50257,
         "stride": 50257, "dtype": "bf16", "masked": 0.25, "kl": 0.05, "backward": True},
        # evaluation: the loss and the log probabilities alone, fp16 logits
        {"name": "policy_eval_2048x32000", "op": "policy", "tokens": 2048, "vocab": 32000,
         "stride": 32000, "dtype": "f16", "masked": 0.1, "kl": 0.05, "backward": False},
        # two short pairs
        {"name": "pref_2x24", "op": "preference", "pairs": 2, "mean_len": 24, "vocab": 32000,
         "stride": 32000, "dtype": "bf16", "masked": 0.25, "smoothing": 0.0},
        # a batch of answer pairs behind masked prompts
        {"name": "pref_16x256", "op": "preference", "pairs": 16, "mean_len": 256, "vocab": 32000,
         "stride": 32000, "dtype": "bf16", "masked": 0.3, "smoothing": 0.1},
        # fp32 logits, odd vocabulary in rows padded to a multiple of 64
        {"name": "pref_f32_4x100", "op": "preference", "pairs": 4, "mean_len": 100, "vocab": 50257,
         "stride": 50304, "dtype": "f32", "masked": 0.2, "smoothing": 0.0},
        # the three tensors of a 9.4M-parameter unit, fp32 accumulated gradients
        {"name": "norm_unit_9m_f32", "op": "norm", "shapes": "unit_9m", "layers": 1,
         "dtype": "f32", "scale": 1.0},
        # GPT-2 small's 148 tensors, fp16 gradients under a loss scale
        {"name": "norm_gpt2_small", "op": "norm", "shapes": "gpt2_small", "layers": 12,
         "dtype": "f16", "scale": 1024.0},
        # the same tensors' update with fp32 moments
        {"name": "adamw32_gpt2_small", "op": "adamw", "shapes": "gpt2_small", "layers": 12,
         "dtype": "bf16", "bits": 32},
        # norm vectors and matrices mixed, as a DDP replica holds them, 8-bit moments
        {"name": "adamw8_ragged", "op": "adamw", "shapes": "ragged", "layers": 1,
         "dtype": "bf16", "bits": 8},
        # a Llama-1B shape's 147 tensors, 8-bit moments
        {"name": "adamw8_llama_1b", "op": "adamw", "shapes": "llama_1b", "layers": 16,
         "dtype": "bf16", "bits": 8},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["policy", "policy", "preference", "norm", "adamw", "adamw"])
    if op in ("policy", "preference"):
        vocab = rng.choice([32000, 50257, _log_int(rng, 1000, 50000), _log_int(rng, 1000, 50000)])
        stride = rng.choice([vocab, vocab, (vocab + 63) // 64 * 64])
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        masked = rng.choice([0.0, round(rng.uniform(0.05, 0.6), 2)])
        most = 8192 * 50257 // vocab * 2 // BYTES[dtype]
    if op == "policy":
        return {"op": op, "tokens": _log_int(rng, 1, min(most, 16384)), "vocab": vocab,
                "stride": stride, "dtype": dtype, "masked": masked,
                "kl": rng.choice([0.0, round(rng.uniform(0.01, 0.2), 3)]),
                "backward": rng.random() < 0.75}
    if op == "preference":
        mean = _log_int(rng, 2, 700)
        return {"op": op, "pairs": _log_int(rng, 1, max(1, min(32, most // (4 * mean)))),
                "mean_len": mean, "vocab": vocab, "stride": stride, "dtype": dtype,
                "masked": masked, "smoothing": rng.choice([0.0, 0.1])}
    shapes = rng.choice(["unit_9m", "gpt2_small", "ragged", "llama_1b", "mix", "mix"])
    layers = {"unit_9m": rng.randint(1, 8), "gpt2_small": rng.randint(1, 12), "ragged": 1,
              "llama_1b": rng.randint(1, 8), "mix": rng.randint(1, 1 << 20)}[shapes]
    if op == "norm":
        return {"op": op, "shapes": shapes, "layers": layers,
                "dtype": rng.choice(["bf16", "f16", "f32"]), "scale": rng.choice([1.0, 256.0])}
    return {"op": op, "shapes": shapes, "layers": layers,
            "dtype": rng.choice(["bf16", "bf16", "f16", "f32"]), "bits": rng.choice([8, 32])}


def _shapes(case):
    """The tensors' element counts, in registration order."""
    kind, layers = case["shapes"], case["layers"]
    if kind == "unit_9m":
        return [1024 * 1024, 1024 * 4096, 4096 * 1024] * layers
    if kind == "gpt2_small":
        h = 768
        block = [h * 3 * h, 3 * h, h * h, h, h * 4 * h, 4 * h, 4 * h * h, h, h, h, h, h]
        return [50257 * h, 1024 * h, h, h] + block * layers
    if kind == "llama_1b":
        h, f = 2048, 8192
        return [32000 * h] + ([h * h] * 4 + [f * h] * 3 + [h, h]) * layers + [h, 32000 * h]
    if kind == "ragged":
        return [768, 768, 768 * 768, 1, 4096 * 4096, 0, 12289, 255, 257, 768 * 2304 + 3, 50257]
    # "mix": `layers` seeds the list: up to 600 tensors of 1 to 3M elements, odd sizes among them
    r = random.Random(layers)
    sizes = [_log_int(r, 1, 3_000_000) for _ in range(_log_int(r, 2, 600))]
    return [n if r.random() < 0.5 else max(8, n // 8 * 8) for n in sizes]


def _lengths(case):
    """Tokens of the 2 * pairs sequences (chosen, rejected, chosen, ...)."""
    r = random.Random(case["pairs"] * 1000 + case["mean_len"])
    return [max(1, int(case["mean_len"] * r.uniform(0.4, 1.6))) for _ in range(2 * case["pairs"])]


def _tokens(case):
    return case["tokens"] if case["op"] == "policy" else sum(_lengths(case))


def _offsets(numels):
    """Start of each tensor in the flat state, whole blocks apart, and the flat length."""
    off = [0]
    for n in numels:
        off.append(off[-1] + (n + BLOCK - 1) // BLOCK * BLOCK)
    return off[:-1], off[-1]


def work(case):
    if case["op"] in ("policy", "preference"):
        n, v, es = _tokens(case), case["vocab"], BYTES[case["dtype"]]
        live = n - int(round(n * case["masked"]))
        back = case["op"] == "preference" or case["backward"]
        # the logits of the tokens that count, every row of the gradient, and
        # per token: id, weight, the given log probabilities, the log probability
        return {"bytes": live * v * es + (n * v * es if back else 0) + 32 * n,
                "flops": live * v * (8 if back else 4)}
    total, es = sum(_shapes(case)), BYTES[case["dtype"]]
    if case["op"] == "norm":
        return {"bytes": total * es, "flops": 2 * total}
    if case["bits"] == 32:     # gradient, three fp32 arrays both ways, the bf16 copy
        return {"bytes": total * (es + 24 + 2), "flops": 18 * total}
    # gradient, master both ways, both codes both ways, the bf16 copy, and the
    # fp32 values that the codes stand for
    return {"bytes": total * (es + 8 + 4 + 2 + 8) + total / BLOCK * 16, "flops": 30 * total}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device=DEV, dtype=dtype)


def _prepare_tokens(case, seed):
    g = _gen(seed)
    n, v, dt = _tokens(case), case["vocab"], DTYPES[case["dtype"]]
    full = torch.full((n, case["stride"]), float("nan"), dtype=dt, device=DEV)
    logits = full[:, :v]                       # padding columns hold NaN: not part of the input
    for a in range(0, n, 1024):
        b = min(n, a + 1024)
        logits[a:b] = (_randn(g, b - a, v) * 1.5).to(dt)
    ids = torch.randint(0, v, (n,), generator=g, device=DEV)
    # the sampled token is usually a likely one
    boost = torch.rand(n, generator=g, device=DEV) * 9 + 4
    rows = torch.arange(n, device=DEV)
    logits[rows, ids] = (logits[rows, ids].float() + boost).to(dt)
    lp = torch.cat([torch.log_softmax(logits[a:a + 1024].float(), 1)
                    .gather(1, ids[a:a + 1024, None])[:, 0] for a in range(0, n, 1024)])
    weights = torch.ones(n, device=DEV)
    weights[torch.randperm(n, generator=g, device=DEV)[:int(round(n * case["masked"]))]] = 0.0
    s = {"case": case, "logits": logits, "ids": ids, "weights": weights,
         "ref": lp + 0.1 * _randn(g, n), "grad": None, "ws": None}
    if case["op"] == "policy":
        old = lp + 0.25 * _randn(g, n)
        # keep the ratio off the clip's two edges, where one rounding decides
        ratio = torch.exp(lp - old)
        for edge in (0.8, 1.2):
            old = torch.where((ratio - edge).abs() < 1e-3, old - 4e-3, old)
        s["old"], s["adv"] = old, _randn(g, n)
    else:
        s["lens"] = _lengths(case)
        ends = torch.tensor(s["lens"], device=DEV).cumsum(0)
        s["seq"] = torch.bucketize(rows, ends, right=True)
    if case["op"] == "preference" or case["backward"]:
        s["grad"] = torch.empty(n, case["stride"], dtype=dt, device=DEV)[:, :v]
    return s


def _prepare_tensors(case, seed):
    g = _gen(seed)
    numels, dt = _shapes(case), DTYPES[case["dtype"]]
    off, flat = _offsets(numels)
    scale = case.get("scale", 1.0)
    s = {"case": case, "numels": numels, "off": off, "flat": flat, "max_norm": 1.0,
         "grads": [(_randn(g, n) * (1e-3 * scale)).to(dt) for n in numels],
         "scale": torch.tensor([scale], device=DEV)}
    if case["op"] == "norm":
        return s
    s["coef"] = torch.tensor([0.7310586], device=DEV)      # the clipping factor, a device word
    held = torch.zeros(flat, dtype=torch.bool, device=DEV)
    for o, n in zip(off, numels):
        held[o:o + n] = True
    s["master"] = torch.where(held, _randn(g, flat) * 0.02, 0.0)
    m = torch.where(held, _randn(g, flat) * 3e-4, 0.0)
    r = torch.where(held, torch.exp(0.5 * _randn(g, flat)) * 8e-4, 0.0)
    if case["bits"] == 32:
        s["m"], s["v"] = m, r * r
    else:
        s["m"], s["m_scale"] = _encode_m(m)
        s["v"], s["v_scale"] = _encode_r(r)
    del m, r, held
    s["params"], s["scalars"] = s["master"].to(torch.bfloat16), _scalars()
    return s


def prepare(case, seed):
    s = _prepare_tokens(case, seed) if case["op"] in ("policy", "preference") \
        else _prepare_tensors(case, seed)
    if own:                     # what a user's program keeps: workspaces and the optimizer
        import sharded_optimizer_step_gb300 as ss
        s["ss"] = ss
        if case["op"] in ("policy", "preference"):
            s["ws"] = ss.LossWorkspace(DEV)
        elif case["op"] == "norm":
            s["ws"] = ss.NormWorkspace(DEV)
            s["list"] = ss.TensorList(s["grads"])
        else:
            s["list"] = ss.TensorList(s["grads"])
            views = [s["params"][o:o + n] for o, n in zip(s["off"], s["numels"])]
            opt = ss.TensorAdamW(views, ss.AdamW(**HP), state_bits=case["bits"])
            opt.t = STEP
            for name in ("master", "m", "v") + (("m_scale", "v_scale") if case["bits"] == 8 else ()):
                getattr(opt, name).copy_(s.pop(name))
            s["opt"] = opt
            if case["bits"] == 8:
                s["moments"] = (torch.empty_like(opt.master), torch.empty_like(opt.master))
    return s


# -------------------------------------------------------------------- plain

def _log_probs(s):
    """exp(x - max) of every row, its sum, and the ids' log probabilities."""
    x = s["logits"].float()
    mx = x.amax(1, keepdim=True)
    e = torch.exp(x - mx)
    total = e.sum(1, keepdim=True)
    a = (x.gather(1, s["ids"][:, None]) - mx - torch.log(total))[:, 0]
    return e, total, a


def _logit_grad(s, e, total, c):
    """c (1[y] - softmax) in the logits' type; rows with c = 0 are zero."""
    g = (e / total) * (-c)[:, None]
    g.scatter_add_(1, s["ids"][:, None], c[:, None])
    return torch.where((s["weights"] != 0)[:, None], g, 0.0).to(s["logits"].dtype)


def _plain_policy(s):
    case, w = s["case"], s["weights"]
    live = w != 0
    e, total, a = _log_probs(s)
    u = torch.exp(a - s["old"])
    one, two = u * s["adv"], torch.clamp(u, 1 - 0.2, 1 + 0.2) * s["adv"]
    pg, clipped = -torch.minimum(one, two), (one > two).float()
    d = s["ref"] - a
    kl = torch.expm1(d) - d
    norm = w.sum()
    k = w / norm
    terms = torch.stack([pg + case["kl"] * kl if case["kl"] else pg, pg,
                         kl if case["kl"] else torch.zeros_like(kl), clipped], 0)
    stats = torch.where(live, terms * k, 0.0).sum(1)
    out = {"stats": stats, "logps": torch.where(live, a, 0.0)}
    if case["backward"]:
        c = torch.where(one > two, 0.0, -one)
        if case["kl"]:
            c = c - case["kl"] * torch.expm1(d)
        out["grad"] = _logit_grad(s, e, total, c * k)
    return out


def _softplus(x):
    return torch.clamp(x, min=0) + torch.log1p(torch.exp(-x.abs()))


def _plain_preference(s, beta=0.1):
    case, w, ls = s["case"], s["weights"], s["case"]["smoothing"]
    live = w != 0
    e, total, a = _log_probs(s)
    r = torch.zeros(2 * case["pairs"], device=DEV)
    r.index_add_(0, s["seq"], torch.where(live, w * (a - s["ref"]), 0.0))
    h = beta * (r[0::2] - r[1::2])
    loss = (1 - ls) * _softplus(-h) + ls * _softplus(h)
    sig = 1 / (1 + torch.exp(-h))
    dh = (ls * sig - (1 - ls) * (1 - sig)) * (beta / case["pairs"])
    c = torch.stack([dh, -dh], 1).reshape(-1)[s["seq"]] * w
    return {"stats": torch.stack([loss.mean(), h.mean(), (h > 0).float().mean()]),
            "log_ratios": r, "logps": torch.where(live, a, 0.0),
            "grad": _logit_grad(s, e, total, c)}


def _plain_norm(s):
    norm = torch.sqrt(torch.cat(s["grads"]).float().square().sum()) / s["scale"][0]
    coef = torch.clamp(s["max_norm"] / (norm + 1e-6), max=1.0) / s["scale"][0]
    return {"norm": torch.stack([norm, coef])}


def _scales(x, top):
    """Of every block: its scale and the factor that brings its largest value to `top`."""
    big = x.abs().amax(1, keepdim=True)
    keep = ~(big < TINY)
    t = torch.full_like(big, top)
    return torch.where(keep, big / t, 0.0), torch.where(keep, t / big, 0.0)


def _encode_m(m):
    x = m.view(-1, BLOCK)
    scale, up = _scales(x, E4M3_MAX)
    code = (x * up).to(torch.float8_e4m3fn).view(torch.uint8)
    return code.reshape(-1), scale[:, 0].contiguous()


def _decode_m(code, scale):
    return (code.view(torch.float8_e4m3fn).float().view(-1, BLOCK) * scale[:, None]).reshape(-1)


def _encode_r(r):
    x = r.view(-1, BLOCK)
    scale, up = _scales(x, ROOT_MAX)
    frac, exp = torch.frexp(x * up)            # frac in [0.5, 1), value frac 2^exp
    q = torch.floor(frac * 32 + 0.5).to(torch.int32) + (exp.to(torch.int32) + 14) * 16 - 16
    code = torch.where(x * up > 0, torch.clamp(q, 1, 255), 0).to(torch.uint8)
    return code.reshape(-1), scale[:, 0].contiguous()


def _decode_r(code, scale):
    c = code.to(torch.int32)
    value = torch.ldexp(1 + (c & 15).float() / 16, (c >> 4) - 15)
    value = torch.where(c > 0, value, 0.0)
    return (value.view(-1, BLOCK) * scale[:, None]).reshape(-1)


def _flat_grads(s):
    """The gradients in the flat state's layout, zeros between them."""
    pad = torch.zeros(BLOCK, dtype=s["grads"][0].dtype, device=DEV)
    return torch.cat([t for x in s["grads"] for t in (x, pad[:-x.numel() % BLOCK])]).float()


def _scalars():
    """The step's fp32 scalars, from double."""
    bc1 = 1 - math.prod([HP["beta1"]] * (STEP + 1))
    bc2 = 1 - math.prod([HP["beta2"]] * (STEP + 1))
    return torch.tensor([HP["lr"] * HP["weight_decay"], HP["beta1"], 1 - HP["beta1"],
                         HP["beta2"], 1 - HP["beta2"], HP["lr"] / bc1, math.sqrt(bc2),
                         HP["eps"]], dtype=torch.float64).float().to(DEV).unbind()


def _plain_adamw(s):
    lr_wd, b1, omb1, b2, omb2, size, root_bc2, eps = s["scalars"]
    small = s["case"]["bits"] == 8
    g = _flat_grads(s) * s["coef"]
    if small:
        m, r = _decode_m(s["m"], s["m_scale"]), _decode_r(s["v"], s["v_scale"])
        v = r * r
    else:
        m, v = s["m"], s["v"]
    p = s["master"] - lr_wd * s["master"]
    m = b1 * m + omb1 * g
    v = b2 * v + (omb2 * g) * g
    del g
    r = torch.sqrt(v)
    s["master"] = p - (size * m) / (r / root_bc2 + eps)
    s["params"] = s["master"].to(torch.bfloat16)
    if small:
        s["m"], s["m_scale"] = _encode_m(m)
        s["v"], s["v_scale"] = _encode_r(r)
        m, r = _decode_m(s["m"], s["m_scale"]), _decode_r(s["v"], s["v_scale"])
        v = r * r
    else:
        s["m"], s["v"] = m, v
    return {"master": s["master"], "params": s["params"], "m": m, "v": v}


# ---------------------------------------------------------------- the paths

def _own(s):
    case, ss = s["case"], s["ss"]
    if case["op"] == "policy":
        out = ss.policy_loss(s["logits"], s["ids"], s["old"], s["adv"],
                             ref_logps=s["ref"] if case["kl"] else None, kl_coef=case["kl"],
                             weights=s["weights"], clip_low=0.2, clip_high=0.2, grad=s["grad"],
                             workspace=s["ws"])
        return {"stats": out.stats, "logps": out.logps,
                **({"grad": out.grad} if case["backward"] else {})}
    if case["op"] == "preference":
        out = ss.preference_loss(s["logits"], s["ids"], s["lens"], s["ref"], beta=0.1,
                                 label_smoothing=case["smoothing"], weights=s["weights"],
                                 grad=s["grad"], workspace=s["ws"])
        return {"stats": out.stats, "log_ratios": out.log_ratios, "logps": out.logps,
                "grad": out.grad}
    if case["op"] == "norm":
        return {"norm": ss.grad_norm_clip(s["list"], s["max_norm"], loss_scale=s["scale"],
                                          workspace=s["ws"])}
    opt = s["opt"]
    opt.t = STEP
    opt.step(s["list"], grad_coef=s["coef"])
    m, v = opt.moments(out=s["moments"]) if case["bits"] == 8 else (opt.m, opt.v)
    return {"master": opt.master, "params": s["params"], "m": m, "v": v}


def run(s):
    if own:
        return _own(s)
    return {"policy": _plain_policy, "preference": _plain_preference, "norm": _plain_norm,
            "adamw": _plain_adamw}[s["case"]["op"]](s)


# -------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    """Row by row and tensor by tensor from the definitions, in double."""
    if case["op"] in ("policy", "preference"):
        s = _prepare_tokens(case, seed)
        return _exact_tokens(case, s)
    s = _prepare_tensors(case, seed)
    if case["op"] == "norm":
        total = sum(float((x.double() ** 2).sum()) for x in s["grads"])
        norm = math.sqrt(total) / case["scale"]
        return {"norm": torch.tensor([norm, min(1.0, 1.0 / (norm + 1e-6)) / case["scale"]],
                                     dtype=torch.float64)}
    return _exact_adamw(case, s)


def _exact_tokens(case, s):
    n, live = _tokens(case), s["weights"].double() != 0
    w = s["weights"].double()
    lse = torch.cat([torch.logsumexp(s["logits"][a:a + 512].double(), 1)
                     for a in range(0, n, 512)])
    picked = s["logits"][torch.arange(n, device=DEV), s["ids"]].double()
    a, ref = picked - lse, s["ref"].double()
    zero = torch.zeros_like(a)
    out = {"logps": torch.where(live, a, zero)}
    if case["op"] == "policy":
        k = w / w.sum()
        adv, ratio = s["adv"].double(), torch.exp(a - s["old"].double())
        best = torch.where((adv > 0) & (ratio > 1.2), 1.2 * adv,
                           torch.where((adv < 0) & (ratio < 0.8), 0.8 * adv, ratio * adv))
        cut = ((adv > 0) & (ratio > 1.2)) | ((adv < 0) & (ratio < 0.8))
        d = ref - a
        kl = torch.expm1(d) - d if case["kl"] else zero
        slope = torch.where(cut, zero, -ratio * adv)
        if case["kl"]:
            slope = slope - case["kl"] * torch.expm1(d)
        terms = [-best + case["kl"] * kl, -best, kl, cut.double()]
        out["stats"] = torch.stack([(torch.where(live, t, zero) * k).sum() for t in terms])
        c = slope * k
        if not case["backward"]:
            return out
    else:
        ls, beta = case["smoothing"], 0.1
        at = [0]
        for x in s["lens"]:
            at.append(at[-1] + x)
        part = torch.where(live, w * (a - ref), zero)
        r = torch.stack([part[i:j].sum() for i, j in zip(at, at[1:])])
        h = beta * (r[0::2] - r[1::2])
        sp = torch.nn.functional.softplus
        loss = (1 - ls) * sp(-h) + ls * sp(h)
        out["stats"] = torch.stack([loss.mean(), h.mean(), (h > 0).double().mean()])
        out["log_ratios"] = r
        dh = ls * torch.sigmoid(h) - (1 - ls) * torch.sigmoid(-h)
        c = torch.cat([w[i:j] * beta * dh[q // 2] * (1 if q % 2 == 0 else -1) / case["pairs"]
                       for q, (i, j) in enumerate(zip(at, at[1:]))])
    # one value of each element, in fp64 where it fits and in the gradient's place
    if n * case["vocab"] > 150_000_000:
        out["grad"] = None
        return out
    grad = torch.empty(n, case["vocab"], dtype=torch.float64, device=DEV)
    for i in range(0, n, 512):
        j = min(n, i + 512)
        p = torch.softmax(s["logits"][i:j].double(), 1)
        p[torch.arange(j - i, device=DEV), s["ids"][i:j]] -= 1
        grad[i:j] = torch.where(live[i:j, None], -c[i:j, None] * p, 0.0)
    out["grad"] = grad
    return out


def _exact_round(x, bits, low):
    """x >= 0 to the nearest float of `bits` mantissa bits and exponent >= low."""
    e = torch.clamp(torch.floor(torch.log2(torch.clamp(x, min=1e-300))), min=low)
    step = torch.exp2(e - bits)
    return torch.floor(x / step + 0.5) * step


def _exact_adamw(case, s):
    t = STEP + 1
    bc1, bc2 = 1 - HP["beta1"] ** t, 1 - HP["beta2"] ** t
    keep = {k: torch.zeros(s["flat"], dtype=torch.float64, device=DEV)
            for k in ("master", "m", "v")}
    for x, o in zip(s["grads"], s["off"]):
        n = x.numel()
        blocks = (n + BLOCK - 1) // BLOCK
        if not n:
            continue
        g = x.double() * s["coef"].double()
        p = s["master"][o:o + n].double()
        if case["bits"] == 8:
            each = torch.arange(n, device=DEV) // BLOCK
            b = o // BLOCK
            ms, vs = s["m_scale"][b:b + blocks].double(), s["v_scale"][b:b + blocks].double()
            m = s["m"][o:o + n].view(torch.float8_e4m3fn).double() * ms[each]
            c = s["v"][o:o + n].long()
            v = (torch.where(c > 0, (16 + c % 16) * torch.exp2((c // 16 - 19).double()), 0.0)
                 * vs[each]) ** 2
        else:
            m, v = s["m"][o:o + n].double(), s["v"][o:o + n].double()
        m = HP["beta1"] * m + (1 - HP["beta1"]) * g
        v = HP["beta2"] * v + (1 - HP["beta2"]) * g * g
        p = p * (1 - HP["lr"] * HP["weight_decay"])
        p = p - HP["lr"] / bc1 * m / (v.sqrt() / math.sqrt(bc2) + HP["eps"])
        if case["bits"] == 8:
            r = v.sqrt()
            top = torch.zeros(blocks, dtype=torch.float64, device=DEV)
            top = top.scatter_reduce(0, each, m.abs(), "amax")[each]
            # e4m3: 3 mantissa bits, exponents from -6, ties as they fall
            y = _exact_round(m.abs() * (E4M3_MAX / top), 3, -6)
            m = torch.where(top >= TINY, torch.sign(m) * y * top / E4M3_MAX, 0.0)
            top = torch.zeros(blocks, dtype=torch.float64, device=DEV)
            top = top.scatter_reduce(0, each, r, "amax")[each]
            z = r * (ROOT_MAX / top)
            y = torch.clamp(_exact_round(z, 4, -15), min=1.0625 * 2.0 ** -15, max=ROOT_MAX)
            v = torch.where((top >= TINY) & (z > 0), y * top / ROOT_MAX, 0.0) ** 2
        keep["master"][o:o + n], keep["m"][o:o + n], keep["v"][o:o + n] = p, m, v
    return {**keep, "params": keep["master"]}
