"""Cases of the operators around a model's own tensors: the token embedding and
its gradient, layer norm and its gradients, and the Newton-Schulz
orthogonalised update of matrices, alone and as an optimizer's step.

``own = False`` computes them in plain torch operations in 32 bits;
``own = True`` through sharded_optimizer_step_gb300.

Formulas:
  embedding   out[i] = scale table[ids[i]]; an id outside [0, vocabulary) gives zeros
  gradient    d table[v] = scale sum of d_out[i] over i with ids[i] = v, written to
              all rows, or added to the rows that occur
  layer norm  xh = (x - mean(x)) r, r = 1 / sqrt(var(x) + eps), out = xh w + b
  gradients   g = d_out w, d_x = r (g - mean(g) - xh mean(g xh)),
              d_w = sum over rows of d_out xh, d_b = sum over rows of d_out
  orthogonal  X = u / (|u| + 1e-7), transposed where u is taller than wide; five times
              A = X X^T, X = a X + (b A + c A A) X
  muon step   g = grad coef, m = mu m + (1 - mu) g, u = mu m + (1 - mu) g,
              p -= lr wd p, p -= lr 0.2 sqrt(max(rows, columns)) orthogonal(u)
"""
import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
EPS = 1e-5                            # layer norm
QUINTIC = (3.4445, -4.7750, 2.0315)   # a, b, c
ROUNDS = 5
HP = {"lr": 1e-3, "momentum": 0.95, "weight_decay": 0.1}
RMS = 0.2
FLAT = 256                            # elements at whose multiples a tensor of the flat state starts


# ------------------------------------------------------------------- cases

def listed():
    return [
        # the next tokens of a few streams
        {"name": "embedding_3x768", "op": "embedding", "tokens": 3, "vocab": 50257, "dim": 768,
         "dtype": "bf16", "ids": "uniform", "masked": 0.0, "scale": 1.0},
        # a packed micro-batch, Llama vocabulary, rows scaled by the root of their length
        {"name": "embedding_16384x4096", "op": "embedding", "tokens": 16384, "vocab": 32000,
         "dim": 4096, "dtype": "bf16", "ids": "zipf", "masked": 0.05, "scale": 64.0},
        # GPT-2's tied table: added to the head's fp32 gradient
        {"name": "embedding_grad_tied_4096x768", "op": "embedding_grad", "tokens": 4096,
         "vocab": 50257, "dim": 768, "dtype": "bf16", "grad": "f32", "ids": "zipf",
         "masked": 0.0, "scale": 1.0, "accumulate": True},
        # a table of its own, every row of the gradient written, some tokens padding
        {"name": "embedding_grad_16384x4096", "op": "embedding_grad", "tokens": 16384,
         "vocab": 32000, "dim": 4096, "dtype": "bf16", "grad": "bf16", "ids": "zipf",
         "masked": 0.05, "scale": 64.0, "accumulate": False},
        # the last norm of a few streams' next tokens, forward alone
        {"name": "layer_norm_3x768", "op": "layer_norm", "rows": 3, "cols": 768, "stride": 768,
         "dtype": "bf16", "backward": False},
        # a micro-batch of GPT-2 small
        {"name": "layer_norm_4096x768", "op": "layer_norm", "rows": 4096, "cols": 768,
         "stride": 768, "dtype": "bf16", "backward": True},
        # a large micro-batch of a wide model
        {"name": "layer_norm_16384x4096", "op": "layer_norm", "rows": 16384, "cols": 4096,
         "stride": 4096, "dtype": "bf16", "backward": True},
        # an odd width in padded fp32 rows
        {"name": "layer_norm_f32_999x5003", "op": "layer_norm", "rows": 999, "cols": 5003,
         "stride": 5056, "dtype": "f32", "backward": True},
        # one small matrix: latency
        {"name": "orthogonalize_256", "op": "orthogonalize", "shapes": "square", "size": 256,
         "dtype": "f32", "out": "bf16"},
        # wide, tall, odd and tiny matrices in one call
        {"name": "orthogonalize_mix", "op": "orthogonalize", "shapes": "mix", "size": 15,
         "dtype": "bf16", "out": "bf16"},
        # the step of a 9.4M-parameter unit
        {"name": "muon_unit_9m", "op": "muon", "shapes": "unit_9m", "size": 1, "dtype": "f32"},
        # the step of two layers of a Llama-1B shape
        {"name": "muon_llama_1b_2_layers", "op": "muon", "shapes": "llama_1b", "size": 2,
         "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["embedding", "embedding_grad", "embedding_grad", "layer_norm", "layer_norm",
                     "orthogonalize", "muon", "muon"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op in ("embedding", "embedding_grad"):
        dim = rng.choice([768, 2048, 4096, _log_int(rng, 8, 500) * 8, _log_int(rng, 5, 4000)])
        vocab = min(rng.choice([32000, 50257, _log_int(rng, 100, 50000)]), 32000 * 4096 // dim)
        case = {"op": op, "tokens": _log_int(rng, 1, 16384), "vocab": vocab, "dim": dim,
                "dtype": dtype, "ids": rng.choice(["uniform", "zipf", "zipf"]),
                "masked": rng.choice([0.0, round(rng.uniform(0.05, 0.5), 2)]),
                "scale": rng.choice([1.0, round(math.sqrt(dim), 3)])}
        if op == "embedding_grad":
            case["grad"] = rng.choice([dtype, "f32"]) if dim <= 2048 else "bf16"
            case["accumulate"] = rng.random() < 0.5
        return case
    if op == "layer_norm":
        cols = rng.choice([768, 4096, _log_int(rng, 2, 1000) * 8, _log_int(rng, 5, 8000)])
        return {"op": op, "rows": _log_int(rng, 1, min(32768, 16384 * 4096 // cols)), "cols": cols,
                "stride": rng.choice([cols, cols, (cols + 63) // 64 * 64]), "dtype": dtype,
                "backward": rng.random() < 0.75}
    shapes = rng.choice(["square", "pair", "mix", "unit_9m"] + (["llama_1b"] if op == "muon" else []))
    size = {"square": _log_int(rng, 16, 2048), "pair": _log_int(rng, 16, 1024),
            "mix": rng.randint(1, 1 << 20), "unit_9m": rng.randint(1, 3), "llama_1b": 1}[shapes]
    case = {"op": op, "shapes": shapes, "size": size, "dtype": dtype}
    if op == "orthogonalize":
        case["out"] = rng.choice(["bf16", "bf16", "f16"])
    return case


def _shapes(case):
    """(rows, columns) of the matrices."""
    kind, size = case["shapes"], case["size"]
    if kind == "square":
        return [(size, size)]
    if kind == "pair":                   # up and down projection
        return [(4 * size, size), (size, 4 * size)]
    if kind == "unit_9m":
        return [(1024, 1024), (1024, 4096), (4096, 1024)] * size
    if kind == "llama_1b":
        h, f = 2048, 8192
        return ([(h, h)] * 4 + [(f, h)] * 2 + [(h, f)]) * size
    # "mix": `size` seeds the list
    r = random.Random(size)
    side = lambda: 1 if r.random() < 0.08 else _log_int(r, 8, 1200)  # noqa: E731
    return [(side(), side()) for _ in range(_log_int(r, 3, 24))]


def _offsets(numels):
    off = [0]
    for n in numels:
        off.append(off[-1] + (n + FLAT - 1) // FLAT * FLAT)
    return off[:-1], off[-1]


def work(case):
    if case["op"] == "embedding":
        row = case["dim"] * BYTES[case["dtype"]]
        return {"bytes": (min(case["tokens"], case["vocab"]) + case["tokens"]) * row
                + 8 * case["tokens"], "flops": case["tokens"] * case["dim"]}
    if case["op"] == "embedding_grad":
        n, row = case["tokens"], case["dim"] * BYTES[case["grad"]]
        table = min(n, case["vocab"]) * 2 if case["accumulate"] else case["vocab"]
        return {"bytes": n * case["dim"] * BYTES[case["dtype"]] + table * row + 8 * n,
                "flops": n * case["dim"]}
    if case["op"] == "layer_norm":
        n = case["rows"] * case["cols"]
        passes = 5 if case["backward"] else 2    # x, out; again x, d_out, d_x
        return {"bytes": passes * n * BYTES[case["dtype"]] + 8 * case["rows"] + 16 * case["cols"],
                "flops": n * (20 if case["backward"] else 8)}
    flops, total = 0, 0
    for r, c in _shapes(case):
        m, n = min(r, c), max(r, c)
        flops += ROUNDS * (3 * m * m * n + m * m * m)     # A and A A: one half, they are symmetric
        total += r * c
    es = BYTES[case["dtype"]]
    # the gradient; momentum and weights both ways and the bf16 copy, or the result
    return {"bytes": total * (es + 18 if case["op"] == "muon" else es + 2), "flops": flops}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _ids(case, g):
    n, v = case["tokens"], case["vocab"]
    u = torch.rand(n, generator=g, device=DEV, dtype=torch.float64)
    if case["ids"] == "zipf":            # frequency about 1 / rank, ranks spread over the ids
        rank = torch.exp(u * math.log(v + 1)).long() - 1
        ids = torch.remainder(rank.clamp(0, v - 1) * 7919, v)
    else:
        ids = (u * v).long().clamp(0, v - 1)
    off = torch.randperm(n, generator=g, device=DEV)[:int(round(n * case["masked"]))]
    ids[off] = -1                        # padding
    return ids


def _prepare_embedding(case, seed):
    g, dt = _gen(seed), DTYPES[case["dtype"]]
    s = {"case": case, "ids": _ids(case, g)}
    if case["op"] == "embedding":
        s["table"] = (_randn(g, case["vocab"], case["dim"]) * 0.02).to(dt)
        s["out"] = torch.empty(case["tokens"], case["dim"], dtype=dt, device=DEV)
        return s
    s["d_out"] = (_randn(g, case["tokens"], case["dim"]) * 1e-3).to(dt)
    shape = (case["vocab"], case["dim"])
    s["grad"] = ((_randn(g, *shape) * 1e-3).to(DTYPES[case["grad"]]) if case["accumulate"]
                 else torch.empty(*shape, dtype=DTYPES[case["grad"]], device=DEV))
    return s


def _prepare_norm(case, seed):
    g, dt = _gen(seed), DTYPES[case["dtype"]]
    rows, cols = case["rows"], case["cols"]
    spread = torch.exp(0.5 * _randn(g, cols))            # some channels are larger than others

    def matrix(x):
        full = torch.full((rows, case["stride"]), float("nan"), dtype=dt, device=DEV)
        full[:, :cols] = x                               # padding columns are not part of it
        return full[:, :cols]

    s = {"case": case, "x": matrix(_randn(g, rows, cols) * spread + 0.5 * _randn(g, rows, 1) + 0.3),
         "w": 1 + 0.2 * _randn(g, cols), "b": 0.1 * _randn(g, cols),
         "out": torch.empty(rows, cols, dtype=dt, device=DEV)}
    if case["backward"]:
        s["d_out"] = matrix(_randn(g, rows, cols) * 1e-2)
        s["d_x"] = torch.empty(rows, cols, dtype=dt, device=DEV)
        s["d_w"], s["d_b"] = torch.empty_like(s["w"]), torch.empty_like(s["b"])
    return s


def _prepare_matrices(case, seed):
    g, dt = _gen(seed), DTYPES[case["dtype"]]
    shapes = _shapes(case)
    s = {"case": case, "shapes": shapes, "grads": []}
    for r, c in shapes:                  # noise and a few strong directions
        k = min(r, c, 4)
        strong = _randn(g, r, k) @ _randn(g, k, c)
        s["grads"].append(((_randn(g, r, c) + 0.5 * strong) * 1e-3).to(dt))
    if case["op"] == "orthogonalize":
        s["outs"] = [torch.empty(r, c, dtype=DTYPES[case["out"]], device=DEV) for r, c in shapes]
        return s
    numels = [r * c for r, c in shapes]
    s["off"], flat = _offsets(numels)
    s["numels"] = numels
    s["coef"] = torch.tensor([0.7310586], device=DEV)     # the clipping factor, a device word
    held = torch.zeros(flat, dtype=torch.bool, device=DEV)
    for o, n in zip(s["off"], numels):
        held[o:o + n] = True
    s["master"] = torch.where(held, _randn(g, flat) * 0.02, 0.0)
    s["m"] = torch.where(held, _randn(g, flat) * 5e-4, 0.0)
    s["params"] = s["master"].to(torch.bfloat16)
    return s


def _inputs(case, seed):
    if case["op"].startswith("embedding"):
        return _prepare_embedding(case, seed)
    return (_prepare_norm if case["op"] == "layer_norm" else _prepare_matrices)(case, seed)


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:                     # what a user's program keeps: workspaces and the optimizer
        import sharded_optimizer_step_gb300 as ss
        s["ss"] = ss
        if case["op"] == "embedding_grad":
            s["ws"] = ss.EmbeddingWorkspace(DEV)
        elif case["op"] == "layer_norm":
            s["ws"] = ss.LayerNormWorkspace(DEV)
        elif case["op"] == "orthogonalize":
            s["ws"] = ss.MatrixWorkspace(DEV)
            s["list"] = ss.TensorList(s["grads"])
        elif case["op"] == "muon":
            s["list"] = ss.TensorList(s["grads"])
            views = [s["params"][o:o + n].view(shape)
                     for o, n, shape in zip(s["off"], s["numels"], s["shapes"])]
            opt = ss.TensorMuon(views, ss.Muon(match_rms=RMS, **HP))
            opt.master.copy_(s.pop("master"))
            opt.m.copy_(s.pop("m"))
            s["opt"] = opt
    return s


# -------------------------------------------------------------------- plain

def _plain_embedding(s):
    case, ids, v = s["case"], s["ids"], s["case"]["vocab"]
    live = (ids >= 0) & (ids < v)
    if case["op"] == "embedding":
        rows = s["table"][torch.where(live, ids, 0)].float() * case["scale"]
        return {"out": torch.where(live[:, None], rows, 0.0).to(s["table"].dtype)}
    total = torch.zeros(v + 1, case["dim"], device=DEV)
    total.index_add_(0, torch.where(live, ids, v), s["d_out"].float())
    total = total[:v] * case["scale"]
    if case["accumulate"]:
        total = s["grad"].float() + total
    s["grad"] = total.to(s["grad"].dtype)
    return {"grad": s["grad"]}


def _plain_norm(s):
    x, dt = s["x"].float(), s["x"].dtype
    mean = x.mean(1, keepdim=True)
    xc = x - mean
    r = 1 / torch.sqrt(xc.square().mean(1, keepdim=True) + EPS)
    xh = xc * r
    out = {"out": (xh * s["w"] + s["b"]).to(dt), "mean": mean[:, 0], "rstd": r[:, 0]}
    if s["case"]["backward"]:
        d = s["d_out"].float()
        g = d * s["w"]
        out["d_x"] = (r * (g - g.mean(1, keepdim=True)
                           - xh * (g * xh).mean(1, keepdim=True))).to(dt)
        out["d_w"], out["d_b"] = (d * xh).sum(0), d.sum(0)
    return out


def _orthogonal(u, norm):
    """The quintic iteration in u's type."""
    a, b, c = QUINTIC
    x = u / (norm + 1e-7)
    tall = x.shape[0] > x.shape[1]
    x = x.T if tall else x
    for _ in range(ROUNDS):
        y = x @ x.T
        x = a * x + (b * y + c * (y @ y)) @ x
    return x.T if tall else x


def _plain_orthogonalize(s):
    return {"outs": [_orthogonal(u.float(), u.float().norm()).to(o.dtype)
                     for u, o in zip(s["grads"], s["outs"])]}


def _plain_muon(s):
    lr, mu, wd = HP["lr"], HP["momentum"], HP["weight_decay"]
    master, m = torch.zeros_like(s["master"]), torch.zeros_like(s["m"])
    for grad, o, n, (r, c) in zip(s["grads"], s["off"], s["numels"], s["shapes"]):
        g = grad.float() * s["coef"]
        new = mu * s["m"][o:o + n].view(r, c) + (1 - mu) * g
        u = mu * new + (1 - mu) * g
        p = s["master"][o:o + n].view(r, c)
        p = p - (lr * wd) * p - (lr * RMS * math.sqrt(max(r, c))) * _orthogonal(u, u.norm())
        master[o:o + n], m[o:o + n] = p.reshape(-1), new.reshape(-1)
    s["master"], s["m"], s["params"] = master, m, master.to(torch.bfloat16)
    return {"master": master, "params": s["params"], "m": m}


# ---------------------------------------------------------------- the paths

def _own(s):
    case, ss = s["case"], s["ss"]
    if case["op"] == "embedding":
        return {"out": ss.embedding(s["table"], s["ids"], scale=case["scale"], out=s["out"])}
    if case["op"] == "embedding_grad":
        return {"grad": ss.embedding_grad(s["d_out"], s["ids"], s["grad"], scale=case["scale"],
                                          accumulate=case["accumulate"], workspace=s["ws"])}
    if case["op"] == "layer_norm":
        y = ss.layer_norm(s["x"], s["w"], s["b"], eps=EPS, out=s["out"])
        out = {"out": y.out, "mean": y.mean, "rstd": y.rstd}
        if case["backward"]:
            d = ss.layer_norm_grad(s["d_out"], s["x"], y.mean, y.rstd, s["w"], d_x=s["d_x"],
                                   d_weight=s["d_w"], d_bias=s["d_b"], workspace=s["ws"])
            out.update(d_x=d.d_x, d_w=d.d_weight, d_b=d.d_bias)
        return out
    if case["op"] == "orthogonalize":
        return {"outs": ss.orthogonalize(s["list"], out=s["outs"], workspace=s["ws"])}
    opt = s["opt"]
    opt.step(s["list"], grad_coef=s["coef"])
    return {"master": opt.master, "params": s["params"], "m": opt.m}


def run(s):
    if own:
        return _own(s)
    return {"embedding": _plain_embedding, "embedding_grad": _plain_embedding,
            "layer_norm": _plain_norm, "orthogonalize": _plain_orthogonalize,
            "muon": _plain_muon}[s["case"]["op"]](s)


# -------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    """Row by row and matrix by matrix from the definitions, in double."""
    if case["op"] in ("orthogonalize", "muon") and work(case)["flops"] > 8e12:
        return None
    s = _inputs(case, seed)
    if case["op"].startswith("embedding"):
        return _exact_embedding(case, s)
    return (_exact_norm if case["op"] == "layer_norm" else _exact_matrices)(case, s)


def _exact_embedding(case, s):
    ids = s["ids"]
    live = torch.nonzero(ids >= 0)[:, 0]
    if case["op"] == "embedding":
        out = torch.zeros(case["tokens"], case["dim"], dtype=torch.float64, device=DEV)
        out[live] = s["table"].index_select(0, ids[live]).double() * case["scale"]
        return {"out": out}
    total = (s["grad"].double() if case["accumulate"]
             else torch.zeros(s["grad"].shape, dtype=torch.float64, device=DEV))
    # runs of equal ids: differences of running sums over the sorted tokens, some columns at a time
    key, at = torch.sort(ids[live], stable=True)
    found, count = torch.unique_consecutive(key, return_counts=True)
    if not found.numel():
        return {"grad": total}
    last = count.cumsum(0) - 1
    for c in range(0, case["dim"], 256):
        run = s["d_out"][live[at], c:c + 256].double().cumsum(0)[last]
        run[1:] -= run[:-1].clone()
        total[found, c:c + 256] += case["scale"] * run
    return {"grad": total}


def _exact_norm(case, s):
    rows, cols = case["rows"], case["cols"]
    keep = {k: [] for k in ("out", "mean", "rstd", "d_x")}
    d_w = torch.zeros(cols, dtype=torch.float64, device=DEV)
    d_b = torch.zeros_like(d_w)
    w, b = s["w"].double(), s["b"].double()
    for i in range(0, rows, 1024):
        x = s["x"][i:i + 1024].double()
        mu = x.sum(1) / cols
        var = ((x - mu[:, None]) ** 2).sum(1) / cols
        r = (var + EPS) ** -0.5
        xh = (x - mu[:, None]) * r[:, None]
        keep["out"].append(xh * w + b)
        keep["mean"].append(mu)
        keep["rstd"].append(r)
        if case["backward"]:
            d = s["d_out"][i:i + 1024].double()
            g = d * w
            c1, c2 = g.sum(1) / cols, (g * xh).sum(1) / cols
            keep["d_x"].append((g - c1[:, None] - xh * c2[:, None]) * r[:, None])
            d_w += (d * xh).sum(0)
            d_b += d.sum(0)
    out = {k: torch.cat(v) for k, v in keep.items() if v}
    return {**out, "d_w": d_w, "d_b": d_b} if case["backward"] else out


def _exact_matrices(case, s):
    def orthogonal(u):
        a, b, c = QUINTIC
        x = u / (torch.sqrt((u * u).sum()) + 1e-7)
        tall = x.shape[0] > x.shape[1]     # the short side's products, from the other side
        for _ in range(ROUNDS):
            y = x.T @ x if tall else x @ x.T
            p = b * y + c * (y @ y)
            x = a * x + (x @ p if tall else p @ x)
        return x

    if case["op"] == "orthogonalize":
        return {"outs": [orthogonal(u.double()) for u in s["grads"]]}
    master, m = s["master"].double(), s["m"].double()
    mu = HP["momentum"]
    for grad, o, n, (r, c) in zip(s["grads"], s["off"], s["numels"], s["shapes"]):
        g = grad.double() * s["coef"].double()
        new = m[o:o + n].view(r, c) * mu + g * (1 - mu)
        p = master[o:o + n].view(r, c) * (1 - HP["lr"] * HP["weight_decay"])
        p -= HP["lr"] * RMS * max(r, c) ** 0.5 * orthogonal(new * mu + g * (1 - mu))
        master[o:o + n], m[o:o + n] = p.reshape(-1), new.reshape(-1)
    return {"master": master, "params": master, "m": m}
