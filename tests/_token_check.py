"""A tight check of the token losses' log probabilities and gradients: every
element against its own size.  torch in float64, on whatever device the logits are.

Derivation, in units of the log probability a = x_y - log(sum exp x):
  T   an exponential's argument is rounded twice at its own size, 2^-24 |x_j - x_y|
      + 2^-24 each (the id's own argument is at most 1/2), and the softmax weighs
      these; the base-2 exponential is 2^-22 off at most, and the sum of V of them,
      added in hundreds of chains side by side, less than that: T = 2^-23 (E_p|x - x_y|
      + 1) + 2^-21.
  a   T, and 2^-24 |a| where it is written as one float.
  c   what the caller says: its sensitivity to a times T, and its own roundings.
  gradient of element j: p_j (|c| (T + 2^-23 (|x_j - x_y| + 1) + 2^-22) + error of c), of
      the id's own also error of c + 2^-23 |c|; one rounding to its type, and the
      type's smallest step.
"""
import torch

ROUND = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
# bf16 and fp32 below 2^-126 may be flushed; fp16's subnormals are rounded to
STEP = {torch.bfloat16: 2.0 ** -126, torch.float16: 2.0 ** -24, torch.float32: 2.0 ** -126}
CHUNK = 64


def row_facts(x, ids):
    """The rows' log probabilities and their T, float64."""
    a, t = [], []
    for i in range(0, x.shape[0], CHUNK):
        z = x[i:i + CHUNK].double()
        xy = z.gather(1, ids[i:i + CHUNK, None])
        lse = torch.logsumexp(z, 1, keepdim=True)
        a.append((xy - lse)[:, 0])
        mean = (torch.exp(z - lse) * (z - xy).abs()).sum(1)
        t.append(2.0 ** -23 * (mean + 1) + 2.0 ** -21)
    return torch.cat(a), torch.cat(t)


def gradient_misses(got, x, ids, c, slack, t):
    """Of each row, how many elements of `got` are outside the bound around
    c (1[y] - softmax x); c, slack (the error of c) and t per row."""
    out = []
    for i in range(0, x.shape[0], CHUNK):
        z, y = x[i:i + CHUNK].double(), ids[i:i + CHUNK, None]
        cc, ss, tt = (q[i:i + CHUNK, None] for q in (c, slack, t))
        p = torch.softmax(z, 1)
        want, size = -cc * p, cc.abs()
        bound = p * (size * (tt + 2.0 ** -22 + 2.0 ** -23 * (1 + (z - z.gather(1, y)).abs())) + ss)
        want.scatter_add_(1, y, cc)
        bound.scatter_add_(1, y, ss + 2.0 ** -23 * size)
        bound += ROUND[got.dtype] * (want.abs() + bound) + STEP[got.dtype]
        out.append((~((got[i:i + CHUNK].double() - want).abs() <= bound)).sum(1))
    return torch.cat(out)


def policy(a, t, old, adv, ref, w, kl, norm, scale=1.0, low=0.2, high=0.2):
    """(stats, their errors, c, error of c) of the policy loss, from the rows' a."""
    live = w != 0
    k = torch.where(live, w / norm, 0.0)
    a = torch.where(live, a, old)
    u = torch.exp(a - old)
    best = torch.clamp(u, 1 - low, 1 + high) * adv
    held = u * adv > best
    d = torch.where(live, ref - a, 0.0)
    term, kls = -torch.minimum(u * adv, best), torch.expm1(d) - d
    slope = torch.where(held, 0.0, -u * adv)
    moves = torch.where(held, 0.0, (u * adv).abs())
    if kl:
        slope = slope - kl * torch.expm1(d)
        moves = moves + kl * torch.exp(d)
    c = k * slope * scale
    # logp - old (and ref - logp) round once at their size, exp and expm1 to 2^-22
    off = t + 2.0 ** -24 * ((a - old).abs() + d.abs()) + 2.0 ** -21
    slack = k.abs() * moves * off * scale + 2.0 ** -21 * c.abs()
    terms = torch.stack([term + kl * kls, term, kls if kl else 0 * kls, held.double()])
    # the policy term's own sensitivity to a is |u A| whether held or not
    rough = k.abs() * ((u * adv).abs() + (torch.exp(d) + 1)) * off
    errors = rough.sum() + 2.0 ** -21 * (terms.abs() * k.abs()).sum(1)
    return (terms * k).sum(1), errors, c, slack


def preference(a, t, lens, ref, w, beta, smoothing, norm, scale=1.0):
    """(stats, errors, log ratios, errors, c, error of c) of the preference loss."""
    live = w != 0
    dev = a.device
    seq = torch.repeat_interleave(torch.arange(len(lens), device=dev),
                                  torch.tensor(lens, device=dev))
    zero = torch.zeros(len(lens), dtype=torch.float64, device=dev)
    part = torch.where(live, w * (a - ref), 0.0)
    off = torch.where(live, w.abs() * (t + 2.0 ** -22 * (a - ref).abs()), 0.0)
    r, roff = zero.index_add(0, seq, part), zero.index_add(0, seq, off)
    h, hoff = beta * (r[0::2] - r[1::2]), abs(beta) * (roff[0::2] + roff[1::2])
    hoff = hoff + 2.0 ** -22 * h.abs()
    sp = torch.nn.functional.softplus
    loss = (1 - smoothing) * sp(-h) + smoothing * sp(h)
    slope = smoothing * torch.sigmoid(h) - (1 - smoothing) * torch.sigmoid(-h)
    sign = torch.ones(len(lens), dtype=torch.float64, device=dev)
    sign[1::2] = -1
    pair = torch.arange(len(lens), device=dev) // 2
    c = (sign * slope[pair])[seq] * w * (beta / norm) * scale
    slack = (hoff[pair] / 4)[seq] * w.abs() * abs(beta / norm) * scale + 2.0 ** -20 * c.abs()
    stats = torch.stack([loss.sum(), h.sum(), (h > 0).double().sum()]) / norm
    errors = torch.stack([hoff.sum() + 2.0 ** -21 * loss.abs().sum(),
                          hoff.sum() + 2.0 ** -21 * h.abs().sum(), 1e-6 + zero.sum()]) / norm
    return stats, errors, r, roff + 2.0 ** -22 * r.abs(), c, slack
