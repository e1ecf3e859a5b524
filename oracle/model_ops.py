"""Embedding, layer norm and the orthogonalised step of matrices in plain
numpy, in float64: the definitions the kernels are held to."""
import numpy as np

QUINTIC = (3.4445, -4.7750, 2.0315)


def embedding(table, ids, scale=1.0):
    """Rows of the table times scale; ids outside it give zeros."""
    out = np.zeros((len(ids), table.shape[1]))
    for i, v in enumerate(ids):
        if 0 <= v < table.shape[0]:
            out[i] = np.float64(scale) * table[v].astype(np.float64)
    return out


def embedding_grad(d_out, ids, vocab, scale=1.0):
    grad = np.zeros((vocab, d_out.shape[1]))
    for i, v in enumerate(ids):
        if 0 <= v < vocab:
            grad[v] += np.float64(scale) * d_out[i].astype(np.float64)
    return grad


def layer_norm(x, weight=None, bias=None, eps=1e-5):
    """(out, mean, rstd) over the rows of x."""
    x = x.astype(np.float64)
    mean = x.mean(1)
    rstd = 1.0 / np.sqrt(((x - mean[:, None]) ** 2).mean(1) + eps)
    out = (x - mean[:, None]) * rstd[:, None]
    if weight is not None:
        out = out * weight
    if bias is not None:
        out = out + bias
    return out, mean, rstd


def layer_norm_grad(d_out, x, mean, rstd, weight=None):
    """(d_x, d_weight, d_bias)."""
    d = d_out.astype(np.float64)
    xh = (x.astype(np.float64) - mean[:, None]) * rstd[:, None]
    g = d if weight is None else d * weight
    d_x = rstd[:, None] * (g - g.mean(1, keepdims=True) - xh * (g * xh).mean(1, keepdims=True))
    return d_x, (d * xh).sum(0), d.sum(0)


def orthogonalize(u, rounds=5, coefficients=QUINTIC, eps=1e-7):
    a, b, c = coefficients
    x = u.astype(np.float64)
    x = x / (np.sqrt((x * x).sum()) + eps)
    tall = x.shape[0] > x.shape[1]
    x = x.T if tall else x
    for _ in range(rounds):
        g = x @ x.T
        x = a * x + (b * g + c * g @ g) @ x
    return x.T if tall else x


def muon_scale(rows, cols, match_rms):
    return match_rms * np.sqrt(max(rows, cols)) if match_rms > 0 else np.sqrt(max(1.0, rows / cols))


def muon_step(p, m, grad, lr, momentum, weight_decay, match_rms, nesterov=True, rounds=5,
              coefficients=QUINTIC, eps=1e-7):
    """(p, m) after one step."""
    g = grad.astype(np.float64)
    m = momentum * m + (1 - momentum) * g
    u = momentum * m + (1 - momentum) * g if nesterov else m
    p = p - lr * weight_decay * p
    return p - lr * muon_scale(*p.shape, match_rms) * orthogonalize(u, rounds, coefficients, eps), m
