"""Tuning a small language model whose vocabulary table is also its head, with the
clipped policy loss: every gradient formed and stepped on one GPU.

  embedding                   the tokens' rows of the table
  layer_norm                  of them
  (two hidden matrices)       products in torch, a residual around them
  (the head)                  the table again, a product in torch
  policy_loss                 the loss and its gradient in the logits
  layer_norm_grad             with the weight's and the bias's gradient
  embedding_grad              added to the head's gradient of the same table
  grad_norm_clip              the global norm, the clipping factor, the found-inf word
  TensorMuon.step             the hidden matrices, orthogonalised momentum
  TensorAdamW.step            the table and the norm's vectors
  GradScaler.update

and nothing waits for the host between the first and the last.  Run:

    python examples/tied_model_tuning.py [--steps 20]
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import sharded_optimizer_step_gb300 as ss  # noqa: E402

NAMES = ("table", "norm_w", "norm_b", "up", "down")


def parameters(vocab, hidden, gen, dtype=torch.bfloat16, device="cuda"):
    """The model's tensors by name."""
    rand = lambda *s: torch.randn(*s, generator=gen, device=device)  # noqa: E731
    return {"table": (rand(vocab, hidden) * 0.05).to(dtype),
            "norm_w": torch.ones(hidden, device=device).to(dtype),
            "norm_b": torch.zeros(hidden, device=device).to(dtype),
            "up": (rand(4 * hidden, hidden) * hidden ** -0.5).to(dtype),
            "down": (rand(hidden, 4 * hidden) * (4 * hidden) ** -0.5).to(dtype)}


def forward(p, prev):
    """The logits after the tokens `prev` (-1: padding), and what backward needs."""
    h = ss.embedding(p["table"], prev, scale=p["table"].shape[1] ** 0.5)
    y = ss.layer_norm(h, p["norm_w"], p["norm_b"])
    a = torch.tanh(y.out @ p["up"].T)
    r = h + a @ p["down"].T
    return r @ p["table"].T, (h, y, a, r)


def backward(p, prev, kept, d_logits, grads, spaces, accumulate=False):
    """The gradients of all tensors, into `grads` by name."""
    h, y, a, r = kept
    put = lambda name, g: grads[name].add_(g) if accumulate else grads[name].copy_(g)  # noqa: E731
    put("table", d_logits.T @ r)
    d_r = d_logits @ p["table"]
    put("down", d_r.T @ a)
    d_pre = ((d_r @ p["down"]).float() * (1 - a.float() ** 2)).to(a.dtype)
    put("up", d_pre.T @ y.out)
    d = ss.layer_norm_grad(d_pre @ p["up"], h, y.mean, y.rstd, p["norm_w"],
                           d_x=torch.empty_like(h), d_weight=grads["norm_w"],
                           d_bias=grads["norm_b"], accumulate=accumulate, workspace=spaces[0])
    # the same table: added to the head's gradient
    ss.embedding_grad(d_r + d.d_x, prev, grads["table"], scale=p["table"].shape[1] ** 0.5,
                      accumulate=True, workspace=spaces[1])


def tune(steps=20, tokens=512, hidden=128, vocab=3000, seed=0, device="cuda"):
    """Each step's mean reward and loss."""
    gen = torch.Generator(device=device).manual_seed(seed)
    p = parameters(vocab, hidden, gen, device=device)
    grads = {k: torch.zeros_like(v) for k, v in p.items()}
    muon = ss.TensorMuon([p["up"], p["down"]], ss.Muon(lr=2e-3))
    adamw = ss.TensorAdamW([p[k] for k in NAMES[:3]],
                           [ss.AdamW(lr=2e-3, beta2=0.95),
                            ss.AdamW(lr=2e-3, beta2=0.95, weight_decay=0.0)], groups=[0, 1, 1])
    every = ss.TensorList([grads[k] for k in NAMES])
    matrices = ss.TensorList([grads["up"], grads["down"]])
    others = ss.TensorList([grads[k] for k in NAMES[:3]])
    scaler = ss.GradScaler(init_scale=256.0, device=device)
    loss_ws, norm_ws = ss.LossWorkspace(device), ss.NormWorkspace(device)
    spaces = (ss.LayerNormWorkspace(device), ss.EmbeddingWorkspace(device))
    good = torch.arange(vocab, device=device) % 7 == 3      # the tokens that are rewarded
    rewards, losses = [], []
    for _ in range(steps):
        prev = torch.randint(0, vocab, (tokens,), generator=gen, device=device)
        prev[::16] = -1                                     # padding
        logits, kept = forward(p, prev)
        logp = torch.log_softmax(logits.float(), 1)
        ids = torch.multinomial(logp.exp(), 1, generator=gen)[:, 0]
        reward = good[ids].float()
        weights = (prev >= 0).float()
        old = logp.gather(1, ids[:, None])[:, 0].contiguous()
        out = ss.policy_loss(logits, ids, old, reward - reward.mean(), weights=weights,
                             grad=logits, loss_scale=scaler.scale, workspace=loss_ws)
        backward(p, prev, kept, logits, grads, spaces)
        clip = ss.grad_norm_clip(every, 1.0, loss_scale=scaler.scale, found_inf=scaler.found_inf,
                                 workspace=norm_ws)
        muon.step(matrices, grad_coef=clip[1:], skip=scaler.found_inf)
        adamw.step(others, grad_coef=clip[1:], skip=scaler.found_inf)
        scaler.update()
        rewards.append(reward.mean())
        losses.append(out.stats[0])
    return torch.stack(rewards).tolist(), torch.stack(losses).tolist()


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=20)
    args = ap.parse_args()
    for t, (r, l) in enumerate(zip(*tune(steps=args.steps))):
        print(f"step {t:3d}  mean reward {r:.3f}  loss {l:+.4f}")
