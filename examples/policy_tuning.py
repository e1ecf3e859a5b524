"""Tuning a small language-model head with the clipped policy loss, data
parallel, on one GPU.

N_d emulated ranks each sample answers from the current policy, score them,
and take M micro-batches through

  policy_loss                 the loss and its gradient in the logits, scaled
                              by the gradient scaler's word on the device
  (the model's backward)      two matrix products per micro-batch, in torch
  fsdp_grad_accumulate        fp32 sums over the micro-batches
  ddp_bucket_allreduce_avg    the ranks' mean, in buckets
  grad_norm_clip              the global norm, the clipping factor and the
                              found-inf word, on the device
  TensorAdamW.step            AdamW with 8-bit moments on the clipped,
                              unscaled gradient, left out on a non-finite norm
  GradScaler.update

and nothing waits for the host between the first and the last.  Run:

    python examples/policy_tuning.py [--steps 20] [--state-bits 8]
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import sharded_optimizer_step_gb300 as ss  # noqa: E402


def tune(steps=20, nd=4, micro=2, tokens=192, hidden=256, vocab=2000, state_bits=8, seed=0,
         device="cuda"):
    """Returns the mean reward of each step's samples and the losses."""
    gen = torch.Generator(device=device).manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=gen, device=device)  # noqa: E731
    # a hidden layer's output projection, the head, and a norm vector without decay
    params = [(rand(hidden, hidden) * hidden ** -0.5).bfloat16(),
              (rand(vocab, hidden) * 0.02).bfloat16(),
              torch.ones(hidden, device=device).bfloat16()]
    hps = [ss.AdamW(lr=2e-3, beta2=0.95), ss.AdamW(lr=2e-3, beta2=0.95, weight_decay=0.0)]
    opt = ss.TensorAdamW(params, hps, groups=[0, 0, 1], state_bits=state_bits)
    scaler = ss.GradScaler(init_scale=256.0, device=device)
    numels = [p.numel() for p in params]
    place, _, offsets = ss.ddp_bucket_plan(numels, 2, 1 << 20)
    total = sum(numels)
    flat = lambda dt: torch.zeros(total, dtype=dt, device=device)  # noqa: E731
    rank_grads = [flat(torch.bfloat16) for _ in range(nd)]
    acc, piece, mean = flat(torch.float32), flat(torch.bfloat16), flat(torch.bfloat16)
    grads = ss.TensorList([mean[o:o + n] for o, n in zip(place, numels)])
    loss_ws, norm_ws = ss.LossWorkspace(device), ss.NormWorkspace(device)
    d_logits = torch.empty(tokens, vocab, dtype=torch.bfloat16, device=device)
    common = rand(hidden)                                   # what all prompts share
    good = torch.arange(vocab, device=device) % 7 == 3      # the tokens that are rewarded
    rewards, losses = [], []

    def forward(x):
        h = torch.tanh(x @ params[0].T) * params[2]
        return h, h @ params[1].T

    for _ in range(steps):
        reward = torch.zeros((), device=device)
        loss = torch.zeros(4, device=device)
        for q in range(nd):
            # the rank's prompts, its samples of the current policy, their rewards
            batches = []
            for _ in range(micro):
                x = (common + 0.5 * rand(tokens, hidden)).bfloat16()
                logp = torch.log_softmax(forward(x)[1].float(), 1)
                ids = torch.multinomial(logp.exp(), 1, generator=gen)[:, 0]
                adv = good[ids].float()
                reward += adv.mean() / (nd * micro)
                old = logp.gather(1, ids[:, None])[:, 0]
                w = (torch.arange(tokens, device=device) % 8 != 0).float()   # prompt tokens
                batches.append((x, ids, old.contiguous(), adv - adv.mean(), w))
            count = float(sum(int(tokens - (tokens + 7) // 8) for _ in batches))
            for m, (x, ids, old, adv, w) in enumerate(batches):
                h, logits = forward(x)
                out = ss.policy_loss(logits, ids, old, adv, ref_logps=old, kl_coef=0.01,
                                     weights=w, norm=count, grad=d_logits,
                                     loss_scale=scaler.scale, workspace=loss_ws)
                loss += out.stats / nd
                d_h = d_logits @ params[1]
                d_pre = (d_h * params[2]).float() * (1 - torch.tanh((x @ params[0].T).float()) ** 2)
                for g, o, n in zip((d_pre.bfloat16().T @ x, d_logits.T @ h,
                                    (d_h * torch.tanh(x @ params[0].T)).sum(0)), place, numels):
                    piece[o:o + n].copy_(g.reshape(-1))
                ss.fsdp_grad_accumulate(piece, acc, 1.0, first=m == 0)
            rank_grads[q].copy_(acc)
        ss.ddp_bucket_allreduce_avg(rank_grads, offsets, mean)
        clip = ss.grad_norm_clip(grads, 1.0, loss_scale=scaler.scale,
                                 found_inf=scaler.found_inf, workspace=norm_ws)
        opt.step(grads, grad_coef=clip[1:], skip=scaler.found_inf)
        scaler.update()
        rewards.append(reward)
        losses.append(loss[0])
    return torch.stack(rewards).tolist(), torch.stack(losses).tolist()


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--state-bits", type=int, default=8, choices=(8, 32))
    args = ap.parse_args()
    for t, (r, l) in enumerate(zip(*tune(steps=args.steps, state_bits=args.state_bits))):
        print(f"step {t:3d}  mean reward {r:.3f}  loss {l:+.4f}")
