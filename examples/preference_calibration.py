"""Trains a small next-token model on paired answers, takes a policy step from its
logits, and calibrates its reward margins.

The model is a table of logits by the token before (a bigram model), so that its
gradient is the loss operators' own, summed by row.  One pass of training is

    logits -> token_logp -> pref_loss -> token_logp_vjp -> update ,

one policy step is policy_loss_logits in the logits' place, and the margins
reward(chosen) - reward(rejected) of pairs with noisy labels become the
probability that the first answer is preferred, a non-decreasing curve
(calib_curve).

    python examples/preference_calibration.py
"""
from __future__ import annotations

import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

VOCAB = 31
BETA = 0.3


def answers(torch, gen, pairs, table, flip):
    """Packed answers of 4 to 40 tokens in pairs, the better one (by the true table)
    first except where labels are flipped: (before, token, offsets, better first)."""
    length = torch.randint(4, 41, (2 * pairs,), generator=gen, device="cuda")
    off = torch.cat([length.new_zeros(1), length.cumsum(0)])
    n = int(off[-1])
    token = torch.randint(0, VOCAB, (n,), generator=gen, device="cuda")
    before = torch.roll(token, 1)
    before[off[:-1]] = 0
    quality = torch.zeros(2 * pairs, device="cuda").index_add_(
        0, torch.repeat_interleave(torch.arange(2 * pairs, device="cuda"), length), table[before, token])
    better = quality[0::2] > quality[1::2]
    better ^= torch.rand(pairs, generator=gen, device="cuda") < flip
    return before, token.to(torch.int32), off.to(torch.int32), better


def swap(torch, token_seq, off, better):
    """The places of the tokens with each pair's preferred answer first."""
    first = torch.arange(0, off.numel() - 1, 2, device="cuda")
    seq = torch.stack([torch.where(better, first, first + 1), torch.where(better, first + 1, first)], 1).reshape(-1)
    length = (off[1:] - off[:-1]).long()[seq]
    start = off[:-1].long()[seq]
    new = torch.cat([length.new_zeros(1), length.cumsum(0)])
    at = torch.arange(int(new[-1]), device="cuda") - torch.repeat_interleave(new[:-1], length)
    return torch.repeat_interleave(start, length) + at, new.to(torch.int32)


def margins(iso, model, ref, data):
    before, token, off, _ = data
    logp, _ = iso.token_logp(model[before], token)
    ref_logp, _ = iso.token_logp(ref[before], token)
    _, _, reward, _ = iso.pref_loss(logp, ref_logp, off, beta=BETA, grad=False)
    return (reward[0::2] - reward[1::2]).double()


def main(steps=40, pairs=2000, rate=10.0, seed=0, out=print):
    import torch

    from lower_convex_hull_amd import iso

    gen = torch.Generator(device="cuda").manual_seed(seed)
    table = torch.randn(VOCAB, VOCAB, generator=gen, device="cuda")
    ref = 0.1 * torch.randn(VOCAB, VOCAB, generator=gen, device="cuda")
    model = ref.clone()
    before, token, off, better = answers(torch, gen, pairs, table, 0.1)
    at, off = swap(torch, token, off, better)
    before, token = before[at], token[at]
    ref_logp, _ = iso.token_logp(ref[before], token)
    trained = []
    for _ in range(steps):
        logits = model[before]
        logp, lse = iso.token_logp(logits, token)
        loss, _, _, g = iso.pref_loss(logp, ref_logp, off, beta=BETA)
        grad = iso.token_logp_vjp(g, logits, token, lse, out=logits)
        model.index_add_(0, before, grad, alpha=-rate)
        trained.append(loss)
    trained = torch.stack(trained).tolist()
    out(f"preference loss {trained[0]:.4f} -> {trained[-1]:.4f}")

    # a step of the clipped policy loss, whole from the logits: the preferred answers are the better actions
    logits = model[before]
    old, _ = iso.token_logp(logits, token)
    adv = torch.ones(2 * pairs, device="cuda")
    adv[1::2] = -1.0
    kw = dict(ref_logp=ref_logp, seq_off=off, kl_coef=0.02, seq_mean=True)
    loss, counts, _, grad = iso.policy_loss_logits(logits, token, old, adv, out=logits, **kw)
    stepped = model.clone().index_add_(0, before, grad, alpha=-rate)
    after, counts, _, _ = iso.policy_loss_logits(stepped[before], token, old, adv, grad=False, **kw)
    out(f"policy loss {float(loss[0]):.4f} -> {float(after[0]):.4f}, {int(counts[1])} of {int(counts[0])} tokens clipped")

    # margins of fresh pairs and how often the first answer is preferred
    fresh = answers(torch, gen, 4 * pairs, table, 0.1)
    margin = margins(iso, model, ref, fresh)
    xp, fp = iso.calib_curve(margin, fresh[3].double())
    raw = torch.sigmoid(margin)
    fitted = fp[torch.searchsorted(xp, margin)]
    brier = [float(((p - fresh[3].double()) ** 2).mean()) for p in (raw, fitted)]
    right = float(((margin > 0) == fresh[3]).double().mean())
    out(f"{right:.3f} of fresh pairs ordered; squared error of the probability {brier[0]:.4f} raw, {brier[1]:.4f} calibrated")
    return {"trained": trained, "policy": (float(loss[0]), float(after[0])), "right": right, "brier": brier,
            "curve": (xp, fp)}


if __name__ == "__main__":
    main()
