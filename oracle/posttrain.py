"""fp64 definitions of the post-training losses and of Muon's update (CPU, tests only).

They share no code with the GPU path. The losses work on logits [N, Vp] of which
the first V columns are real ids, and return the gradient of dscale * sum(losses).
"""
from __future__ import annotations

import numpy as np

from .gpt2 import F64, KINDS, KIND_NAMES, clip_adamw, global_norm, lr_at

NS_COEFFS = (3.4445, -4.7750, 2.0315)
MUON_KINDS = ("qkvw", "attprojw", "fcw", "fcprojw")


def token_logps(z, targets, V, ignore_index=-1):
    """(lp [N], p [N, V], keep [N]): log-probabilities of the targets, 0 where ignored."""
    z = np.asarray(z, F64)[:, :V]
    keep = targets != ignore_index
    t = np.where(keep, targets, 0)
    m = z.max(axis=1, keepdims=True)
    e = np.exp(z - m)
    s = e.sum(axis=1, keepdims=True)
    lp = z[np.arange(len(t)), t] - m[:, 0] - np.log(s[:, 0])
    return np.where(keep, lp, 0.0), e / s, keep


def logit_gradient(p, targets, keep, g, Vp):
    """dz[i, j] = g[i] ([j = t_i] - p[i, j]) for kept rows, 0 elsewhere and for padded columns."""
    dz = np.zeros((p.shape[0], Vp))
    dz[:, :p.shape[1]] = -g[:, None] * p
    rows = np.flatnonzero(keep)
    dz[rows, targets[rows]] += g[rows]
    dz[~keep] = 0.0
    return dz


def policy_rows(lp, old, adv, ref, w, clip_low, clip_high, kl):
    """Per-row loss and its derivative by lp; an advantage of 0 gives 0 for any ratio, any other NaN is a NaN in both."""
    with np.errstate(invalid="ignore", over="ignore"):
        r = np.exp(lp - old)
        none = (adv == 0) & ~np.isnan(lp)
        free = np.where(none, 0.0, r * adv)
        cut = np.where(none, 0.0, np.clip(r, 1 - clip_low, 1 + clip_high) * adv)
    loss = -np.minimum(free, cut)
    g = np.where(free > cut, 0.0, -free)
    if ref is not None and kl:
        d = ref - lp
        # e^d grows past d: +inf where d is
        loss = loss + kl * (np.expm1(d) - np.minimum(d, np.finfo(F64).max))
        g = g - kl * np.expm1(d)
    return w * loss, w * g


def policy_loss(z, targets, V, old, adv, ref=None, weight=None, ignore_index=-1, clip_low=0.2, clip_high=0.2,
                kl=0.0, dscale=1.0):
    """(losses [N], lp [N], dz [N, Vp])."""
    lp, p, keep = token_logps(z, targets, V, ignore_index)
    w = np.ones(len(lp)) if weight is None else np.asarray(weight, F64)
    loss, g = policy_rows(lp, np.asarray(old, F64), np.asarray(adv, F64),
                          None if ref is None else np.asarray(ref, F64), w, clip_low, clip_high, kl)
    loss, g = np.where(keep, loss, 0.0), np.where(keep, g, 0.0) * dscale
    return loss, lp, logit_gradient(p, targets, keep, g, z.shape[1])


def pair_loss(delta, kind, beta, smoothing):
    """The pair's loss and its derivative by the margin."""
    if kind == "sigmoid":
        loss = (1 - smoothing) * np.logaddexp(0, -beta * delta)
        if smoothing:                                      # (0 of an infinite loss is 0)
            loss = loss + smoothing * np.logaddexp(0, beta * delta)
        d = -beta * ((1 - smoothing) * np.exp(-np.logaddexp(0, beta * delta))
                     - smoothing * np.exp(-np.logaddexp(0, -beta * delta)))
        return loss, d
    off = delta - 1 / (2 * beta)
    return off * off, 2 * off


def preference_loss(z, targets, V, seq_start, ref=None, ignore_index=-1, kind="sigmoid", average=False, beta=0.1,
                    smoothing=0.0, dscale=1.0):
    """(losses [P], seq_logps [2P], lp [N], dz [N, Vp]); rows in no sequence get gradient 0 here."""
    lp, p, keep = token_logps(z, targets, V, ignore_index)
    S = len(seq_start) - 1
    score, share = np.zeros(S), np.ones(S)
    for i in range(S):
        rows = slice(seq_start[i], seq_start[i + 1])
        n = int(keep[rows].sum())
        share[i] = 1.0 / max(n, 1) if average else 1.0
        score[i] = lp[rows].sum() * share[i]
    gap = score - (0.0 if ref is None else np.asarray(ref, F64))
    losses, d = pair_loss(gap[0::2] - gap[1::2], kind, beta, smoothing)
    g = np.zeros(len(lp))
    for i in range(S):
        g[seq_start[i]:seq_start[i + 1]] = (d[i // 2] if i % 2 == 0 else -d[i // 2]) * share[i] * dscale
    g = np.where(keep, g, 0.0)
    return losses, score, lp, logit_gradient(p, targets, keep, g, z.shape[1])


def newton_schulz(x, steps=5):
    """The quintic Newton-Schulz rounds on x / (|x|_F + 1e-7)."""
    a, b, c = NS_COEFFS
    y = np.asarray(x, F64)
    tall = y.shape[0] > y.shape[1]
    y = y.T if tall else y
    y = y / (np.linalg.norm(y) + 1e-7)
    for _ in range(steps):
        g = y @ y.T
        y = a * y + (b * g + c * (g @ g)) @ y
    return y.T if tall else y


def clip_muon(cfg, params, grads, m, v, step, accum=1, momentum=0.95):
    """Muon for the blocks' 2-D weights, clip_adamw for everything else; in place, returns the norm."""
    norm = global_norm(grads, accum)
    scale = min(1.0, cfg.grad_clip / norm) if norm > 0 else 1.0
    lr = lr_at(cfg, step)
    keep = {n: (np.array(params[n], F64), np.array(m[n], F64), v[n]) for n in MUON_KINDS}
    clip_adamw(cfg, params, grads, m, v, step, accum)
    for name in MUON_KINDS:
        w, mk, v[name] = keep[name]
        g = np.asarray(grads[name], F64) / accum * scale
        mk = momentum * mk + g
        u = g + momentum * mk
        new = np.empty_like(w)
        for l in range(w.shape[0]):
            o = newton_schulz(u[l])
            new[l] = w[l] - lr * (0.2 * np.sqrt(max(o.shape)) * o + cfg.weight_decay * w[l])
        params[name], m[name] = new, mk
    return norm


assert set(MUON_KINDS) <= {n for n in KIND_NAMES} and all(is2d for n, _, is2d, _ in KINDS if n in MUON_KINDS)
