"""Speed cases of the post-training operators: the clipped policy loss and the paired
preference loss over a head's logits (each with its gradient), and the Newton-Schulz
orthogonalisation of weight-shaped matrices.

`listed()` and `draw()` give cases, `prepare()` a case's inputs on the GPU, `run()` one
pass: with `own` false in elementary torch operations, with `own` true through
`gpt_step_b200`. `exact()` is the definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

IGNORE = -1
NS = (3.4445, -4.7750, 2.0315)   # coefficients of the quintic Newton-Schulz step


def listed():
    return [
        # one step of reinforcement on the smallest configuration: 4 sequences of 64 over 1,000 ids; latency counts
        {"name": "policy 256 x 1000", "op": "policy", "N": 256, "T": 64, "V": 1000, "Vp": 1024,
         "masked": 0.0, "kl": 0.0, "weighted": False},
        # a packed, odd-sized batch with its prompts masked and one weight a row (1 / answer length)
        {"name": "policy 333 x 4353", "op": "policy", "N": 333, "T": 111, "V": 4353, "Vp": 4480,
         "masked": 0.5, "kl": 0.04, "weighted": True},
        # the small configuration's whole batch: 16 sequences of 1,024
        {"name": "policy 16384 x 4353", "op": "policy", "N": 16384, "T": 1024, "V": 4353, "Vp": 4480,
         "masked": 0.25, "kl": 0.04, "weighted": False},
        # the 124M configuration's micro-batch: 19 sequences of 1,024 over 50,257 ids
        {"name": "policy 19456 x 50257", "op": "policy", "N": 19456, "T": 1024, "V": 50257, "Vp": 50304,
         "masked": 0.25, "kl": 0.04, "weighted": False},
        # two pairs of 64 rows on the smallest configuration; latency counts
        {"name": "preference 2 x 64 x 1000", "op": "preference", "P": 2, "T": 64, "V": 1000, "Vp": 1024,
         "masked": 0.0, "ragged": False, "kind": "sigmoid", "average": False},
        # three ragged pairs, answers only, the squared loss on mean log-probabilities
        {"name": "preference 3 x 201 x 8449", "op": "preference", "P": 3, "T": 201, "V": 8449, "Vp": 8576,
         "masked": 0.4, "ragged": True, "kind": "squared", "average": True},
        # the small configuration: eight ragged pairs of up to 1,024
        {"name": "preference 8 x 1024 x 4353", "op": "preference", "P": 8, "T": 1024, "V": 4353, "Vp": 4480,
         "masked": 0.3, "ragged": True, "kind": "sigmoid", "average": False},
        # the 124M configuration: nine pairs of 1,024, the prompts masked
        {"name": "preference 9 x 1024 x 50257", "op": "preference", "P": 9, "T": 1024, "V": 50257, "Vp": 50304,
         "masked": 0.3, "ragged": False, "kind": "sigmoid", "average": False},
        # one square projection of the smallest configuration; fifteen dependent products, latency counts
        {"name": "orthogonalize 1 x 128 x 128", "op": "orthogonalize", "batch": 1, "rows": 128, "cols": 128,
         "fp32": True},
        # odd sizes, bf16 gradients
        {"name": "orthogonalize 3 x 333 x 517", "op": "orthogonalize", "batch": 3, "rows": 333, "cols": 517,
         "fp32": False},
        # the QKV weights of the 124M configuration's twelve blocks, tall
        {"name": "orthogonalize 12 x 2304 x 768", "op": "orthogonalize", "batch": 12, "rows": 2304, "cols": 768,
         "fp32": True},
        # the MLP projections of the wide configuration's sixteen blocks
        {"name": "orthogonalize 16 x 1536 x 6144", "op": "orthogonalize", "batch": 16, "rows": 1536, "cols": 6144,
         "fp32": True},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["policy", "preference", "orthogonalize"])
    if op == "orthogonalize":
        batch, rows, cols = _log_int(rng, 1, 16), _log_int(rng, 16, 6144), _log_int(rng, 16, 6144)
        small = min(rows, cols)
        if small > 1536:      # no drawn case costs more than the largest listed one
            rows, cols = (1536, cols) if rows <= cols else (rows, 1536)
        return {"op": op, "batch": batch, "rows": rows, "cols": cols, "fp32": rng.random() < 0.5}
    V = _log_int(rng, 300, 50257)
    Vp = (V + 127) // 128 * 128 if rng.random() < 0.6 else (V + 7) // 8 * 8
    masked = rng.choice([0.0, rng.uniform(0.05, 0.9)])
    T = _log_int(rng, 2, 1024)
    if op == "policy":
        return {"op": op, "N": _log_int(rng, 1, 19) * T, "T": T, "V": V, "Vp": Vp, "masked": masked,
                "kl": rng.choice([0.0, 0.04]), "weighted": rng.random() < 0.5}
    return {"op": op, "P": _log_int(rng, 1, 9), "T": T, "V": V, "Vp": Vp, "masked": masked,
            "ragged": rng.random() < 0.6, "kind": rng.choice(["sigmoid", "sigmoid", "squared"]),
            "average": rng.random() < 0.3}


# -- inputs ------------------------------------------------------------------------------------


def _lens(case):
    """Rows of each of a preference case's 2 P sequences: T, or spread over a third of T to T."""
    P, T = case["P"], case["T"]
    if not case["ragged"]:
        return np.full(2 * P, T)
    return np.random.default_rng(1000 * P + T).integers(max(1, T // 3), T + 1, 2 * P)


def _logits(case, N, gen):
    """bf16 logits of a trained head: a spread of 2 over the vocabulary, the row's target well above it."""
    V, Vp = case["V"], case["Vp"]
    z = torch.empty(N, Vp, dtype=torch.bfloat16, device="cuda").normal_(0.0, 2.0, generator=gen)
    t = torch.randint(0, V, (N,), device="cuda", generator=gen)
    rows = torch.arange(N, device="cuda")
    up = math.log(V) + 2.0 + 2.0 * torch.randn(N, device="cuda", generator=gen)
    z[rows, t] = (z[rows, t].float() + up).to(torch.bfloat16)
    return z, t


def _row_logp64(z, t, V):
    """Each row's log-probability of its target, to the 64 bits of a value stored once and reused."""
    out = torch.empty(z.shape[0], dtype=torch.float64, device="cuda")
    for i in range(0, z.shape[0], 4096):
        zi = z[i:i + 4096, :V].float()
        lse = zi.logsumexp(1).double()
        out[i:i + 4096] = zi.gather(1, t[i:i + 4096, None])[:, 0].double() - lse
    return out


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case, "err": torch.zeros(1, dtype=torch.int32, device="cuda")}
    if case["op"] == "orthogonalize":
        # a momentum: singular values falling like 1 / k, the scale of a mean gradient
        b, r, c = case["batch"], case["rows"], case["cols"]
        k = min(r, c)
        u = torch.randn(b, r, k, device="cuda", generator=gen)
        v = torch.randn(b, k, c, device="cuda", generator=gen)
        d = 1.0 / torch.arange(1, k + 1, device="cuda", dtype=torch.float32)
        x = torch.empty(b, r, c, device="cuda")
        for i in range(b):
            x[i] = (u[i] * d) @ v[i]
        x *= 1e-3 / math.sqrt(k)
        s["x"] = x if case["fp32"] else x.to(torch.bfloat16)
        s["out"] = torch.empty(b, r, c, dtype=torch.bfloat16, device="cuda")
        return s
    V = case["V"]
    if case["op"] == "policy":
        N, T = case["N"], case["T"]
        z, t = _logits(case, N, gen)
        lp = _row_logp64(z, t, V)
        s.update(clip_low=0.2, clip_high=0.28, kl=case["kl"])
        # the sampling policy a few updates back; log-ratios next to a clip border are moved off it
        d = 0.15 * torch.randn(N, device="cuda", generator=gen, dtype=torch.float64)
        for edge in (math.log(1 - s["clip_low"]), math.log(1 + s["clip_high"])):
            d = torch.where((d - edge).abs() < 2e-3, d + 5e-3, d)
        s["old"] = (lp - d).float()
        s["ref"] = (lp + 0.3 * torch.randn(N, device="cuda", generator=gen, dtype=torch.float64)).float() \
            if case["kl"] else None
        seq = torch.arange(N, device="cuda") // T
        s["adv"] = torch.randn(N // T + 1, device="cuda", generator=gen)[seq].contiguous()
        prompt = (torch.arange(N, device="cuda") % T) < int(case["masked"] * T)
        kept = max(1, int((~prompt).sum()))
        if case["weighted"]:
            s["weight"] = torch.full((N,), 1.0 / max(1, T - int(case["masked"] * T)), device="cuda")
            s["dscale"] = T / N
        else:
            s["weight"], s["dscale"] = None, 1.0 / kept
    else:
        P, T = case["P"], case["T"]
        lens = _lens(case)
        start = np.concatenate([[0], np.cumsum(lens)])
        N = int(start[-1])
        z, t = _logits(case, N, gen)
        lp = _row_logp64(z, t, V)
        s["start"] = torch.tensor(start, dtype=torch.int32, device="cuda")
        at = torch.arange(N, device="cuda")
        seq = torch.searchsorted(s["start"][1:].long(), at, right=True)
        n = torch.tensor(lens, device="cuda")[seq]
        prompt = (at - s["start"].long()[seq]) < (case["masked"] * n).floor()
        sums = torch.zeros(2 * P, dtype=torch.float64, device="cuda").index_add_(0, seq, torch.where(prompt, 0.0, lp))
        if case["average"]:
            count = torch.zeros(2 * P, dtype=torch.float64, device="cuda").index_add_(0, seq, (~prompt).double())
            sums = sums / count.clamp(min=1)
        spread = 0.3 if case["average"] else 5.0
        noise = torch.randn(2 * P, device="cuda", generator=gen, dtype=torch.float64)
        s["ref"] = (sums + spread * noise).float()
        s.update(kind=case["kind"], average=case["average"], beta=0.1, smoothing=0.05, dscale=1.0 / P)
        if case["kind"] == "squared":
            s["smoothing"] = 0.0
        s["seq_logps"] = torch.empty(2 * P, device="cuda")
        s["losses"] = torch.empty(P, device="cuda")
    s["logits"] = z
    s["targets"] = torch.where(prompt, IGNORE, t).to(torch.int32)
    s["dlogits"] = torch.empty_like(z)
    s["logps"] = torch.empty(N, device="cuda")
    if "losses" not in s:
        s["losses"] = torch.empty(N, device="cuda")
    return s


# -- one pass ----------------------------------------------------------------------------------


def _softmax_rows(z, targets, V):
    """fp32 softmax over the real ids, kept rows, their targets, and log-probabilities (64 bits from fp32 sums)."""
    zf = z[:, :V].float()
    m = zf.max(1, keepdim=True).values
    e = torch.exp(zf - m)
    total = e.sum(1, keepdim=True)
    keep = targets != IGNORE
    t = torch.where(keep, targets, 0).long()
    zt = torch.gather(zf, 1, t[:, None])[:, 0].double()
    lp = torch.where(keep, zt - m[:, 0].double() - torch.log(total[:, 0].double()), 0.0)
    return e / total, keep, t, lp


def _logit_gradient(z, p, t, g):
    """dz_j = g ([j = t] - p_j) on the real ids, 0 on the padded ones, rounded once."""
    d = p * -g[:, None]
    d.scatter_add_(1, t[:, None], g[:, None])
    out = torch.zeros_like(z)
    out[:, :p.shape[1]] = d.to(z.dtype)
    return out


def _plain_policy(s):
    p, keep, t, lp = _softmax_rows(s["logits"], s["targets"], s["case"]["V"])
    adv = s["adv"].double()
    r = torch.exp(lp - s["old"].double())
    free, cut = r * adv, torch.clamp(r, 1 - s["clip_low"], 1 + s["clip_high"]) * adv
    loss = -torch.minimum(free, cut)
    g = torch.where(free <= cut, -free, 0.0)
    if s["ref"] is not None:
        d = s["ref"].double() - lp
        loss = loss + s["kl"] * (torch.exp(d) - d - 1)
        g = g + s["kl"] * (1 - torch.exp(d))
    w = keep.double() if s["weight"] is None else keep.double() * s["weight"].double()
    dz = _logit_gradient(s["logits"], p, t, (w * g * s["dscale"]).float())
    return dz, (w * loss).float(), lp.float()


def _plain_preference(s):
    p, keep, t, lp = _softmax_rows(s["logits"], s["targets"], s["case"]["V"])
    P = s["case"]["P"]
    at = torch.arange(lp.shape[0], device=lp.device)
    seq = torch.searchsorted(s["start"][1:].long(), at, right=True)
    score = torch.zeros(2 * P, dtype=torch.float64, device=lp.device).index_add_(0, seq, lp)
    share = torch.ones_like(score)
    if s["average"]:
        count = torch.zeros_like(score).index_add_(0, seq, keep.double())
        share = 1 / count.clamp(min=1)
        score = score * share
    gap = (score - s["ref"].double()).view(P, 2)
    delta = gap[:, 0] - gap[:, 1]
    b, eps = s["beta"], s["smoothing"]
    if s["kind"] == "sigmoid":
        up, down = torch.log1p(torch.exp(-b * delta)), torch.log1p(torch.exp(b * delta))
        loss = (1 - eps) * up + eps * down
        dd = -b * ((1 - eps) / (1 + torch.exp(b * delta)) - eps / (1 + torch.exp(-b * delta)))
    else:
        loss = (delta - 1 / (2 * b)) ** 2
        dd = 2 * (delta - 1 / (2 * b))
    g = (torch.stack([dd, -dd], 1).view(-1) * share)[seq] * keep.double() * s["dscale"]
    return _logit_gradient(s["logits"], p, t, g.float()), loss.float(), score.float(), lp.float()


def _newton_schulz_step(x):
    a, b, c = NS
    g = x @ x.transpose(1, 2)
    return a * x + (b * g + c * (g @ g)) @ x


def _plain_orthogonalize(s):
    x = s["x"].float()
    tall = x.shape[1] > x.shape[2]
    if tall:
        x = x.transpose(1, 2)
    x = x / (torch.sqrt((x * x).sum((1, 2), keepdim=True)) + 1e-7)
    step = _newton_schulz_step
    x = step(step(step(step(step(x)))))
    return (x.transpose(1, 2) if tall else x).to(torch.bfloat16).contiguous()


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"policy": _plain_policy, "preference": _plain_preference, "orthogonalize": _plain_orthogonalize}[op](s)
    import gpt_step_b200 as gs
    if op == "orthogonalize":
        if "ws" not in s:
            b, r, c = s["x"].shape
            s["ws"] = torch.empty(gs.orthogonalize_workspace(b, r, c), dtype=torch.uint8, device="cuda")
        gs.orthogonalize(s["x"], s["out"], s["ws"], s["err"])
        return s["out"]
    V = s["case"]["V"]
    if op == "policy":
        gs.policy_loss(s["logits"], s["targets"], s["old"], s["adv"], s["dlogits"], s["logps"], s["losses"], V,
                       s["err"], ref_logp=s["ref"], weight=s["weight"], ignore_index=IGNORE,
                       clip_low=s["clip_low"], clip_high=s["clip_high"], kl_coef=s["kl"], dscale=s["dscale"])
        return s["dlogits"], s["losses"], s["logps"]
    if "ws" not in s:
        s["ws"] = torch.empty(gs.preference_loss_workspace(s["logits"].shape[0], s["case"]["P"]),
                              dtype=torch.uint8, device="cuda")
    gs.preference_loss(s["logits"], s["targets"], s["start"], s["dlogits"], s["logps"], s["seq_logps"], s["losses"],
                       V, s["ws"], s["err"], ref_logp=s["ref"], ignore_index=IGNORE, kind=s["kind"],
                       average=s["average"], beta=s["beta"], smoothing=s["smoothing"], dscale=s["dscale"])
    return s["dlogits"], s["losses"], s["seq_logps"], s["logps"]


# -- the definition in 64 bits -----------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "orthogonalize":
        a, b, c = NS
        out = []
        for m in s["x"].double():
            y = m / (torch.linalg.norm(m) + 1e-7)
            # the step from the side of the smaller Gram matrix: y q(y'y) = q(yy') y
            for _ in range(5):
                if y.shape[0] >= y.shape[1]:
                    g = y.T @ y
                    y = y @ (a * torch.eye(len(g), device=y.device, dtype=y.dtype) + b * g + c * (g @ g))
                else:
                    g = y @ y.T
                    y = (a * torch.eye(len(g), device=y.device, dtype=y.dtype) + b * g + c * (g @ g)) @ y
            out.append(y)
        return torch.stack(out)
    V, t = case["V"], s["targets"].long()
    keep = t != IGNORE
    full = torch.zeros(s["logits"].shape, dtype=torch.float64, device="cuda")
    z = s["logits"][:, :V].double().requires_grad_(True)
    lp = torch.log_softmax(z, 1).gather(1, torch.where(keep, t, 0)[:, None])[:, 0]
    lp = torch.where(keep, lp, torch.zeros_like(lp))
    if case["op"] == "policy":
        adv = s["adv"].double()
        ratio = torch.exp(lp - s["old"].double())
        clipped = ratio.clamp(1 - s["clip_low"], 1 + s["clip_high"])
        loss = torch.where(ratio * adv <= clipped * adv, -ratio * adv, -clipped.detach() * adv)
        if s["ref"] is not None:
            away = s["ref"].double() - lp
            loss = loss + s["kl"] * (torch.expm1(away) - away)
        loss = torch.where(keep, loss, torch.zeros_like(loss))
        if s["weight"] is not None:
            loss = loss * s["weight"].double()
        full[:, :V] = torch.autograd.grad((loss * s["dscale"]).sum(), z)[0]
        return full, loss.detach(), lp.detach()
    start, scores = s["start"].tolist(), []
    for i in range(2 * case["P"]):
        total, n = lp[start[i]:start[i + 1]].sum(), int(keep[start[i]:start[i + 1]].sum())
        scores.append(total / max(n, 1) if s["average"] else total)
    score = torch.stack(scores)
    gap = score - s["ref"].double()
    delta = gap[0::2] - gap[1::2]
    if s["kind"] == "sigmoid":
        ls = torch.nn.functional.logsigmoid
        loss = -(1 - s["smoothing"]) * ls(s["beta"] * delta) - s["smoothing"] * ls(-s["beta"] * delta)
    else:
        loss = (delta - 1 / (2 * s["beta"])) ** 2
    full[:, :V] = torch.autograd.grad((loss * s["dscale"]).sum(), z)[0]
    return full, loss.detach(), score.detach(), lp.detach()


def work(case):
    """Every input read once and every output written once; of a masked row's logits nothing is needed."""
    if case["op"] == "orthogonalize":
        b, r, c = case["batch"], case["rows"], case["cols"]
        n, m = min(r, c), max(r, c)
        # per step: half of a symmetric product n n m, half of one n n n, and one full product n n m
        return {"bytes": b * r * c * ((4 if case["fp32"] else 2) + 2), "flops": 5 * b * n * n * (3 * m + n)}
    rows = case["N"] if case["op"] == "policy" else int(_lens(case).sum())
    kept = int(rows * (1 - case["masked"]))
    return {"bytes": 2 * kept * case["V"] + 2 * rows * case["Vp"] + 24 * rows, "flops": 8 * kept * case["V"]}
