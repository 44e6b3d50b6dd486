"""The post-training micro-steps where the head's GEMM leaves its rows' partial sums.

With a large vocabulary that GEMM runs on CTA pairs and the losses take each row's sum
from its partials; `token_logps` then has no logits at all. Those kernels are held to the
cross-entropy micro-step, which the model tests hold to the definition, on the same model
and tokens: where a loss has the cross-entropy's gradient (a policy loss on the sampling
policy itself, advantage 1; a preference loss as the sum of its two sequences'), the two
must agree to the roundings of the logit gradients.
"""
import math

import numpy as np
import pytest

import gpt_step_b200 as gs
from gpt_step_b200 import workloads

from gpu_util import f32, host, i32, rel_l2, require_gpu, torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


# 256 rows over 50,257 and 12,001 ids (partials), 256 rows over 1,000 (128-wide tiles: stored rows), 128 rows (the same)
SIZES = [(4, 50257), (4, 12001), (4, 1000), (2, 20001)]


def model(B, V, **over):
    return gs.GPT2(gs.Config.make(**workloads.model_args("tiny", micro_batch=B, vocab_real=V, **over)), 1337)


def batch(m, V, seed):
    rng = np.random.default_rng(seed)
    return rng, rng.integers(0, V, (m.B, m.T)), rng.integers(0, V, (m.B, m.T))


def spread(m):
    """Weights of a trained model's size: logits a few units apart instead of near 0."""
    for i, t in enumerate(m.tensors()):
        if t.name == "wte.weight":
            m.write(gs.GPT2_PARAMS, i, m.read(gs.GPT2_PARAMS, i) * 8)


def grads_of(m, run):
    m.state_tensor(gs.GPT2_GRADS).zero_()
    run()
    return {n: g.copy() for n, g in m.read_all(gs.GPT2_GRADS).items()}


# Between two gradients whose logit gradients differ by roundings to bf16 only: half a step (2^-9 of the
# value's binade) each way is 2^-8 of an element at most, uncorrelated over the 256 rows and the ids a sum
# runs over, and the backward rounds its own bf16 activations again some ten times the same way; in
# quadrature sqrt(11) 2^-9 / sqrt(3) = 3.7e-3 of a tensor's norm where every one of them fell differently.
SAME = 4e-3


def check_same(a, b, tol=SAME):
    assert a.keys() == b.keys()
    whole = math.sqrt(sum(float(np.sum(v.astype(np.float64) ** 2)) for v in b.values()))
    for n in a:
        # (a key bias's gradient is exactly 0, what is there is rounding: against the whole gradient)
        d = float(np.linalg.norm(a[n].astype(np.float64) - b[n]))
        assert d <= tol * float(np.linalg.norm(b[n])) + 1e-6 * whole, (n, rel_l2(a[n], b[n]))


@pytest.mark.parametrize("B,V", SIZES)
def test_log_probabilities_are_the_cross_entropys(B, V):
    m = model(B, V)
    spread(m)
    _, x, y = batch(m, V, 1)
    m.fwd_bwd(i32(x), i32(y))
    loss = m.token_losses().astype(np.float64)
    assert loss.std() > 0.5                                  # (not the flat start)
    lp = torch.empty(B, m.T, device="cuda")
    m.token_logps(i32(x), i32(y), lp)
    # the same bf16 logits; each side sums their exponentials in fp32: 2^-19, and roundings of 2^-22 of the values
    tol = 2 * (2.0 ** -19 + 2.0 ** -22 * (loss + 16))
    assert np.all(np.abs(host(lp) + loss) <= tol)
    cut = y.copy()
    cut[:, ::3] = -1
    out = torch.full((B, m.T), 5.0, device="cuda")
    m.token_logps(i32(x), i32(cut), out)                     # rows left out change no other
    assert torch.equal(out, torch.where(i32(cut) >= 0, lp, torch.zeros_like(lp)))
    whole = m.eval_loss(i32(x), i32(y))
    assert abs(whole + float(lp.double().mean())) <= 1e-5


@pytest.mark.parametrize("B,V", SIZES)
def test_policy_gradient_on_the_sampling_policy_is_the_cross_entropys(B, V):
    m = model(B, V)
    spread(m)
    rng, x, y = batch(m, V, 2)
    xt, yt, n = i32(x), i32(y), B * m.T
    ce = grads_of(m, lambda: m.fwd_bwd(xt, yt))
    old = torch.empty(B, m.T, device="cuda")
    m.token_logps(xt, yt, old)
    one, now = torch.ones(B, m.T, device="cuda"), torch.empty(B, m.T, device="cuda")
    pol = grads_of(m, lambda: m.fwd_bwd_policy(xt, yt, old, one, scale=1.0 / n, logps=now))
    assert torch.allclose(now, old, atol=2.0 ** -18, rtol=2.0 ** -21)
    check_same(pol, ce)
    # the KL term alone (advantages 0): its slope at ref = lp + log 2 is -kl, as an advantage of kl
    zero, ref = torch.zeros_like(one), old + math.log(2.0)
    kl = grads_of(m, lambda: m.fwd_bwd_policy(xt, yt, old, zero, ref_logp=ref, kl_coef=1.0, scale=1.0 / n))
    check_same(kl, ce)
    # weights and advantages that differ by row are linear: two halves make the whole
    part = torch.tensor(rng.random((B, m.T)) < 0.5, device="cuda")
    halves = [grads_of(m, lambda w=w: m.fwd_bwd_policy(xt, yt, old, one, weight=w.float(), scale=1.0 / n))
              for w in (part, ~part)]
    # (each half's norm is that of the whole or less; two sums of roundings, and the sum's own)
    check_same({k: halves[0][k].astype(np.float64) + halves[1][k] for k in ce}, ce, tol=2 * SAME)


@pytest.mark.parametrize("B,V", SIZES)
@pytest.mark.parametrize("average", [False, True])
def test_preference_gradient_is_that_of_its_rows(B, V, average):
    """dL/dlp is one number a sequence: the policy loss with those as advantages has the same gradient."""
    m = model(B, V)
    spread(m)
    rng, x, y = batch(m, V, 3)
    y[:, : m.T // 4] = -1
    y[1, m.T // 2:] = -1
    xt, yt = i32(x), i32(y)
    lp = torch.empty(B, m.T, device="cuda")
    m.token_logps(xt, yt, lp)
    count = torch.tensor((y >= 0).sum(1), device="cuda", dtype=torch.float64)
    score = lp.double().sum(1) / (count if average else 1)
    ref = score + torch.tensor(rng.standard_normal(B), device="cuda")
    seq = torch.empty(B, device="cuda")
    beta, losses = 0.3, []
    pref = grads_of(m, lambda: losses.append(m.fwd_bwd_preference(
        xt, yt, ref_logp=ref.float(), beta=beta, smoothing=0.1, average=average, seq_logps=seq, want_loss=True)))
    gap = score - ref.float().double()
    delta = gap[0::2] - gap[1::2]
    want = (-0.9 * torch.nn.functional.logsigmoid(beta * delta)
            - 0.1 * torch.nn.functional.logsigmoid(-beta * delta)).mean()
    # a sequence's sum: 64 log-probabilities, each within 2^-18 and 2^-21 of its size
    off = m.T * (2.0 ** -18 + 2.0 ** -21 * float(lp.abs().max())) + 2.0 ** -23 * float(score.abs().max())
    assert torch.allclose(seq.double(), score, atol=off, rtol=0)
    assert abs(losses[0] - float(want)) <= 2 * beta * off + 1e-6
    slope = -beta * (0.9 * torch.sigmoid(-beta * delta) - 0.1 * torch.sigmoid(beta * delta)) * 2 / B
    per = torch.stack([slope, -slope], 1).flatten() / (count if average else 1)
    adv = (-per)[:, None].expand(B, m.T).float().contiguous()
    pol = grads_of(m, lambda: m.fwd_bwd_policy(xt, yt, lp, adv))
    check_same(pref, pol)


@pytest.mark.parametrize("B,V", SIZES)
def test_log_probabilities_leave_the_micro_steps_results(B, V):
    m = model(B, V)
    _, x, y = batch(m, V, 5)
    xt, yt = i32(x), i32(y)
    m.fwd_bwd(xt, yt)
    losses, grads = m.token_losses(), m.state_tensor(gs.GPT2_GRADS).clone()
    m.token_logps(i32(x[:, ::-1].copy()), yt, torch.empty(B, m.T, device="cuda"))
    assert np.array_equal(m.token_losses(), losses)
    assert torch.equal(m.state_tensor(gs.GPT2_GRADS), grads)
    m.clip_adamw(0)
    assert abs(m.last_step_stats()[0] - losses.mean()) <= 1e-5


@pytest.mark.parametrize("B,V", SIZES)
def test_policy_micro_step_with_log_probabilities_over_the_old_ones(B, V):
    m = model(B, V)
    spread(m)
    rng, x, y = batch(m, V, 6)
    xt, yt = i32(x), i32(y)
    old = torch.empty(B, m.T, device="cuda")
    m.token_logps(xt, yt, old)
    old -= f32(0.1 * rng.standard_normal((B, m.T)))
    adv, lp = f32(rng.standard_normal((B, m.T))), torch.empty_like(old)
    want = grads_of(m, lambda: m.fwd_bwd_policy(xt, yt, old, adv, logps=lp))
    losses = m.token_losses()
    for _ in range(3):
        over = old.clone()
        got = grads_of(m, lambda: m.fwd_bwd_policy(xt, yt, over, adv, logps=over))
        assert torch.equal(over, lp) and np.array_equal(m.token_losses(), losses)
        # (the gradients' atomics add in any order)
        check_same(got, want, tol=1e-5)


def launches_of(m, run):
    before = m.kernel_launches()
    run()
    return m.kernel_launches() - before


def device_launches(run):
    with torch.profiler.profile(activities=[torch.profiler.ProfilerActivity.CUDA]) as prof:
        run()
        torch.cuda.synchronize()
    return sum(1 for e in prof.events() if e.device_type == torch.autograd.DeviceType.CUDA
               and not e.name.lower().startswith("mem"))


# B, T, V and the launches behind the rows' log-probabilities: the pairs in the gradient's launch, or a launch before it
@pytest.mark.parametrize("B,T,V,pair_launches", [(4, 64, 1000, 1), (2, 64, 20001, 2), (4, 64, 50257, 2), (10, 1024, 300, 2)])
def test_launch_count_of_the_preference_micro_step(B, T, V, pair_launches):
    m = model(B, V, seq_len=T, n_layer=1)
    _, x, y = batch(m, V, 4)
    xt, yt = i32(x), i32(y)
    one = torch.ones(B, T, device="cuda")
    # the policy micro-step differs by one launch for the rows in place of two or three
    policy = launches_of(m, lambda: m.fwd_bwd_policy(xt, yt, one, one))
    pref = launches_of(m, lambda: m.fwd_bwd_preference(xt, yt))
    assert pref - policy == pair_launches
    made = [device_launches(lambda: m.fwd_bwd_policy(xt, yt, one, one)),
            device_launches(lambda: m.fwd_bwd_preference(xt, yt))]
    if made[0]:                                             # (0 where the profiler has no access to the device)
        assert made[1] - made[0] == pair_launches
