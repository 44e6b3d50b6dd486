"""The post-training losses where numbers end: NaN and infinities in logits and inputs.

What has a finite value is held to the bounds of test_gpu_posttrain.py (`lp_tol`,
`grad_tol`); what has none must not look as if it had.
"""
import math

import numpy as np
import pytest

import gpt_step_b200 as gs
from oracle import posttrain as PT

from gpu_util import bf16, err_word, f32, host, i32, require_gpu, torch
from test_gpu_posttrain import grad_tol, lp_tol, rows_case

pytestmark = pytest.mark.gpu

# a row by one warp, by sixteen, and from global memory
WIDTHS = [(40, 48), (1000, 1024), (5000, 5008), (50257, 50304), (120001, 120008)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def policy(z, t, V, old, adv, grad=True, **kw):
    N, Vp = z.shape
    dz = torch.full((N, Vp), 7.0, dtype=torch.bfloat16, device="cuda") if grad else None
    logps, losses, err = torch.full((N,), 7.0, device="cuda"), torch.full((N,), 7.0, device="cuda"), err_word()
    gs.policy_loss(bf16(z), i32(t), f32(old), f32(adv), dz, logps, losses, V, err,
                   **{k: f32(v) if isinstance(v, np.ndarray) else v for k, v in kw.items()})
    assert int(err.sum()) == 0
    return host(logps), host(losses), host(dz) if grad else None


@pytest.mark.parametrize("V,Vp", WIDTHS)
def test_policy_loss_of_numbers_that_are_none(V, Vp):
    """A NaN anywhere in a kept row's formula is a NaN in its loss and its gradient."""
    rng, z, t = rows_case(9, V, Vp, V, masked=0.0)
    lp, _, _ = PT.token_logps(z, t, V)
    adv = np.array([1.0, -1.0, 1.0, 1.0, 0.0, 0.0, 1.0, -2.0, 1.0])
    old = lp.astype(np.float32).astype(np.float64)
    ref, w = old.copy(), np.ones(9)
    z[0, (t[0] + 1) % V] = np.nan              # the row's logits
    z[1, t[1]] = np.nan
    old[2] = np.nan                            # the sampling policy's log-probability
    adv[3] = np.nan
    z[4, (t[4] + 1) % V] = np.nan              # an advantage of 0 does not hide the row's own logits
    old[5] = np.nan                            # but it gives 0 for any ratio
    w[6] = np.nan
    bad = [0, 1, 2, 3, 4, 6]
    got_lp, loss, dz = policy(z, t, V, old, adv, weight=w)
    assert np.isnan(loss[bad]).all() and np.isnan(dz[bad][:, :V]).all() and np.all(dz[:, V:] == 0)
    assert np.isnan(got_lp[[0, 1, 4]]).all()
    fine = [2, 3, 5, 6, 7, 8]
    assert np.all(np.abs(got_lp - lp)[fine] <= lp_tol(lp)[fine])
    assert loss[5] == 0 and np.all(dz[5] == 0)
    rl, _, rdz = PT.policy_loss(z[7:], t[7:], V, old[7:], adv[7:])
    # the ratio is 1 within the log-probability's bound
    assert np.all(np.abs(loss[7:] - rl) <= 2 * np.abs(adv[7:]) * (lp_tol(lp[7:]) + 2.0 ** -23))
    assert np.all(np.abs(dz[7:] - rdz) <= grad_tol(rdz, np.abs(adv[7:])))
    # the losses alone, and with a KL term whose reference is a NaN too
    assert np.isnan(policy(z, t, V, old, adv, grad=False, weight=w)[1][bad]).all()
    ref[8] = np.nan
    _, loss, dz = policy(z, t, V, old, adv, weight=w, ref_logp=ref, kl_coef=0.1)
    bad.append(8)
    assert np.isnan(loss[bad]).all() and np.isnan(dz[bad][:, :V]).all() and np.isfinite(loss[[5, 7]]).all()


@pytest.mark.parametrize("V,Vp", WIDTHS)
def test_oracle_and_kernel_agree_on_infinite_ratios(V, Vp):
    """old_logp of -inf and +inf, an advantage of 0 among them: losses as defined, none a NaN."""
    _, z, t = rows_case(6, V, Vp, V + 1, masked=0.0)
    old = np.array([-np.inf, -np.inf, np.inf, np.inf, -np.inf, np.inf])
    adv = np.array([1.0, -1.0, 1.0, -1.0, 0.0, 0.0])
    with np.errstate(invalid="ignore"):
        rl, _, rdz = PT.policy_loss(z, t, V, old, adv)
    _, loss, dz = policy(z, t, V, old, adv)
    rest = np.isfinite(rl)
    assert np.all(loss[~rest] == rl[~rest]) and np.all(np.abs(loss - rl)[rest] <= 2.0 ** -23 * np.abs(rl)[rest])
    assert np.all(dz[rest] == rdz[rest]) and loss[1] == np.inf


@pytest.mark.parametrize("V,Vp", [(40, 48), (100, 104), (1000, 1024), (9001, 9008), (50257, 50304), (120001, 120008)])
def test_no_nan_is_lost_from_a_row(V, Vp):
    """Whole 16-byte pieces of NaN, at all places of two lanes whose sums are joined first."""
    rng = np.random.default_rng(V)
    z = rng.standard_normal((4, Vp))
    lanes = (np.arange(Vp) // 8) % 32
    t = np.full(4, 3)                                   # a piece of its own
    z[0, 8:16] = np.nan
    z[1, (lanes == 5) | (lanes == 21)] = np.nan
    z[2, (lanes == 5) | (lanes == 21)] = -np.inf
    z[2, 5 * 8] = np.nan
    z[:, V:] = 1.0
    if V < 45:
        z[2, 8] = np.nan
    zd, err = bf16(z), err_word()
    lp = torch.zeros(4, device="cuda")
    gs.token_logps(zd, i32(t), lp, V, err)
    want = [True, bool(V > 40) or bool(np.isnan(z[1, :V]).any()), True, False]
    assert [bool(v) for v in np.isnan(host(lp))] == want
    for inplace in (False, True):
        seq, losses = torch.zeros(2, device="cuda"), torch.zeros(1, device="cuda")
        ws = torch.empty(gs.preference_loss_workspace(4, 1), dtype=torch.uint8, device="cuda")
        src = zd.clone()
        dz = src if inplace else torch.zeros_like(zd)
        gs.preference_loss(src, i32(t), i32([0, 3, 4]), dz, lp, seq, losses, V, ws, err)
        assert np.isnan(host(seq)[0]) and np.isfinite(host(seq)[1]) and np.isnan(host(losses)[0])
        assert [bool(v) for v in np.isnan(host(lp))] == want


@pytest.mark.parametrize("rows", [1, 5000])             # the coefficient inside the gradient's launch, and in its own
@pytest.mark.parametrize("V,Vp", [(40, 48), (50257, 50304)])
def test_preference_loss_of_tokens_that_are_ruled_out(rows, V, Vp):
    """A token of logit -inf: its sequence's log-probability is -inf, and the losses are their limits."""
    if rows > 1 and V > 40:
        rows = 40
    rng = np.random.default_rng(V + rows)
    N = 4 * rows
    z = np.round(rng.standard_normal((N, Vp)) * 4) / 4
    t = rng.integers(0, V, N)
    z[rows, t[rows]] = -np.inf                          # pair 0: the rejected sequence; pair 1: the chosen one
    z[2 * rows, t[2 * rows]] = -np.inf
    start = np.arange(5) * rows
    for kind, smoothing, want in (("sigmoid", 0.0, (0.0, np.inf)), ("sigmoid", 0.1, (np.inf, np.inf)),
                                  ("squared", 0.0, (np.inf, np.inf))):
        lp, seq = torch.empty(N, device="cuda"), torch.empty(4, device="cuda")
        losses, err = torch.empty(2, device="cuda"), err_word()
        dz = torch.full((N, Vp), 7.0, dtype=torch.bfloat16, device="cuda")
        ws = torch.empty(gs.preference_loss_workspace(N, 2), dtype=torch.uint8, device="cuda")
        gs.preference_loss(bf16(z), i32(t), i32(start), dz, lp, seq, losses, V, ws, err, kind=kind, beta=0.3,
                           smoothing=smoothing)
        assert tuple(host(losses)) == want and int(err.sum()) == 0
        rl, rs, rlp, rdz = PT.preference_loss(z, t, V, start, kind=kind, beta=0.3, smoothing=smoothing)
        assert tuple(rl) == want
        assert host(seq)[1] == -np.inf and host(seq)[2] == -np.inf and np.isfinite(host(seq)[[0, 3]]).all()
        if kind == "sigmoid":                           # slopes -beta (0, or -smoothing's part) and -beta (1 - smoothing)
            g = np.repeat([0.3 * smoothing, 0.3 * (1 - smoothing)], 2 * rows)
            assert np.all(np.abs(host(dz) - rdz) <= grad_tol(rdz, g))


@pytest.mark.parametrize("V,Vp", WIDTHS)
def test_policy_loss_of_a_token_that_only_the_reference_allows(V, Vp):
    """The policy rules the token out, the reference does not: the KL term is +inf, not a NaN."""
    _, z, t = rows_case(3, V, Vp, V + 2, masked=0.0)
    z[1, t[1]] = -np.inf
    old, adv = np.zeros(3), np.ones(3)
    ref = np.array([-1.0, -1.0, -np.inf])               # row 2 the other way round: infinite too
    _, loss, _ = policy(z, t, V, old, adv, ref_logp=ref, kl_coef=0.1)
    rl = PT.policy_loss(z, t, V, old, adv, ref=ref, kl=0.1)[0]
    assert loss[1] == np.inf and loss[2] == np.inf and rl[1] == np.inf and rl[2] == np.inf
    assert math.isfinite(loss[0]) and abs(loss[0] - rl[0]) <= 1e-5 * (1 + abs(rl[0]))


BAD_BOUNDS = [
    # bounds, pairs that have theirs
    ([2000000000, 5, 10, 15, 20], [False, True]),
    ([-3, 5, 10, 15, 20], [False, True]),
    ([0, 5, 10, 15, 21], [True, False]),
    ([0, 5, 9, 4, 20], [True, False]),
    ([0, 15, 20, 20, 12], [False, False]),      # the first pair ends behind the last bound
    ([4, 6, 9, 9, 2], [True, False]),          # the last bound before the first: every row may be in a pair
    ([0, 5, 10, 19, 12, 14, 16], [True, False, True]),
    ([6, 2, 7, 9, 12, 14, 16], [False, True, True]),
    ([0, 3, 5, 1000000, -5, 8, 13], [True, False, False]),
    ([9, 3, 1], [False]),
]


@pytest.mark.parametrize("start,good", BAD_BOUNDS)
@pytest.mark.parametrize("V,Vp,rows", [(30, 32, 20), (5001, 5008, 20), (20001, 20008, 20), (30, 32, 9000)])
def test_pairs_beside_bounds_that_are_not_bounds(start, good, V, Vp, rows):
    """Pairs of sound bounds get their loss, and their rows their gradient or none; the others 0 and none; flag 1."""
    _, z, t = rows_case(rows, V, Vp, 8, masked=0.2)
    start, P = np.array(start), len(good)
    err, losses = err_word(), torch.full((P,), 9.0, device="cuda")
    dz = torch.full((rows, Vp), 5.0, dtype=torch.bfloat16, device="cuda")
    logps = torch.full((rows,), float("nan"), device="cuda")
    ws = torch.full((gs.preference_loss_workspace(rows, P),), 0xFF, dtype=torch.uint8, device="cuda")
    if rows > 20:
        start = np.where(start == 20, rows, np.where(start == 21, rows + 1, start))
    gs.preference_loss(bf16(z), i32(t), i32(start), dz, logps, None, losses, V, ws, err, beta=0.5, dscale=1.0)
    assert int(err[0]) == 1
    got, covered = host(dz), np.zeros(rows, bool)
    for p in range(P):
        if not good[p]:
            assert float(losses[p]) == 0.0
            continue
        b = start[2 * p:2 * p + 3]
        rl, _, rlp, rdz = PT.preference_loss(z, t, V, b, beta=0.5)
        tol = (b[2] - b[0]) * lp_tol(np.abs(rlp).max())
        assert abs(float(losses[p]) - rl[0]) <= 0.5 * tol + 2.0 ** -22 * abs(rl[0])
        in_pair = slice(b[0], b[2])
        g = np.full(rows, 0.5)
        # (the slope's change over the margin's error: beta^2 / 4 of it); the search may miss a row's sequence
        right = np.all(np.abs(got - rdz) <= grad_tol(rdz, g) + 0.07 * tol, axis=1)
        none = np.all(got == 0, axis=1)
        assert np.all((right | none)[in_pair])
        if len(good) < 3:
            assert np.all(right[in_pair])
        covered[in_pair] = True
    rest = got[~covered]
    assert np.all((rest == 0) | (rest == 5.0)) and np.all(rest.min(1) == rest.max(1))


@pytest.mark.parametrize("V,Vp", WIDTHS)
def test_policy_loss_with_outputs_in_the_inputs_place(V, Vp):
    """logps over old_logp (or the reference), losses over the advantages (or weights)."""
    rng, z, t = rows_case(400, V, Vp, V + 3)
    zd, td, err = bf16(z), i32(t), err_word()
    ins = [f32(-1 - 3 * rng.random(400)), f32(rng.standard_normal(400)), f32(-1 - 3 * rng.random(400)),
           f32(rng.uniform(0.5, 2, 400))]

    def call(old, adv, ref, w, logps, losses, dz):
        gs.policy_loss(zd, td, old, adv, dz, logps, losses, V, err, ref_logp=ref, weight=w, kl_coef=0.2)
        return [v.clone() for v in (logps, losses, dz)]

    want = call(*ins, torch.empty(400, device="cuda"), torch.empty(400, device="cuda"), torch.empty_like(zd))
    for lp_at, loss_at in ((0, 1), (2, 3), (1, 0), (3, 2)):
        for _ in range(3):
            c = [v.clone() for v in ins]
            got = call(*c, c[lp_at], c[loss_at], torch.empty_like(zd))
            assert all(torch.equal(a, b) for a, b in zip(got, want)), (lp_at, loss_at)


def test_preference_loss_beside_its_reference():
    """One buffer may hold the reference and the outputs side by side, but not over it."""
    rng, z, t = rows_case(40, 100, 104, 9)
    start = i32([0, 10, 20, 30, 40])
    one = torch.zeros(4 + 4 + 2 + 40, device="cuda")
    ref, seq, losses, logps = one[:4], one[4:8], one[8:10], one[10:]
    ws, err = torch.empty(gs.preference_loss_workspace(40, 2), dtype=torch.uint8, device="cuda"), err_word()
    gs.preference_loss(bf16(z), i32(t), start, None, logps, seq, losses, 100, ws, err, ref_logp=ref)
    rl, rs, rlp, _ = PT.preference_loss(z, t, 100, host(start).astype(int), ref=np.zeros(4))
    assert np.all(np.abs(host(logps) - rlp) <= lp_tol(rlp)) and np.allclose(host(losses), rl, atol=1e-4)
    for over in (dict(seq=ref), dict(losses=ref[1:3]), dict(seq=one[3:7]), dict(seq=None, logps=one[3:43])):
        a = dict(seq=seq, losses=losses, logps=logps)
        a.update(over)
        with pytest.raises(gs.GPT2Error):
            gs.preference_loss(bf16(z), i32(t), start, None, a["logps"], a["seq"], a["losses"], 100, ws, err, ref_logp=ref)
    assert np.all(host(ref) == 0)
