"""The post-training losses, the orthogonalisation and the model calls on them, against
their fp64 definitions.

Bounds. A row's (c, S) holds sums of non-negative fp32 terms, each from an FFMA (half
a step, 2^-24 of an exponent below 2^6) and an ex2 (2^-22): relative error of S below
2^-19 in the worst case, so |lp error| <= 2^-19 + 2^-22 (|lp| + 1): `lp_tol`. A
gradient element is one bf16 rounding (half a step, 2^-8 of its value) of g ([j=t] - p)
with relative errors of p and g of that size: `grad_tol`.
"""
import math

import numpy as np
import pytest

import gpt_step_b200 as gs
from gpt_step_b200 import workloads
from oracle import gpt2 as G
from oracle import posttrain as PT

from gpu_util import bf16, err_word, f32, host, i32, rel_l2, require_gpu, rounded, torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def lp_tol(lp):
    return 2.0 ** -19 + 2.0 ** -22 * (np.abs(lp) + 1)


def grad_tol(ref, g):
    """ref: the gradient, g: each row's largest possible coefficient."""
    return 2.0 ** -8 * np.abs(ref) * (1 + 2.0 ** -6) + 2.0 ** -17 * np.abs(g)[:, None] + 1e-38


def rows_case(N, V, Vp, seed, masked=0.3, spread=2.0):
    rng = np.random.default_rng(seed)
    z = rounded(rng.standard_normal((N, Vp)) * spread)
    t = rng.integers(0, V, N)
    z[np.arange(N), t] = rounded(z[np.arange(N), t] + math.log(V))
    t[rng.random(N) < masked] = -1
    return rng, z, t


def policy_inputs(rng, z, t, V):
    N = len(t)
    lp, _, keep = PT.token_logps(z, t, V)
    d = 0.3 * rng.standard_normal(N)
    for edge in (math.log(0.8), math.log(1.28)):      # off the clip borders, where one rounding decides
        d[np.abs(d - edge) < 1e-3] += 4e-3
    f = lambda a: np.asarray(a, np.float32).astype(np.float64)  # noqa: E731
    old, ref = f(lp - d), f(lp + 0.4 * rng.standard_normal(N))
    adv, w = f(rng.standard_normal(N)), f(rng.uniform(0.25, 2, N))
    adv[::5] = 0.0
    return lp, keep, old, ref, adv, w


SIZES = [(1, 1, 8), (3, 2, 8), (5, 9, 16), (64, 1000, 1024), (37, 1000, 1000), (33, 4353, 4480), (7, 8449, 8576),
         (130, 2040, 2048), (9, 50257, 50304), (5, 30011, 30016), (700, 33001, 33008), (4, 90003, 90008),
         (4, 120001, 120008)]


def scale_of(lp, old, ref, adv, w, kl, ds):
    g = np.abs(np.exp(lp - old) * adv)
    if kl:
        g = g + kl * (1 + np.exp(ref - lp))
    return g * w * ds


@pytest.mark.parametrize("N,V,Vp", SIZES)
@pytest.mark.parametrize("kl,weighted,inplace", [(0.0, False, False), (0.1, True, True)])
def test_policy_loss(N, V, Vp, kl, weighted, inplace):
    rng, z, t = rows_case(N, V, Vp, N + V)
    lp, keep, old, ref, adv, w = policy_inputs(rng, z, t, V)
    ds = 1.0 / N
    rl, rlp, rdz = PT.policy_loss(z, t, V, old, adv, ref=ref if kl else None, weight=w if weighted else None,
                                  clip_high=0.28, kl=kl, dscale=ds)
    # nothing of a row left out, and no padded column, may be read into a result
    z = z.copy()
    z[~keep] = np.nan
    z[:, V:] = np.inf
    for a in (old, ref, adv, w):
        a[~keep] = np.nan
    zd = bf16(z)
    dz = zd if inplace else torch.full_like(zd, 7.0)
    logps, losses, err = torch.full((N,), 9.0, device="cuda"), torch.full((N,), 9.0, device="cuda"), err_word()
    gs.policy_loss(zd, i32(t), f32(old), f32(adv), dz, logps, losses, V, err, ref_logp=f32(ref) if kl else None,
                   weight=f32(w) if weighted else None, clip_high=0.28, kl_coef=kl, dscale=ds)
    old, ref, adv, w = (np.where(keep, a, 0.0) for a in (old, ref, adv, w))
    got = host(dz)
    wk = w if weighted else np.ones(N)
    g = scale_of(rlp, old, ref, adv, wk, kl, ds)
    assert np.all(np.abs(host(logps) - rlp) <= lp_tol(rlp))
    assert np.all(np.abs(host(losses) - rl) <= 2 * g / ds * lp_tol(rlp) + 2.0 ** -21 * (np.abs(rl) + g / ds))
    assert np.all(np.abs(got - rdz) <= grad_tol(rdz, g))
    assert np.all(got[~keep] == 0) and np.all(got[:, V:] == 0)
    assert np.all(host(losses)[~keep] == 0) and np.all(host(logps)[~keep] == 0)
    assert int(err.sum()) == 0


def test_policy_loss_alone_and_bad_targets():
    rng, z, t = rows_case(12, 100, 104, 5, masked=0.0)
    lp, keep, old, ref, adv, w = policy_inputs(rng, z, t, 100)
    rl, rlp, rdz = PT.policy_loss(z, t, 100, old, adv)
    losses, err = torch.empty(12, device="cuda"), err_word()
    gs.policy_loss(bf16(z), i32(t), f32(old), f32(adv), None, None, losses, 100, err)
    assert np.all(np.abs(host(losses) - rl) <= 1e-5 * (1 + np.abs(rl)))
    assert int(err.sum()) == 0
    t[3], t[7] = 100, -7                                   # not ids, not the ignore index
    dz = torch.empty(12, 104, dtype=torch.bfloat16, device="cuda")
    gs.policy_loss(bf16(z), i32(t), f32(old), f32(adv), dz, None, losses, 100, err)
    assert int(err[0]) == 1
    assert np.all(host(dz)[[3, 7]] == 0) and np.all(host(losses)[[3, 7]] == 0)
    rest = np.setdiff1d(np.arange(12), [3, 7])
    tol = grad_tol(rdz, scale_of(rlp, old, ref, adv, 1.0, 0.0, 1.0))
    assert np.all((np.abs(host(dz) - rdz) <= tol)[rest])


@pytest.mark.parametrize("V,Vp", [(40, 48), (5000, 5008), (40001, 40008)])
def test_rows_without_a_finite_log_probability_stay_in_their_rows(V, Vp):
    z = np.zeros((5, Vp))
    z[0, 3] = np.nan
    z[1, :V] = -np.inf
    z[2, 7] = -np.inf                                      # one id ruled out
    z[3, 7] = -np.inf                                      # the target ruled out: ratio 0
    t = np.array([1, 1, 5, 7, 2])
    losses, logps, err = torch.empty(5, device="cuda"), torch.empty(5, device="cuda"), err_word()
    zd = bf16(z)
    dz = torch.empty_like(zd)
    zero, one = torch.zeros(5, device="cuda"), torch.ones(5, device="cuda")
    gs.policy_loss(zd, i32(t), zero, one, dz, logps, losses, V, err)
    lp, d, ls = host(logps), host(dz), host(losses)
    assert np.isnan(lp[0]) and np.isnan(lp[1]) and lp[3] == -np.inf
    assert abs(lp[2] + math.log(V - 1)) < 1e-6 and abs(lp[4] + math.log(V)) < 1e-6
    assert ls[3] == 0 and np.all(d[3] == 0) and d[2, 7] == 0
    assert np.all(np.isfinite(d[[2, 4]])) and np.all(d[:, V:] == 0)


@pytest.mark.parametrize("V,Vp", [(1000, 1024), (9000, 9000), (40001, 40008), (120001, 120008)])
def test_targets_far_below_the_largest_logit(V, Vp):
    """Differences past the exponents of fp32, both ways: log-probabilities and gradients stay finite."""
    rng = np.random.default_rng(V)
    z = rounded(rng.standard_normal((12, Vp)))
    t = np.array([3, 5, 7, V - 1, 11, 13, 15, 17, 19, 21, 23, 25])
    z[0, 4] = z[1, 6] = 400.0                              # the target 400 below another id
    z[2, 7] = 400.0                                        # and above all
    z[3, :V] -= 30000.0
    z[4, :V] += 30000.0
    for row, up in zip(range(6, 12), (20.0, 40.0, 60.0, 80.0, 86.0, 90.0)):
        z[row, 4] = up                                      # around the exponents' end, and well before it
    z = rounded(z)
    lp, p, keep = PT.token_logps(z, t, V)
    old = np.where(lp < -15, lp, 0.0)
    ds = 1e-7
    rl, rlp, rdz = PT.policy_loss(z, t, V, old.astype(np.float32), np.ones(12), clip_high=0.5, dscale=ds)
    losses, logps, err = torch.empty(12, device="cuda"), torch.empty(12, device="cuda"), err_word()
    dz = torch.empty(12, Vp, dtype=torch.bfloat16, device="cuda")
    gs.policy_loss(bf16(z), i32(t), f32(old), f32(np.ones(12)), dz, logps, losses, V, err, clip_high=0.5, dscale=ds)
    # the logits themselves are large here: y - c is one rounding of a difference, its factor log2(e) 2^-25
    tol = 2.0 ** -19 + 2.0 ** -22 * np.abs(rlp)
    assert np.all(np.abs(host(logps) - rlp) <= tol)
    g = np.abs(np.exp(np.minimum(rlp - old, 1.0))) * ds
    # the ratio's error: lp's, and old's rounding to fp32 (2^-24 of it)
    rough = tol + 2.0 ** -24 * np.abs(old)
    assert np.all(np.abs(host(dz) - rdz) <= grad_tol(rdz, g) + rough[:, None] * np.abs(rdz) + (rough * g)[:, None])
    # elements far from the target's are exact to their rounding: p must not fall to 0
    assert np.all((host(dz)[:, 4] != 0) == (np.abs(rdz[:, 4]) > 1e-37))
    assert int(err.sum()) == 0


def test_policy_loss_of_enormous_advantages():
    """Gradients up to the end of bf16's range are finite values."""
    rng, z, t = rows_case(6, 300, 304, 4, masked=0.0)
    lp, _, _ = PT.token_logps(z, t, 300)
    adv = np.array([1e30, 1e33, -1e36, 1e38, 3.0, -1e31])
    rl, rlp, rdz = PT.policy_loss(z, t, 300, lp.astype(np.float32), adv)
    losses, dz, err = torch.empty(6, device="cuda"), torch.empty(6, 304, dtype=torch.bfloat16, device="cuda"), err_word()
    gs.policy_loss(bf16(z), i32(t), f32(lp), f32(adv), dz, None, losses, 300, err)
    got = host(dz)
    assert np.all(np.isfinite(got))
    assert np.all(np.abs(got - rdz) <= grad_tol(rdz, np.abs(adv) * 1.1))


def ragged(rng, S, most, gap=True):
    lens = rng.integers(0, most + 1, S)
    lens[rng.integers(0, S)] = 0
    first = 3 if gap else 0
    return np.concatenate([[0], np.cumsum(lens)]) + first


@pytest.mark.parametrize("P,most,V,Vp", [(1, 1, 2, 8), (1, 5, 9, 16), (3, 40, 1000, 1024), (5, 300, 333, 336),
                                         (2, 700, 1001, 1008), (40, 3, 50, 56), (2, 6, 50257, 50304), (2, 5, 120001, 120008)])
@pytest.mark.parametrize("kind,average,smoothing,inplace", [("sigmoid", False, 0.1, False), ("squared", True, 0.0, True)])
def test_preference_loss(P, most, V, Vp, kind, average, smoothing, inplace):
    rng = np.random.default_rng(P * most + V)
    start = ragged(rng, 2 * P, most)
    N = int(start[-1]) + 4                                 # rows in front of the first and behind the last sequence
    rng, z, t = rows_case(N, V, Vp, N + V + 1)
    lp, p, keep = PT.token_logps(z, t, V)
    sums = np.array([lp[start[i]:start[i + 1]].sum() / (max(1, keep[start[i]:start[i + 1]].sum()) if average else 1)
                     for i in range(2 * P)])
    ref = (sums + rng.standard_normal(2 * P)).astype(np.float32).astype(np.float64)
    beta, ds = 0.25, 1.0 / P
    rl, rs, rlp, rdz = PT.preference_loss(z, t, V, start, ref=ref, kind=kind, average=average, beta=beta,
                                          smoothing=smoothing, dscale=ds)
    inside = np.zeros(N, bool)
    inside[start[0]:start[-1]] = True
    zb = z.copy()
    zb[~keep & inside] = np.nan
    zd = bf16(zb)
    before = host(zd)
    dz = zd if inplace else torch.full_like(zd, 5.0)
    logps, err = torch.full((N,), 9.0, device="cuda"), err_word()
    seq, losses = torch.empty(2 * P, device="cuda"), torch.empty(P, device="cuda")
    ws = torch.empty(gs.preference_loss_workspace(N, P), dtype=torch.uint8, device="cuda")
    gs.preference_loss(zd, i32(t), i32(start), dz, logps, seq, losses, V, ws, err, ref_logp=f32(ref), kind=kind,
                       average=average, beta=beta, smoothing=smoothing, dscale=ds)
    assert int(err.sum()) == 0
    got, ls = host(dz), host(losses)
    # a sequence's sum: its positions' errors and one rounding; a margin: two sums' and references'
    most_lp = lp_tol(np.abs(lp).max())
    stol = np.diff(start) * most_lp + 2.0 ** -23 * np.abs(rs)
    assert np.all(np.abs(host(logps) - rlp)[inside] <= lp_tol(rlp)[inside])
    assert np.all(host(logps)[~inside] == 9.0)
    assert np.all(np.abs(host(seq) - rs) <= stol)
    dtol = stol[0::2] + stol[1::2]
    slope = np.abs(PT.pair_loss((rs - ref)[0::2] - (rs - ref)[1::2], kind, beta, smoothing)[1])
    assert np.all(np.abs(ls - rl) <= (slope + dtol) * dtol * (1 + beta) + 2.0 ** -22 * np.abs(rl))
    # the coefficient's error: the slope's change over the margin's error (second derivative <= 2) and roundings
    g = np.zeros(N)
    gerr = np.zeros(N)
    for i in range(2 * P):
        n = max(1, int(keep[start[i]:start[i + 1]].sum())) if average else 1
        g[start[i]:start[i + 1]] = slope[i // 2] / n * ds
        gerr[start[i]:start[i + 1]] = 2 * dtol[i // 2] / n * ds
    tol = grad_tol(rdz, g) + gerr[:, None]
    assert np.all((np.abs(got - rdz) <= tol)[inside])
    assert np.all(got[~keep & inside] == 0) and np.all(got[inside][:, V:] == 0)
    untouched = before[~inside] if inplace else np.full_like(before[~inside], 5.0)
    assert np.array_equal(got[~inside], untouched, equal_nan=True)


# pairs of few rows of medium length; long pairs, whose coefficients take a launch of their own
@pytest.mark.parametrize("P,most,V,Vp", [(3, 60, 5001, 5008), (2, 1500, 4700, 4704), (2, 4000, 37, 40)])
@pytest.mark.parametrize("kind,average,smoothing,inplace", [("sigmoid", True, 0.2, True), ("squared", False, 0.0, False)])
def test_preference_loss_by_pair_length(P, most, V, Vp, kind, average, smoothing, inplace):
    test_preference_loss(P, most, V, Vp, kind, average, smoothing, inplace)


def test_preference_loss_of_many_rows_and_without_a_gradient():
    """More rows than the gradient's launch takes on the pairs as well, and losses alone."""
    N, V, Vp, P = 33000, 40, 40, 3
    rng, z, t = rows_case(N, V, Vp, 17)
    start = np.array([0, 30000, 30001, 30001, 31000, 32000, 33000])
    rl, rs, rlp, rdz = PT.preference_loss(z, t, V, start, average=True, beta=0.5, dscale=1.0)
    out = []
    for grad in (True, False):
        dz = torch.full((N, Vp), 5.0, dtype=torch.bfloat16, device="cuda") if grad else None
        logps, losses, seq, err = (torch.empty(N, device="cuda"), torch.empty(P, device="cuda"),
                                   torch.empty(2 * P, device="cuda"), err_word())
        ws = torch.empty(gs.preference_loss_workspace(N, P), dtype=torch.uint8, device="cuda")
        gs.preference_loss(bf16(z), i32(t), i32(start), dz, logps, seq, losses, V, ws, err, average=True, beta=0.5)
        assert np.max(np.abs(host(seq) - rs)) <= lp_tol(np.abs(rlp).max()) + 1e-6
        assert np.max(np.abs(host(losses) - rl)) <= 1e-4 and int(err.sum()) == 0
        out.append((host(losses), host(logps)))
        if grad:
            n = np.array([(t[start[i]:start[i + 1]] != -1).sum() for i in range(2 * P)])
            g = np.repeat(0.5 / np.maximum(n, 1), np.diff(start))
            # the margins' errors change the slope by less than beta^2 times them: 1e-4 of it
            assert np.all(np.abs(host(dz) - rdz) <= grad_tol(rdz, g) + 1e-4 * np.abs(g)[:, None])
    assert all(np.array_equal(a, b) for a, b in zip(*out))


def test_preference_loss_flags_bounds_that_are_not_bounds():
    rng, z, t = rows_case(20, 30, 32, 8, masked=0.0)
    for start in ([0, 5, 9, 4, 20], [0, 5, 10, 15, 21], [-3, 5, 10, 15, 20], [2000000000, 5, 10, 15, 20]):
        err, losses = err_word(), torch.full((2,), 9.0, device="cuda")
        dz = torch.zeros(20, 32, dtype=torch.bfloat16, device="cuda")
        ws = torch.zeros(gs.preference_loss_workspace(20, 2), dtype=torch.uint8, device="cuda")
        gs.preference_loss(bf16(z), i32(t), i32(start), dz, torch.zeros(20, device="cuda"), None, losses, 30, ws, err)
        ok = [0 <= start[2 * p] <= start[2 * p + 1] <= start[2 * p + 2] <= 20 for p in (0, 1)]
        assert int(err[0]) == 1
        assert [float(x) != 0.0 for x in host(losses)] == ok, start
        torch.cuda.synchronize()


def test_token_logps():
    for N, V, Vp in SIZES:
        _, z, t = rows_case(N, V, Vp, 3 * N + V)
        lp, _, _ = PT.token_logps(z, t, V)
        out, err = torch.empty(N, device="cuda"), err_word()
        gs.token_logps(bf16(z), i32(t), out, V, err)
        assert np.all(np.abs(host(out) - lp) <= lp_tol(lp)) and int(err.sum()) == 0


@pytest.mark.parametrize("V,Vp", [(30, 32), (1000, 1024), (9001, 9008), (50257, 50304)])
def test_token_logps_of_rows_with_infinities_and_nan(V, Vp):
    """At every place of a 16-byte piece: -inf has probability 0, a NaN or +inf gives no number."""
    rng = np.random.default_rng(V)
    N = 40
    z = rng.standard_normal((N, Vp)) * 1.5
    z[:, V:] = np.nan                                # padded ids are not read
    t = rng.integers(0, 8, N)
    at = V - 9 - np.arange(8)
    for i in range(8):
        z[i, at[i]] = -np.inf
        z[8 + i, at[i]] = np.nan
        z[16 + i, at[i]] = np.inf
    z[24:32, 8:V] = -np.inf                          # eight ids left
    z[32:36, t[32]] = z[32:36, :V].max() + 130.0     # the others below 2^-127 of the target
    t[32:36] = t[32]
    t[36:] = at[0]
    z[36:, 3] = 250.0                                # the target's log-probability is below -230
    zd = bf16(z)
    out, err = torch.empty(N, device="cuda"), err_word()
    gs.token_logps(zd, i32(t), out, V, err)
    got = host(out)
    assert np.isnan(got[8:24]).all()
    fine = np.r_[0:8, 24:N]
    lp, _, _ = PT.token_logps(host(zd)[fine], t[fine], V)
    assert np.all(np.abs(got[fine] - lp) <= lp_tol(lp))


# -- Newton-Schulz -----------------------------------------------------------------------------

# Bound of the result (relative, Frobenius): bf16 rounding, at most half a step 2^-8 = 3.9e-3; X's
# fp16 rounding before the last two rounds, uniform within half a step (2^-11 / sqrt 3 = 2.8e-4 rms),
# grown by 3.44^2 and 3.44: 4.3e-3; A's and Q's roundings, 2.8e-4 of terms of size up to 5: 1.4e-3 a
# round. In quadrature 3.9, 4.3 and 5 x 1.4 (2 sqrt 5 = 3.1) give 6.6e-3.
NS_TOL = 7e-3
# That averages over many independent roundings. With one singular value there is nothing to
# average, and the half steps (u = 2^-11) add up. It runs 1, 0.70, 1.11, 0.72, 1.13, 0.70. At 1.11 and
# 1.13, Q = -2.8 against a + Q = 0.65: Q's rounding is 4.3 u of the result, A's 0.5 u, X's 1 u; at 0.70
# and 0.72 (Q = -1.9 against 1.6) they are 1.2 u, 0.9 u, 1 u. An error is carried on by s p'(s) / p(s),
# 2.0 at the large values and 0.72 at the small ones: from the end 5.8 u + 2.0 (3.1 u + 0.72 (5.8 u +
# 2.0 (3.1 u + 0.72 (at 1, Q = -2.74: 5 u)))) = 36 u = 1.76e-2, and the result's 2^-8: 2.15e-2.
NS_TOL_ONE = 2.2e-2


def ns_tol(r, c):
    return NS_TOL if min(r, c) >= 16 else NS_TOL_ONE


def spectrum(rng, r, c, power):
    k = min(r, c)
    d = np.arange(1, k + 1) ** -power
    return (rng.standard_normal((r, k)) * d) @ rng.standard_normal((k, c)) * 1e-2


def run_ns(x, steps=5, **kw):
    b, r, c = x.shape if x.dim() == 3 else (1, *x.shape)
    out, err = torch.empty(x.shape, dtype=torch.bfloat16, device="cuda"), err_word()
    ws = torch.empty(gs.orthogonalize_workspace(b, r, c), dtype=torch.uint8, device="cuda").fill_(0xFF)
    gs.orthogonalize(x, out, ws, err, steps=steps, **kw)
    assert int(err.sum()) == 0
    return host(out)


@pytest.mark.parametrize("r,c", [(1, 1), (1, 7), (9, 1), (5, 7), (16, 16), (64, 64), (63, 65), (65, 64), (128, 128),
                                 (129, 127), (130, 257), (300, 200), (257, 1000), (384, 384), (640, 200), (100, 2100),
                                 (513, 770), (100, 140), (128, 256), (77, 333), (520, 96), (1000, 128), (1500, 33),
                                 (128, 2048), (2048, 100), (17, 2049)])
@pytest.mark.parametrize("fp32", [True, False])
def test_orthogonalize(r, c, fp32):
    rng = np.random.default_rng(r * 10000 + c)
    x = np.stack([spectrum(rng, r, c, p) for p in (0.0, 0.5, 1.0)])
    xd = f32(x) if fp32 else bf16(x)
    ref = np.stack([PT.newton_schulz(m) for m in host(xd)])
    got = run_ns(xd)
    for g, q in zip(got, ref):
        assert rel_l2(g, q) <= ns_tol(r, c)
    assert np.array_equal(run_ns(xd[1]), got[1])           # a matrix alone, the same bits
    many = xd.repeat(20, 1, 1) if r * c < 300000 else xd    # more matrices than fit at a time
    assert np.array_equal(run_ns(many)[-3:], got)


@pytest.mark.parametrize("steps", [1, 2, 3, 4, 6, 8])
def test_orthogonalize_other_step_counts(steps):
    rng = np.random.default_rng(steps)
    x = f32(spectrum(rng, 150, 220, 0.5))
    assert rel_l2(run_ns(x, steps=steps), PT.newton_schulz(host(x), steps)) <= NS_TOL


def test_orthogonalize_gives_singular_values_near_one():
    rng = np.random.default_rng(3)
    s = np.linalg.svd(run_ns(f32(rng.standard_normal((200, 330)))), compute_uv=False)
    assert 0.6 < s.min() and s.max() < 1.25


def test_orthogonalize_scales_zeros_and_non_finite_matrices():
    rng = np.random.default_rng(4)
    x = np.stack([spectrum(rng, 70, 90, 0.5)] * 6)
    x[1] = 0.0
    x[2, 3, 4] = np.nan
    x[3, 69, 89] = np.inf
    x[4] *= 2.0 ** 90
    x[5] *= 2.0 ** 20
    got = run_ns(f32(x))
    ref = PT.newton_schulz(host(f32(x[0])))
    assert np.all(got[1] == 0) and np.isnan(got[2]).all() and np.isnan(got[3]).any()
    for i in (0, 4, 5):
        assert rel_l2(got[i], ref) <= NS_TOL


def test_orthogonalize_strided_and_unaligned_matrices():
    rng = np.random.default_rng(5)
    for dt in (torch.float32, torch.bfloat16):
        big = torch.tensor(rng.standard_normal(5000), device="cuda").to(dt)
        x = torch.as_strided(big, (3, 20, 31), (701, 31, 1), 3)        # element-aligned only
        out = torch.full((3, 1000), 4.0, dtype=torch.bfloat16, device="cuda")
        o = torch.as_strided(out, (3, 20, 31), (777, 31, 1), 1)
        ws, err = torch.empty(gs.orthogonalize_workspace(3, 20, 31), dtype=torch.uint8, device="cuda"), err_word()
        gs.orthogonalize(x, o, ws, err)
        for i in range(3):
            assert rel_l2(host(o[i]), PT.newton_schulz(host(x[i]))) <= NS_TOL
        flat = host(out).ravel()
        for a, b in ((0, 1), (1 + 620, 778), (778 + 620, 1555), (1555 + 620, 3000)):
            assert np.all(flat[a:b] == 4.0)
    # matrices and their results in turn in one buffer
    buf = torch.empty(3, 20 * 31 * 3, dtype=torch.bfloat16, device="cuda")
    x, o = buf[:, :1240].view(torch.float32).view(3, 20, 31), buf[:, 1240:].view(3, 20, 31)
    x.copy_(torch.tensor(rng.standard_normal((3, 20, 31))))
    given = host(x).copy()
    gs.orthogonalize(x, o, ws, err)
    assert np.array_equal(host(x), given)
    for i in range(3):
        assert rel_l2(host(o[i]), PT.newton_schulz(given[i])) <= NS_TOL
    with pytest.raises(gs.GPT2Error):
        gs.orthogonalize(x, buf[:, 1239:1859].as_strided((3, 20, 31), (1860, 31, 1)), ws, err)


@pytest.mark.parametrize("b,r,c", [(12, 768, 768), (2, 2304, 768), (3, 384, 1536), (1, 1536, 6144)])
def test_orthogonalize_at_weight_sizes(b, r, c):
    gen = torch.Generator(device="cuda").manual_seed(r + c)
    x = torch.randn(b, r, c, device="cuda", generator=gen)
    k = min(r, c)
    x[0] = (torch.randn(r, k, device="cuda", generator=gen) / torch.arange(1, k + 1, device="cuda")) @ x[0, :k] \
        if r >= c else torch.randn(r, k, device="cuda", generator=gen) / torch.arange(1, k + 1, device="cuda") @ x[0]
    got = run_ns(x)
    a, q, cc = PT.NS_COEFFS
    for i in range(b):
        y = x[i].double()
        y = y / (y.norm() + 1e-7)
        y = y.T if r > c else y
        for _ in range(5):
            g = y @ y.T
            y = a * y + (q * g + cc * (g @ g)) @ y
        ref = (y.T if r > c else y).cpu().numpy()
        assert rel_l2(got[i], ref) <= NS_TOL


# -- streams, graphs ---------------------------------------------------------------------------

def test_operators_on_another_stream_and_in_a_graph():
    rng, z, t = rows_case(48, 1000, 1024, 11)
    lp, keep, old, ref, adv, w = policy_inputs(rng, z, t, 1000)
    start = np.array([0, 10, 20, 33, 48])
    x = rng.standard_normal((2, 90, 60))
    b = dict(z=bf16(z), t=i32(t), old=f32(old), adv=f32(adv), start=i32(start), x=f32(x))
    o = dict(dz=torch.empty_like(b["z"]), lp=torch.empty(48, device="cuda"), ls=torch.empty(48, device="cuda"),
             dz2=torch.empty_like(b["z"]), lp2=torch.empty(48, device="cuda"), pl=torch.empty(2, device="cuda"),
             x=torch.empty(2, 90, 60, dtype=torch.bfloat16, device="cuda"))
    ws = torch.empty(gs.preference_loss_workspace(48, 2), dtype=torch.uint8, device="cuda")
    wx = torch.empty(gs.orthogonalize_workspace(2, 90, 60), dtype=torch.uint8, device="cuda")
    err = err_word()

    def all_three(stream=None):
        gs.policy_loss(b["z"], b["t"], b["old"], b["adv"], o["dz"], o["lp"], o["ls"], 1000, err, stream=stream)
        gs.preference_loss(b["z"], b["t"], b["start"], o["dz2"], o["lp2"], None, o["pl"], 1000, ws, err, stream=stream)
        gs.orthogonalize(b["x"], o["x"], wx, err, stream=stream)

    def take():
        torch.cuda.synchronize()
        return [host(v) for v in o.values()]

    all_three()
    first = take()
    side = torch.cuda.Stream()
    for v in o.values():
        v.zero_()
    torch.cuda.synchronize()
    all_three(side)                                        # the stream as an argument
    assert all(np.array_equal(a, c) for a, c in zip(first, take()))
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        all_three()
    with torch.cuda.graph(g2):                             # shares the workspaces; replayed in order
        all_three()
    for v in o.values():
        v.zero_()
    g1.replay()
    assert all(np.array_equal(a, c) for a, c in zip(first, take()))
    b["x"].copy_(f32(rng.standard_normal((2, 90, 60))))    # new inputs in the same buffers
    b["adv"].mul_(-1)
    g2.replay()
    g1.replay()
    replayed = take()
    for v in o.values():
        v.zero_()
    all_three()
    assert all(np.array_equal(a, c) for a, c in zip(replayed, take()))
    assert not np.array_equal(replayed[0], first[0]) and not np.array_equal(replayed[-1], first[-1])


@pytest.mark.parametrize("b,r,c", [(3, 333, 517), (1, 700, 300), (4, 100, 900)])
def test_orthogonalize_captured_replayed_and_twice_at_once(b, r, c):
    """Every launch form in a graph, and two calls at a time on two streams with workspaces of their own."""
    rng = np.random.default_rng(b * r + c)
    xs = [f32(rng.standard_normal((b, r, c))) for _ in range(2)]
    ref = [run_ns(x) for x in xs]
    outs = [torch.zeros(b, r, c, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    wss = [torch.empty(gs.orthogonalize_workspace(b, r, c), dtype=torch.uint8, device="cuda") for _ in range(2)]
    err = err_word()
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            gs.orthogonalize(xs[i], outs[i], wss[i], err, stream=streams[i])
    torch.cuda.synchronize()
    assert all(np.array_equal(host(outs[i]), ref[i]) for i in range(2)) and int(err.sum()) == 0
    buf = xs[0].clone()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g in graphs:                                        # two graphs on one workspace, replayed in order
        with torch.cuda.graph(g):
            gs.orthogonalize(buf, outs[0], wss[0], err)
    outs[0].zero_()
    graphs[0].replay()
    torch.cuda.synchronize()
    assert np.array_equal(host(outs[0]), ref[0])
    buf.copy_(xs[1])
    graphs[1].replay()
    graphs[0].replay()
    torch.cuda.synchronize()
    assert np.array_equal(host(outs[0]), ref[1]) and int(err.sum()) == 0


@pytest.mark.parametrize("V,Vp,T", [(1000, 1024, 37), (4353, 4480, 148), (9001, 9008, 64)])
def test_policy_loss_over_more_rows_than_stay_resident(V, Vp, T):
    """Rows in windows, most of them left out, the last window short: every row is written once."""
    N = 9000 if V < 4000 else 6000
    gen = torch.Generator(device="cuda").manual_seed(V)
    z = torch.randn(N, Vp, device="cuda", generator=gen).to(torch.bfloat16)
    t = torch.randint(0, V, (N,), device="cuda", generator=gen)
    t[torch.arange(N, device="cuda") % T < int(0.7 * T)] = -1
    t = t.to(torch.int32)
    lp = torch.log_softmax(z[:, :V].double(), 1).gather(1, t.clamp(min=0).long()[:, None])[:, 0]
    old = (lp - 0.1).float()
    dz, logps, losses = torch.full_like(z, 3.0), torch.full((N,), 5.0, device="cuda"), torch.full((N,), 5.0, device="cuda")
    err = err_word()
    gs.policy_loss(z, t, old, torch.ones(N, device="cuda"), dz, logps, losses, V, err)
    keep = t >= 0
    want = torch.where(keep, lp, 0.0).cpu().numpy()
    assert np.all(np.abs(host(logps) - want) <= np.where(keep.cpu().numpy(), lp_tol(want), 0.0))
    g = torch.where(keep, -torch.exp(lp - old.double()), 0.0)
    ref = -g[:, None] * torch.softmax(z[:, :V].double(), 1)
    ref[torch.arange(N, device="cuda"), t.clamp(min=0).long()] += g
    off = (dz[:, :V].double() - ref).abs()
    tol = 2.0 ** -8 * ref.abs() * (1 + 2.0 ** -6) + 2.0 ** -17 * g.abs()[:, None] + 1e-38
    assert bool((off <= tol).all()) and bool((dz[:, V:] == 0).all()) and bool((dz[~keep] == 0).all())
    assert int(err.sum()) == 0
    seq = torch.tensor([0, 11, N - 1500, N - 700, N - 3], dtype=torch.int32, device="cuda")
    out2 = torch.full((N,), 5.0, device="cuda")
    ws = torch.empty(gs.preference_loss_workspace(N, 2), dtype=torch.uint8, device="cuda")
    dz2 = torch.full_like(z, 3.0)
    gs.preference_loss(z, t, seq, dz2, out2, None, torch.empty(2, device="cuda"), V, ws, err)
    assert torch.equal(out2[:N - 3], logps[:N - 3]) and bool((out2[N - 3:] == 5.0).all())
    assert bool((dz2[N - 3:] == 3.0).all()) and bool((dz2[:N - 3][~keep[:N - 3]] == 0).all())
    assert bool((dz2[:N - 3][keep[:N - 3]][:, :V] != 3.0).all())


# -- the model calls ---------------------------------------------------------------------------

# bars of the whole step for bf16 activations, as in test_gpu_model.py
LOSS_TOL, GRAD_TOL = 2e-2, 3e-2


def tiny(**over):
    args = workloads.model_args("tiny", **over)
    return gs.GPT2(gs.Config.make(**args), 1337), G.Config(**args)


def tiny_batch(ocfg, seed, B=None):
    rng = np.random.default_rng(seed)
    B = B or ocfg.micro_batch
    x = rng.integers(0, ocfg.V, (B, ocfg.T))
    y = np.concatenate([x[:, 1:], rng.integers(0, ocfg.V, (B, 1))], 1)
    y[:, : ocfg.T // 4] = -1                                # a prompt
    y[1, ocfg.T // 2:] = -1                                 # a shorter answer
    return rng, x, y


def oracle_grads(ocfg, params, x, dz):
    _, _, cache = G.forward(ocfg, params, x)
    cache["dz"] = dz
    return G.backward(ocfg, params, cache)


def check_grads(ocfg, got, ref):
    ref = G.split_named(ocfg, ref)
    whole = {n: np.linalg.norm(ref[n]) for n in ref}
    for n, a in got.items():
        if n.endswith("attn.c_attn.bias"):                  # the key third is exactly 0 on one side
            C = a.shape[0] // 3
            a, r = np.delete(a, slice(C, 2 * C)), np.delete(ref[n], slice(C, 2 * C))
        else:
            r = ref[n]
        assert rel_l2(a, r) <= GRAD_TOL, (n, rel_l2(a, r), whole[n])


@pytest.mark.parametrize("B", [4, 2])                       # 256 rows: paired GEMM and its partials; 128 rows: row scans
def test_token_logps_of_the_model(B):
    m, ocfg = tiny(micro_batch=B)
    _, x, y = tiny_batch(ocfg, 1, B=7)                      # whole micro-batches and a part of one
    out = torch.full((7, ocfg.T), 3.0, device="cuda")
    m.token_logps(i32(x), i32(y), out)
    p = G.init_params(ocfg, 1337)
    z = G.forward(ocfg, p, x)[2]["logits"]
    lp, _, keep = PT.token_logps(z, y.reshape(-1), ocfg.V)
    got = host(out).ravel()
    assert np.max(np.abs(got - lp)) <= LOSS_TOL and np.all(got[~keep] == 0)
    assert math.isfinite(m.fwd_bwd(i32(x[:B]), i32(np.maximum(y[:B], 0)), want_loss=True))


@pytest.mark.parametrize("B,V", [(4, 1000), (2, 1000), (4, 50257), (2, 20001)])
def test_policy_micro_step_of_the_model(B, V):
    m, ocfg = tiny(micro_batch=B, vocab_real=V)
    rng, x, y = tiny_batch(ocfg, 2)
    n = x.size
    p = G.init_params(ocfg, 1337)
    z = G.forward(ocfg, p, x)[2]["logits"]
    lp, _, keep = PT.token_logps(z, y.reshape(-1), ocfg.V)
    # log-ratios of 0.1 and 0.5 in size: further from the clip borders (0.18 .. 0.22) than bf16 activations move lp
    old = lp - rng.choice([-0.5, -0.1, 0.1, 0.5], n)
    ref = lp + 0.3 * rng.standard_normal(n)
    adv = np.repeat(rng.standard_normal(B), ocfg.T)
    scale = 1.0 / keep.sum()
    losses, _, dz = PT.policy_loss(z, y.reshape(-1), ocfg.V, old, adv, ref=ref, kl=0.1, dscale=scale)
    logps = torch.empty(B, ocfg.T, device="cuda")
    f = lambda a: f32(a.reshape(B, ocfg.T))  # noqa: E731
    loss = m.fwd_bwd_policy(i32(x), i32(y), f(old), f(adv), ref_logp=f(ref), kl_coef=0.1, scale=scale, logps=logps,
                            want_loss=True)
    assert abs(loss - scale * losses.sum()) <= LOSS_TOL
    assert np.max(np.abs(host(logps).ravel() - lp)) <= LOSS_TOL
    assert abs(m.token_losses().sum() * scale - loss) <= 1e-5
    check_grads(ocfg, m.read_all(gs.GPT2_GRADS), oracle_grads(ocfg, p, x, dz))


@pytest.mark.parametrize("B,kind,average,V", [(4, "sigmoid", False, 1000), (2, "squared", True, 1000),
                                              (4, "sigmoid", False, 50257)])
def test_preference_micro_step_of_the_model(B, kind, average, V):
    m, ocfg = tiny(micro_batch=B, vocab_real=V)
    rng, x, y = tiny_batch(ocfg, 3)
    p = G.init_params(ocfg, 1337)
    z = G.forward(ocfg, p, x)[2]["logits"]
    start = np.arange(B + 1) * ocfg.T
    _, score, lp, _ = PT.preference_loss(z, y.reshape(-1), ocfg.V, start, average=average)
    ref = score + rng.standard_normal(B)
    losses, _, _, dz = PT.preference_loss(z, y.reshape(-1), ocfg.V, start, ref=ref, kind=kind, average=average,
                                          beta=0.2, dscale=2.0 / B)
    seq = torch.empty(B, device="cuda")
    loss = m.fwd_bwd_preference(i32(x), i32(y), ref_logp=f32(ref), kind=kind, average=average, beta=0.2, seq_logps=seq,
                                want_loss=True)
    n = 1 if average else ocfg.T
    assert np.max(np.abs(host(seq) - score)) <= LOSS_TOL * math.sqrt(n)
    assert abs(loss - losses.mean()) <= LOSS_TOL * math.sqrt(n)
    assert np.max(np.abs(m.token_losses().ravel() - lp)) <= LOSS_TOL
    check_grads(ocfg, m.read_all(gs.GPT2_GRADS), oracle_grads(ocfg, p, x, dz))


def test_preference_micro_step_needs_an_even_micro_batch():
    m, ocfg = tiny(micro_batch=3)
    _, x, y = tiny_batch(ocfg, 3)
    with pytest.raises(gs.GPT2Error):
        m.fwd_bwd_preference(i32(x), i32(y))


def test_muon_step():
    """The update on given gradients, two steps, against the definition in 64 bits."""
    m, ocfg = tiny(warmup_steps=3, total_steps=10)
    ws = torch.empty(gs.muon_workspace(m.cfg), dtype=torch.uint8, device="cuda")
    with pytest.raises(gs.GPT2Error):                       # no micro-step yet
        m.clip_muon(0, ws)
    params = G.init_params(ocfg, 1337)
    om, ov = G.zeros_like_params(ocfg), G.zeros_like_params(ocfg)
    names = [t.name for t in m.tensors()]
    kinds = {n: k for n, k, _, _ in G.tensor_names(ocfg)}
    for step in range(2):
        _, x, y = tiny_batch(ocfg, 10 + step)
        m.fwd_bwd(i32(x), i32(np.maximum(y, 0)))
        grads = m.read_all(gs.GPT2_GRADS)
        full = {k: np.zeros_like(v) for k, v in params.items()}
        for (n, k, layer, _) in G.tensor_names(ocfg):
            if layer < 0:
                full[k][...] = grads[n]
            else:
                full[k][layer] = grads[n]
        before = {n: a.copy() for n, a in G.split_named(ocfg, params).items()}
        norm = m.clip_muon(step, ws, want_norm=True)
        onorm = PT.clip_muon(ocfg, params, full, om, ov, step)
        assert abs(norm - onorm) <= 1e-5 * onorm
        got, ref = m.read_all(gs.GPT2_PARAMS), G.split_named(ocfg, params)
        gm, rm = m.read_all(gs.GPT2_ADAM_M), G.split_named(ocfg, om)
        for n in names:
            if kinds[n] in PT.MUON_KINDS:
                # fp32 storage of w, and the update within the orthogonalisation's bound
                moved = np.linalg.norm(ref[n] - before[n])
                assert np.linalg.norm(got[n] - ref[n]) <= NS_TOL * moved + 2.0 ** -22 * np.linalg.norm(ref[n]), n
                assert moved > 0
            else:
                assert rel_l2(got[n], ref[n]) <= 2e-6, n
            assert rel_l2(gm[n], rm[n]) <= 1e-5, n
        for n, a in got.items():                            # both sides go on from the same weights
            k, layer = next((kk, l) for nn, kk, l, _ in G.tensor_names(ocfg) if nn == n)
            if layer < 0:
                params[k] = a.astype(np.float64)
            else:
                params[k][layer] = a
        assert all(np.all(g == 0) for g in m.read_all(gs.GPT2_GRADS).values())
        assert torch.equal(m.state_tensor(gs.GPT2_WEIGHTS_BF16), m.state_tensor(gs.GPT2_PARAMS).to(torch.bfloat16))


def test_muon_leaves_the_weights_of_a_non_finite_step():
    m, ocfg = tiny()
    ws = torch.empty(gs.muon_workspace(m.cfg), dtype=torch.uint8, device="cuda")
    _, x, y = tiny_batch(ocfg, 1)
    m.fwd_bwd(i32(x), i32(np.maximum(y, 0)))
    before = {w: m.state_tensor(w).clone() for w in (gs.GPT2_PARAMS, gs.GPT2_ADAM_M, gs.GPT2_ADAM_V)}
    m.state_tensor(gs.GPT2_GRADS)[-7680] = float("inf")
    with pytest.raises(gs.GPT2Error) as e:
        m.clip_muon(0, ws, want_norm=True)
    assert e.value.status == 4
    for w, a in before.items():
        assert torch.equal(m.state_tensor(w), a)
    assert int(m.state_tensor(gs.GPT2_GRADS).count_nonzero()) == 0
    with pytest.raises(gs.GPT2Error):
        m.clip_muon(0, ws[:-256])


def test_post_training_run():
    """Reference log-probabilities, preference micro-steps, policy micro-steps and both updates in one run."""
    m, ocfg = tiny(max_lr=2e-3, warmup_steps=0, total_steps=50)
    ws = torch.empty(gs.muon_workspace(m.cfg), dtype=torch.uint8, device="cuda")
    rng, x, y = tiny_batch(ocfg, 21)
    xt, yt = i32(x), i32(y)
    lp = torch.empty(4, ocfg.T, device="cuda")
    m.token_logps(xt, yt, lp)
    ref = lp.sum(1)
    seq = torch.empty(4, device="cuda")
    first = m.fwd_bwd_preference(xt, yt, ref_logp=ref, seq_logps=seq, want_loss=True)
    # against its own log-probabilities every margin is 0; the two sums differ by fp32 summation order
    assert abs(first - math.log(2)) <= 1e-4 and torch.allclose(seq, ref, rtol=1e-5)
    m.fwd_bwd_preference(xt, yt, ref_logp=ref)
    assert m.clip_muon(0, ws, want_norm=True) > 0
    loss = m.fwd_bwd_preference(xt, yt, ref_logp=ref, want_loss=True)
    assert math.isfinite(loss) and loss != first
    m.clip_adamw(1)
    mean, norm = m.last_step_stats()
    assert abs(mean - loss) <= 1e-5 and norm > 0
    adv = torch.tensor([1.0, -1.0, 0.5, 0.0], device="cuda")[:, None].expand(4, ocfg.T).contiguous()
    m.token_logps(xt, yt, lp)
    now = torch.empty_like(lp)
    kept = int((yt != -1).sum())
    loss = m.fwd_bwd_policy(xt, yt, lp, adv, ref_logp=lp, kl_coef=0.1, scale=1.0 / kept, logps=now, want_loss=True)
    # on the sampling policy itself the ratio is 1 and the KL term 0
    assert torch.equal(now, lp)
    assert abs(loss + float((adv * (yt != -1)).sum()) / kept) <= 1e-5
    m.clip_muon(2, ws)
    assert m.last_step_stats()[1] > 0
    assert math.isfinite(m.eval_loss(xt, i32(np.maximum(y, 0))))
