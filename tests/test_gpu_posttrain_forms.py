"""The preference loss in each of its launch forms: rows by warp or by CTA, the pair's
coefficient in the gradient's launch or in one of its own, pairs alike and one with nearly
all rows. Bounds and cases are those of test_gpu_posttrain.py."""
import numpy as np
import pytest

import gpt_step_b200 as gs
from oracle import posttrain as PT

from gpu_util import bf16, err_word, f32, host, i32, require_gpu, torch
from test_gpu_posttrain import grad_tol, lp_tol, rows_case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("N,V,Vp", [(1024, 500, 504), (1025, 500, 504), (1026, 3079, 3080), (2895, 40, 40), (2900, 40, 40),
                                    (1448, 5001, 5008), (1450, 5001, 5008), (1030, 2049, 2056), (300, 16385, 16392),
                                    (4100, 700, 704)])
@pytest.mark.parametrize("skew", [False, True])
@pytest.mark.parametrize("average", [False, True])
def test_preference_loss_in_every_form(N, V, Vp, skew, average):
    P = 5
    lens = np.full(2 * P, N // (2 * P))
    if skew:
        lens[:] = [1, 0, N - 20, 3, 2, 2, 0, 0, 4, 1]
    start = np.concatenate([[0], np.cumsum(lens)])
    assert start[-1] <= N                                  # rows behind the last sequence
    rng, z, t = rows_case(N, V, Vp, N + V + skew)
    ref = rng.standard_normal(2 * P).astype(np.float32).astype(np.float64)
    lp, _, keep = PT.token_logps(z, t, V)
    sums = np.array([lp[start[i]:start[i + 1]].sum() / (max(1, keep[start[i]:start[i + 1]].sum()) if average else 1)
                     for i in range(2 * P)])
    ref = (sums + ref).astype(np.float32).astype(np.float64)
    beta, eps = 0.25, 0.1
    rl, rs, rlp, rdz = PT.preference_loss(z, t, V, start, ref=ref, average=average, beta=beta, smoothing=eps)
    inside = np.arange(N) < start[-1]
    zd = bf16(z)
    dz, logps = torch.full_like(zd, 5.0), torch.full((N,), 9.0, device="cuda")
    seq, losses, err = torch.empty(2 * P, device="cuda"), torch.empty(P, device="cuda"), err_word()
    ws = torch.empty(gs.preference_loss_workspace(N, P), dtype=torch.uint8, device="cuda").fill_(0xFF)
    gs.preference_loss(zd, i32(t), i32(start), dz, logps, seq, losses, V, ws, err, ref_logp=f32(ref), average=average,
                       beta=beta, smoothing=eps)
    assert int(err.sum()) == 0
    got = host(dz)
    stol = np.maximum(lens, 1) * lp_tol(np.abs(lp).max()) + 2.0 ** -23 * np.abs(rs)
    dtol = stol[0::2] + stol[1::2]
    assert np.all(np.abs(host(logps) - rlp)[inside] <= lp_tol(rlp)[inside]) and np.all(host(logps)[~inside] == 9.0)
    assert np.all(np.abs(host(seq) - rs) <= stol)
    # the loss's slope is below beta, its second derivative below beta^2 / 4
    assert np.all(np.abs(host(losses) - rl) <= beta * dtol + 2.0 ** -22 * np.abs(rl))
    n = np.array([max(1, int(keep[start[i]:start[i + 1]].sum())) if average else 1 for i in range(2 * P)])
    g, gerr = np.zeros(N), np.zeros(N)
    g[inside] = np.repeat(beta / n, lens)
    gerr[inside] = np.repeat(beta ** 2 / 4 * np.repeat(dtol, 2) / n, lens)
    assert np.all((np.abs(got - rdz) <= grad_tol(rdz, g) + gerr[:, None])[inside])
    assert np.all(got[~inside] == 5.0) and np.all(got[inside][:, V:] == 0)


def test_rows_past_two_to_the_31_elements():
    """The last rows of 44,000 x 50,304 logits give what they give by themselves, to the bit."""
    N, V, Vp, n = 44000, 50257, 50304, 300
    gen = torch.Generator(device="cuda").manual_seed(1)
    z = torch.empty(N, Vp, dtype=torch.bfloat16, device="cuda").normal_(0.0, 2.0, generator=gen)
    t = torch.randint(0, V, (N,), dtype=torch.int32, device="cuda", generator=gen)
    old = torch.full((N,), -11.0, device="cuda")
    adv = torch.randn(N, device="cuda", generator=gen)
    logps, losses, err = torch.empty(N, device="cuda"), torch.empty(N, device="cuda"), err_word()
    dz = torch.full_like(z, 3.0)
    last = slice(N - n, N)
    lp1, ls1, dz1 = torch.empty(n, device="cuda"), torch.empty(n, device="cuda"), torch.empty_like(z[last])
    gs.policy_loss(z, t, old, adv, dz, logps, losses, V, err)
    gs.policy_loss(z[last], t[last], old[last], adv[last], dz1, lp1, ls1, V, err)
    assert torch.equal(dz[last], dz1) and torch.equal(logps[last], lp1) and torch.equal(losses[last], ls1)
    out = []
    for rows, first in ((slice(0, N), N - n), (last, 0)):
        dz.fill_(3.0)
        seq, pair = torch.empty(4, device="cuda"), torch.empty(2, device="cuda")
        start = i32([first, first, first + 90, first + 200, first + n - 7])
        ws = torch.empty(gs.preference_loss_workspace(z[rows].shape[0], 2), dtype=torch.uint8, device="cuda")
        gs.preference_loss(z[rows], t[rows], start, dz[rows], logps[rows], seq, pair, V, ws, err)
        out.append((seq, pair, logps[last][:n - 7].clone(), dz[last].clone()))
    assert all(torch.equal(a, b) for a, b in zip(*out))
    assert bool((out[0][3][n - 7:] == 3.0).all()) and int(err.sum()) == 0
