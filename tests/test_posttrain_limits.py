"""The post-training definitions where numbers end, on the CPU."""
import ctypes

import numpy as np

import gpt_step_b200 as gs
from gpt_step_b200 import build
from oracle import posttrain as PT


def rows(**kw):
    a = dict(lp=-1.0, old=-1.0, adv=1.0, ref=None, w=1.0)
    a.update(kw)
    n = 1
    f = lambda v: None if v is None else np.full(n, v)  # noqa: E731
    with np.errstate(invalid="ignore"):
        loss, g = PT.policy_rows(f(a["lp"]), f(a["old"]), f(a["adv"]), f(a["ref"]), f(a["w"]), 0.2, 0.2,
                                 0.1 if a["ref"] is not None else 0.0)
    return float(loss[0]), float(g[0])


def test_a_policy_row_with_a_nan_has_no_loss_and_no_slope():
    nan, inf = np.nan, np.inf
    for bad in (dict(lp=nan), dict(old=nan), dict(adv=nan), dict(w=nan), dict(ref=nan), dict(lp=nan, adv=0.0),
                dict(lp=-inf, old=-inf)):
        assert all(np.isnan(rows(**bad))), bad
    for fine in (dict(old=nan), dict(old=-inf), dict(old=inf), dict(lp=-inf, old=-inf)):
        assert rows(adv=0.0, **fine) == (0.0, 0.0), fine      # an advantage of 0 gives 0 for any ratio


def test_a_pair_whose_margin_is_infinite_has_its_limits():
    delta = np.array([np.inf, -np.inf, 3000.0, -3000.0])
    loss, d = PT.pair_loss(delta, "sigmoid", 0.5, 0.0)
    assert loss.tolist() == [0.0, np.inf, 0.0, 1500.0] and d.tolist() == [0.0, -0.5, 0.0, -0.5]
    loss, d = PT.pair_loss(delta, "sigmoid", 0.5, 0.25)
    assert loss.tolist() == [np.inf, np.inf, 375.0, 1125.0] and d.tolist() == [0.125, -0.375, 0.125, -0.375]
    assert np.isnan(PT.pair_loss(np.array([np.nan]), "sigmoid", 0.5, 0.0)[0]).all()


def test_the_kl_term_of_infinite_log_ratios_is_infinite():
    assert rows(lp=-np.inf, old=0.0, ref=-1.0) == (np.inf, -np.inf)      # ruled out by the policy alone
    loss, g = rows(ref=-np.inf)                                          # and by the reference alone
    assert loss == np.inf and g == -1.0 + 0.1


def test_preference_loss_refuses_outputs_over_the_reference():
    """Arguments are checked before any is read: the pointers stand for device memory."""
    build.build()
    at = lambda k: ctypes.c_void_p(4096 + 4 * k)  # noqa: E731  float k of one buffer
    far, F = ctypes.c_void_p(1 << 20), ctypes.c_float

    def pref(ref, logps, seq, losses, N=40, P=4):
        return gs.lib().gpt2op_preference_loss(far, far, far, ref, None, logps, seq, losses, N, P, 100, 104, -1, 0, 0,
                                               F(0.1), F(0.0), F(1.0), far, 40 * 8 + 4 * 8, far, None)
    for bad in (dict(seq=at(0)), dict(seq=at(7)), dict(losses=at(7)), dict(losses=at(-3)), dict(logps=at(7)),
                dict(logps=at(-39))):
        args = dict(ref=at(0), logps=far, seq=None, losses=far)
        args.update(bad)
        assert pref(**args) == 1, bad
