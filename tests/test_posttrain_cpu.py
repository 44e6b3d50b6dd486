"""The post-training definitions (finite differences, closed forms) and the refusals
of the entry points, without a GPU."""
import ctypes

import numpy as np
import pytest

import gpt_step_b200 as gs
from gpt_step_b200 import build, workloads
from oracle import posttrain as PT

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lib():
    build.build()
    return gs.lib()


# -- the definitions ---------------------------------------------------------------------------

def _logits(N, V, Vp, seed):
    rng = np.random.default_rng(seed)
    z = rng.standard_normal((N, Vp)) * 1.5
    t = rng.integers(0, V, N)
    t[::4] = -1
    return rng, z, t


def _differences(f, z, at, h=1e-5):
    out = []
    for i, j in at:
        up, down = z.copy(), z.copy()
        up[i, j] += h
        down[i, j] -= h
        out.append((f(up) - f(down)) / (2 * h))
    return np.array(out)


@pytest.mark.parametrize("kl", [0.0, 0.3])
def test_policy_gradient_is_the_derivative(kl):
    rng, z, t = _logits(9, 11, 16, 1)
    lp, _, keep = PT.token_logps(z, t, 11)
    old = lp + 0.3 * rng.standard_normal(9)
    r = np.exp(lp - old)
    assert np.all(np.abs(r - 0.8)[keep] > 1e-3) and np.all(np.abs(r - 1.2)[keep] > 1e-3)
    args = dict(old=old, adv=rng.standard_normal(9), ref=lp + 0.2 * rng.standard_normal(9),
                weight=rng.uniform(0.5, 2, 9), kl=kl, dscale=0.7)
    _, _, dz = PT.policy_loss(z, t, 11, **args)
    at = [(i, j) for i in range(9) for j in range(16)]
    num = _differences(lambda q: 0.7 * PT.policy_loss(q, t, 11, **args)[0].sum(), z, at)
    # central differences: truncation h^2 f''' ~ 1e-10, rounding 1e-16 / h ~ 1e-11
    assert np.max(np.abs(num - dz.ravel())) < 1e-8
    assert np.all(dz[:, 11:] == 0) and np.all(dz[~keep] == 0)


@pytest.mark.parametrize("kind,average,smoothing", [("sigmoid", False, 0.0), ("sigmoid", True, 0.2),
                                                    ("squared", True, 0.0), ("squared", False, 0.0)])
def test_preference_gradient_is_the_derivative(kind, average, smoothing):
    rng, z, t = _logits(14, 7, 8, 2)
    start = np.array([0, 3, 3, 9, 13])
    args = dict(ref=rng.standard_normal(4), kind=kind, average=average, smoothing=smoothing, beta=0.4, dscale=0.5)
    losses, score, lp, dz = PT.preference_loss(z, t, 7, start, **args)
    assert losses.shape == (2,) and score[1] == 0.0
    at = [(i, j) for i in range(14) for j in range(8)]
    num = _differences(lambda q: 0.5 * PT.preference_loss(q, t, 7, start, **args)[0].sum(), z, at)
    assert np.max(np.abs(num - dz.ravel())) < 1e-7
    assert np.all(dz[13] == 0)


def test_policy_on_the_sampling_policy_is_the_plain_policy_gradient():
    """At old = lp the ratio is 1: loss -A, gradient -A (onehot - p)."""
    rng, z, t = _logits(8, 10, 16, 3)
    lp, p, keep = PT.token_logps(z, t, 10)
    adv = rng.standard_normal(8)
    losses, _, dz = PT.policy_loss(z, t, 10, lp, adv)
    assert np.allclose(losses, np.where(keep, -adv, 0), atol=1e-15)
    i = int(np.flatnonzero(keep)[0])
    assert np.isclose(dz[i, t[i]], -adv[i] * (1 - p[i, t[i]]), rtol=1e-12)


def test_newton_schulz_moves_singular_values_by_the_quintic():
    rng = np.random.default_rng(4)
    for shape in ((6, 9), (9, 6), (5, 5)):
        x = rng.standard_normal(shape)
        u, s, vt = np.linalg.svd(x, full_matrices=False)
        q = s / (np.linalg.norm(x) + 1e-7)
        a, b, c = PT.NS_COEFFS
        for _ in range(5):
            q = a * q + b * q ** 3 + c * q ** 5
        assert np.max(np.abs(PT.newton_schulz(x) - (u * q) @ vt)) < 1e-10
    assert np.all(PT.newton_schulz(np.zeros((3, 4))) == 0)


# -- refusals ----------------------------------------------------------------------------------

D = ctypes.c_void_p(4096)     # never dereferenced: the checks come first
ODD = ctypes.c_void_p(4100)
F = ctypes.c_float


def test_loss_entry_points_refuse_bad_arguments(lib):
    inf, nan = float("inf"), float("nan")

    def policy(logits=D, targets=D, old=D, ref=D, adv=D, w=None, dl=D, lp=D, losses=D, N=4, V=100, Vp=128, ign=-1,
               lo=0.2, hi=0.2, kl=0.1, ds=1.0, err=D):
        return lib.gpt2op_policy_loss(logits, targets, old, ref, adv, w, dl, lp, losses, N, V, Vp, ign, F(lo), F(hi),
                                      F(kl), F(ds), err, None)
    for bad in (dict(logits=None), dict(targets=None), dict(old=None), dict(adv=None), dict(losses=None),
                dict(err=None), dict(N=0), dict(V=0), dict(V=129), dict(Vp=125, V=100), dict(logits=ODD),
                dict(dl=ODD), dict(dl=ctypes.c_void_p(4096 + 512)), dict(ref=None), dict(lo=-0.1), dict(lo=1.5),
                dict(lo=nan), dict(hi=-1.0), dict(hi=inf), dict(kl=-0.1), dict(kl=nan), dict(ds=inf)):
        assert policy(**bad) == 1, bad

    def pref(logits=D, targets=D, start=D, dl=D, lp=D, losses=D, N=4, P=2, V=100, Vp=128, kind=0, beta=0.1, sm=0.0,
             ds=1.0, ws=D, nb=1 << 20, err=D):
        return lib.gpt2op_preference_loss(logits, targets, start, None, dl, lp, None, losses, N, P, V, Vp, -1, kind, 0,
                                          F(beta), F(sm), F(ds), ws, nb, err, None)
    for bad in (dict(logits=None), dict(targets=None), dict(start=None), dict(lp=None), dict(losses=None),
                dict(ws=None), dict(err=None), dict(P=0), dict(N=0), dict(V=129), dict(Vp=130), dict(kind=2),
                dict(kind=-1), dict(beta=0.0), dict(beta=nan), dict(sm=1.0), dict(sm=-0.1), dict(kind=1, sm=0.1),
                dict(ds=nan), dict(nb=4 * 8 + 2 * 8 - 1), dict(ws=ctypes.c_void_p(4100)), dict(dl=ODD)):
        assert pref(**bad) == 1, bad
    assert lib.gpt2op_preference_loss_workspace(0, 1) == 0
    assert lib.gpt2op_token_logps(D, D, None, 4, 100, 128, -1, D, None) == 1
    assert lib.gpt2op_token_logps(D, D, D, 4, 100, 100, -1, D, None) == 1     # 100 columns: not a multiple of 8


def test_orthogonalize_refuses_bad_arguments(lib):
    ws = lib.gpt2op_orthogonalize_workspace
    assert ws(0, 4, 4) == 0 and ws(1, 0, 4) == 0 and ws(1, 4, 16385) == 0 and ws(65536, 4, 4) == 0
    n = ws(2, 8, 24)
    assert n > 0

    at = ctypes.c_void_p
    far = at(1 << 20)

    def ns(x=D, xs=192, out=far, os=192, b=2, r=8, c=24, steps=5, w=D, nb=n, err=D):
        return lib.gpt2op_orthogonalize(x, 1, xs, out, os, b, r, c, steps, w, nb, err, None)
    for bad in (dict(x=None), dict(out=None), dict(w=None), dict(err=None), dict(b=0), dict(r=0), dict(c=-1),
                dict(r=20000), dict(xs=191), dict(os=191), dict(steps=0), dict(steps=17), dict(nb=n - 1),
                dict(w=at(4096 + 128)),
                # results over the inputs (fp32, 768 bytes a matrix): the same place, inside, across the end,
                # from below, and between two matrices without room
                dict(out=D), dict(out=at(4096 + 700)), dict(out=at(4096 + 1500)), dict(out=at(4096 - 600)),
                dict(xs=256, os=512, out=at(4096 + 768))):
        assert ns(**bad) == 1, bad


def test_model_calls_refuse_bad_arguments(lib):
    assert lib.gpt2_token_logps(None, D, D, 1, -1, D) == 1
    assert lib.gpt2_fwd_bwd_policy(None, D, D, D, None, D, None, -1, F(.2), F(.2), F(0), F(1), None, None) == 1
    assert lib.gpt2_fwd_bwd_preference(None, D, D, None, -1, 0, 0, F(.1), F(0), None, None) == 1
    assert lib.gpt2_clip_muon(None, 0, F(0.95), D, 1 << 30, None) == 1
    assert gs.muon_workspace(gs.Config.make(**workloads.model_args("tiny"))) > 0
    assert gs.muon_workspace(gs.Config.make(n_layer=1, n_head=3, n_embd=144, seq_len=64, vocab_real=100)) == 0


def test_wrappers_refuse_tensors_the_kernels_do_not_take(lib):
    z = torch.zeros(4, 128, dtype=torch.bfloat16)
    t, f, e = torch.zeros(4, dtype=torch.int32), torch.zeros(4), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="device tensor"):
        gs.policy_loss(z, t, f, f, z, f, f, 100, e)
    with pytest.raises(ValueError, match="real ids"):
        gs.policy_loss(z, t, f, f, z, f, f, 129, e)
    with pytest.raises(ValueError, match="2P"):
        gs.preference_loss(z, t, torch.zeros(4, dtype=torch.int32), z, f, None, f, 100, torch.zeros(64, dtype=torch.uint8), e)
    with pytest.raises(ValueError, match="device tensor"):
        gs.token_logps(z, t, f, 100, e)
    x, o = torch.zeros(3, 8, 24), torch.zeros(3, 8, 24, dtype=torch.bfloat16)
    w = torch.zeros(1 << 20, dtype=torch.uint8)
    with pytest.raises(ValueError, match="device tensor"):
        gs.orthogonalize(x, o, w, e)
    with pytest.raises(ValueError, match="not contiguous"):
        gs.orthogonalize(x.transpose(1, 2), o.transpose(1, 2), w, e)
    with pytest.raises(ValueError, match="out:"):
        gs.orthogonalize(x, o[:2], w, e)
    with pytest.raises(ValueError, match="not float32 or bfloat16"):
        gs.orthogonalize(x.double(), o, w, e)
    with pytest.raises(ValueError, match="kind"):
        gs._kind("hinge")
