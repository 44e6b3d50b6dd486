"""The orthogonalisation's accuracy, held to the arithmetic it documents, on both of its kernels.

Bound. `emulated` does the documented roundings and nothing else: operands fp16 (X, A and
P, held times 2^10), fp32 sums, X as hi + lo fp16 in the term a X of all but the last two
rounds. Its distance from the 64-bit result, rounded to bf16, is the distance that these
roundings cost. Its sums run as coarsely as an adder of 16 products and an accumulator may:
all 17 aligned to the largest and cut below its 24 bits is up to 17 units of its last place
in 16 products, 2^4 and one more; they are cut to 20 bits after each 16. (At five rounds that
changes nothing; from eight on, with sums of a thousand terms and a steep spectrum, it is
what counts.) The kernels round the same values, and a sum that differs by some 2^-22 turns
a rounding to fp16 (2^-12) the other way for about one element in a thousand. Two such draws
of n m roundings each differ in norm by no more than a few hundredths from n = 100 on: 15%
is the bound.
"""
import numpy as np
import pytest

import gpt_step_b200 as gs
from oracle import posttrain as PT

from gpu_util import err_word, require_gpu, torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


SLACK = 1.15
SCALE = 1024.0
# the small singular values are where roundings grow
SPECTRA = {"flat": lambda k: torch.ones_like(k), "1/k": lambda k: 1 / k, "1/k^2": lambda k: 1 / k ** 2,
           "e^-k/20": lambda k: torch.exp(-k / 20)}


def matrix(r, c, spectrum, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    n = min(r, c)
    d = SPECTRA[spectrum](torch.arange(1, n + 1, device="cuda", dtype=torch.float64))
    u = torch.randn(r, n, device="cuda", generator=gen, dtype=torch.float64)
    return (u * d) @ torch.randn(n, c, device="cuda", generator=gen, dtype=torch.float64)


def defined(x, steps):
    """The definition in 64 bits."""
    a, b, c = PT.NS_COEFFS
    y = x.double()
    y = y.T if y.shape[0] > y.shape[1] else y
    y = y / (y.norm() + 1e-7)
    for _ in range(steps):
        g = y @ y.T
        y = a * y + (b * g + c * (g @ g)) @ y
    return y.T if x.shape[0] > x.shape[1] else y


def cut(x):
    """x towards zero to 20 bits."""
    f = x.float()
    bits = f.view(torch.int32)
    bits = torch.where(f.double().abs() > x.abs(), bits - 1, bits)
    return (bits & ~15).view(torch.float32).double()


def product(p, q):
    acc = torch.zeros(p.shape[0], q.shape[1], device=p.device, dtype=torch.float64)
    for k in range(0, p.shape[1], 16):
        acc = cut(acc + p[:, k:k + 16] @ q[k:k + 16])
    return acc


def emulated(x, steps):
    """The same with the documented roundings."""
    a, b, c = PT.NS_COEFFS
    half = lambda t: t.half().double()  # noqa: E731
    y = x.double()
    y = y.T if y.shape[0] > y.shape[1] else y
    y = y * (SCALE / (y.norm() + 1e-7))
    eye = torch.eye(y.shape[0], device=y.device, dtype=torch.float64)
    for i in range(steps):
        hi = half(y)
        lo = half(y - hi) if i < steps - 2 else torch.zeros_like(y)
        g = half(product(hi, hi.T) / SCALE)
        p = half(a * SCALE * eye + b * g + c * product(g, g) / SCALE)
        y = product(p, hi) / SCALE + a * lo
    y = y / SCALE
    return y.T if x.shape[0] > x.shape[1] else y


def off(y, ref):
    return float((y.double() - ref).norm() / ref.norm())


def run(x, steps=5, out=None):
    b, r, c = x.shape
    out = torch.empty(x.shape, dtype=torch.bfloat16, device="cuda") if out is None else out
    ws = torch.empty(gs.orthogonalize_workspace(b, r, c), dtype=torch.uint8, device="cuda").fill_(0xFF)
    err = err_word()
    gs.orthogonalize(x, out, ws, err, steps=steps)
    assert int(err.sum()) == 0
    return out


def check(got, x, steps):
    ref = defined(x, steps)
    most = off(emulated(x, steps).to(torch.bfloat16), ref)
    assert off(got, ref) <= SLACK * most, (off(got, ref), most)


# on chip alone, on chip in a cluster, tiles of 128 and of 256 columns (from a batch of one on), odd sizes, tall
SHAPES = [(1, 128, 128), (1, 120, 384), (2, 100, 900), (1, 900, 120), (3, 333, 517), (1, 150, 220), (2, 701, 300),
          (3, 2304, 768), (1, 1536, 1600), (40, 257, 300)]


@pytest.mark.parametrize("b,r,c", SHAPES)
@pytest.mark.parametrize("steps", [5, 8])
def test_accuracy_is_that_of_the_documented_roundings(b, r, c, steps):
    kinds = list(SPECTRA)
    for first in range(0, len(kinds), b):
        names = [kinds[(first + i) % len(kinds)] for i in range(b)]
        x = torch.stack([matrix(r, c, k, r + c + i) for i, k in enumerate(names)]).float()
        got = run(x, steps)
        for i in range(min(b, len(kinds))):
            check(got[i], x[i], steps)


@pytest.mark.parametrize("r,c", [(150, 220), (301, 700), (700, 301)])
@pytest.mark.parametrize("steps", [1, 2, 3, 4])
def test_accuracy_of_few_steps(r, c, steps):
    """Where the second half of X is carried through no, or one, round."""
    x = torch.stack([matrix(r, c, k, steps) for k in SPECTRA]).float()
    got = run(x, steps)
    for g, m in zip(got, x):
        check(g, m, steps)


# matrices that go through memory: tall and wide, rows that are no whole 16 bytes, tiles of both widths, few columns
LAYOUTS = [(2, 517, 333), (1, 701, 301), (2, 333, 517), (40, 300, 257), (40, 257, 300), (80, 131, 2050), (1, 2100, 130),
           (3, 2100, 24), (3, 24, 2100), (2, 2049, 9)]


def layouts(b, r, c, dt, gap_x, gap_o, off_x, off_o):
    """x and out inside larger buffers: matrices gap elements apart, the first off elements in."""
    n = r * c
    xb = torch.full((off_x + b * (n + gap_x),), 3.0, dtype=dt, device="cuda")
    ob = torch.full((off_o + b * (n + gap_o),), 4.0, dtype=torch.bfloat16, device="cuda")
    x = torch.as_strided(xb, (b, r, c), (n + gap_x, c, 1), off_x)
    o = torch.as_strided(ob, (b, r, c), (n + gap_o, c, 1), off_o)
    return x, o, ob


@pytest.mark.parametrize("b,r,c", LAYOUTS)
@pytest.mark.parametrize("fp32", [True, False])
@pytest.mark.parametrize("gap_x,gap_o,off_x,off_o", [(0, 0, 0, 0), (64, 8, 16, 8), (7, 5, 3, 1), (8, 3, 0, 0)])
def test_layouts_of_larger_matrices(b, r, c, fp32, gap_x, gap_o, off_x, off_o):
    """Against the definition, in any layout the same bits, and nothing written beside a result."""
    kinds = list(SPECTRA)
    some = [matrix(r, c, kinds[i % 4], r * c + i).float() for i in range(min(b, 4))]
    x, o, ob = layouts(b, r, c, torch.float32 if fp32 else torch.bfloat16, gap_x, gap_o, off_x, off_o)
    for i in range(b):
        x[i] = some[i % 4]
    given = x.clone()
    run(x, out=o)
    assert torch.equal(x, given)
    if min(r, c) >= 100:
        for i in range(min(b, 4)):
            check(o[i], x[i], 5)
    else:
        for i in range(min(b, 4)):
            # few singular values: the half steps may add up (2^-11 each, three in a round, grown to 36 in all)
            assert off(o[i], defined(x[i], 5)) <= 2.2e-2
    assert torch.equal(o, run(given.contiguous()))
    n = r * c
    ob[off_o:].view(b, n + gap_o)[:, :n] = 4.0
    assert bool((ob == 4.0).all())


@pytest.mark.parametrize("r,c", [(150, 220), (220, 150), (513, 300), (300, 520)])
@pytest.mark.parametrize("fp32", [True, False])
@pytest.mark.parametrize("many", [1, 8])
def test_zeros_and_non_finite_larger_matrices(r, c, fp32, many):
    """Each matrix by itself: zeros stay zeros, a NaN or an infinity makes its own matrix NaN, scale does not count."""
    base = matrix(r, c, "1/k", 7).float()
    x = torch.stack([base] * 7)
    x[1] = 0.0
    x[2, 3, 4] = float("nan")
    x[3, r - 1, c - 1] = float("inf")
    x[4] *= 2.0 ** 90
    x[5] *= 2.0 ** -20
    x = x.repeat(many, 1, 1)
    x = x if fp32 else x.to(torch.bfloat16)
    got = run(x).view(many, 7, r, c)
    assert bool((got[:, 1] == 0).all()) and bool(torch.isnan(got[:, 2]).all()) and bool(torch.isnan(got[:, 3]).all())
    for i in (0, 4, 6):
        check(got[0, i], x[i], 5)
    check(got[0, 5], x[5], 5)
    assert all(torch.equal(got[k, i], got[0, i]) for k in range(many) for i in (0, 4, 5, 6))
    assert torch.equal(got[0, 0], got[0, 6])
