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
