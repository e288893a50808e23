"""sgd_verify at logits of any size: what matters is how they differ.

The definition in 64 bits and its tolerance are those of test_gpu_verify.py;
both references of an exponent (the maximum over the temperature rounded, or
the difference from the maximum) give (l - m) / t within 2^-22 of itself.
"""
import numpy as np
import pytest
import torch

from test_gpu_verify import DTYPES, SD, Case, _drafter, _refill  # noqa: F401 (SD: the fixture)

pytestmark = pytest.mark.gpu


def _rows(c, b):
    return slice(b * (c.k + 1), (b + 1) * (c.k + 1))


def _check(SD, c):
    """Drawn, and greedy; nothing is reported."""
    with _drafter(SD, c) as dr:
        c.check(c.run(dr, temperature=c.temp.float().cuda()))
        c.temp = torch.zeros(c.B)
        out, _ = c.check(c.run(dr))
        assert (out[:, 0] >= 0).all()
        assert dr.get_error() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", [1e6, 1e7, 1e9, 1e10, 1e12, 1e20, 1e29, 1e31])
def test_large_logits(SD, dtype, size):
    """A constant row, a forced token, a few that share everything, a row far
    below zero with one token less far, and ordinary rows that a bias has moved."""
    V = 2500
    c = _refill(Case(10, 3, V, seed=21))
    c.nv[:] = 3
    x = c.logits.double()
    x[_rows(c, 0)] = size
    x[_rows(c, 1)] = -size
    x[_rows(c, 2), 1234] = size                     # one token forced; the drafts are not it
    x[_rows(c, 3), 7] = size
    c.drafts[3] = 7                                 # forced and drafted
    x[_rows(c, 4), 100:110] = size                  # ten share everything
    c.drafts[4] = [103, 5, 103]
    x[_rows(c, 5)] -= size
    x[_rows(c, 6)] = -size
    x[_rows(c, 6), 2001] = -size / 2
    x[_rows(c, 7), ::2] = -size                     # a mask of that size
    x[_rows(c, 8)] += size
    x[_rows(c, 9), 1::3] = size
    c.logits = x.to(DTYPES[dtype])
    c.temp = torch.tensor([1.0, 1.0, 0.5, 1.0, 2.0, 0.9, 1.0, 0.7, 1.3, 100.0])
    _check(SD, c)


@pytest.mark.parametrize("temperature", [1e-5, 3e-5, 1e-3])
@pytest.mark.parametrize("dtype", ["f16", "f32"])
def test_low_temperatures(SD, dtype, temperature):
    c = _refill(Case(6, 3, 1500, seed=22))
    c.nv[:] = 3
    x = c.logits
    x[_rows(c, 0)] = 5e4
    x[_rows(c, 1)] = -5e4
    x[_rows(c, 2), 40:45] = 5e4
    c.drafts[2] = 42
    x[_rows(c, 3)] = x[_rows(c, 3)].round() * 64
    c.logits = x.to(DTYPES[dtype])
    c.temp = torch.full((6,), temperature, dtype=torch.float64)   # (as 32 bits, 1e-5 is the limit itself: not greedy)
    _check(SD, c)


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("power", range(15, 26))
def test_close_logits_about_a_large_value(SD, power, sign):
    """Logits a few units apart about 2^power / log2(e), where the reference of
    one thread's part may be of one kind and another's of the other."""
    V = 6000
    c = _refill(Case(6, 2, V, seed=power))
    c.nv[:] = 2
    at = float(np.float32(2.0 ** power / 1.4426950408889634))
    step = float(np.spacing(np.float32(at * 1.5)))
    x = torch.round(torch.randn(18, V, generator=c.g, dtype=torch.float64) * 1.5 / step) * step
    for b in range(6):
        for i in range(2):
            x[b * 3 + i, c.drafts[b, i]] = 8.0
    c.logits = (x + sign * at).float()
    c.temp = torch.tensor([1.0] * 5 + [0.75])
    _check(SD, c)
