"""The arithmetic of the 8-bit cache's rows, and of the 8-bit parts that the attention over
it makes of its softmax weights, over every value they can have."""
import os
import re

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import context_oracle as co  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def cut(x):
    """An f16 cut off to e5m2: its upper byte."""
    return (x.view(torch.int16) & -256).view(torch.float16)


def test_three_e5m2_parts_hold_a_weight():
    """hi and mid cut off, lo rounded: within 2^-9 of the f16 or 2^-17 (half e5m2's smallest
    step), whichever is more, 2^-11 in the mean square and without a bias; the
    remainders are exact in f16."""
    h = torch.arange(0, 0x7801, dtype=torch.int32).to(torch.int16).view(torch.float16)     # 0 .. 2^15
    assert float(h[-1]) == 2.0 ** 15
    hi = cut(h)
    rest = h - hi
    mid = cut(rest)
    last = rest - mid
    assert torch.equal(rest.double(), h.double() - hi.double())
    assert torch.equal(last.double(), rest.double() - mid.double())
    for part in (hi, mid):
        assert torch.equal(part.to(torch.float8_e5m2).to(torch.float16), part)
    lo = last.to(torch.float8_e5m2)
    x = h.double()
    err = hi.double() + mid.double() + lo.double() - x
    assert bool((err.abs() <= torch.maximum(x * 2.0 ** -9, torch.full_like(x, 2.0 ** -17))).all())
    normal = x >= 2.0 ** -5
    rel = err[normal] / x[normal]
    assert float(rel.square().mean().sqrt()) <= 2.0 ** -11 and abs(float(rel.mean())) <= 2.0 ** -20


def stated_range():
    """The k of the header's "elements of at least 2^-k of the row's amax"."""
    text = " ".join(open(os.path.join(ROOT, "include", "bastion.h")).read().replace("*", " ").split())
    return int(re.search(r"at most 2\^-4, for elements of at least 2\^-(\d+) of the row's amax", text).group(1))


@pytest.mark.parametrize("amax", [224.0 * (1 + 2.0 ** -20), 225.0, 300.0, 447.0, 448.0])
def test_the_stated_relative_error_of_a_row(amax):
    """Every element from the stated share of the amax on is within 2^-4 of itself, at the amax
    that wastes most of the scale as well."""
    low = amax * 2.0 ** -stated_range()
    x = np.concatenate([[amax], np.geomspace(low, amax, 20001), [low]])[None]
    codes, byte = co.q8_quantise(x)
    assert int(byte[0]) == 127
    assert np.all(np.abs(co.q8_value(codes, byte) - x) <= x * 2.0 ** -4)
