"""The arithmetic of the 8-bit parts that the attention over the 8-bit cache makes
of its softmax weights, over every value they can have."""
import pytest

torch = pytest.importorskip("torch")


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
