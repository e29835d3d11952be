"""Attention over the 8-bit cache and behind a shared prefix at the ends of its
range: values and scales of every size, rows of very different sizes, long tails
of small weights; element by element against the 64-bit reference."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from tree_speculative_decoding_bastion_gb300 import binding as bn  # noqa: E402

from .context_cases import Case  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def built():
    from tree_speculative_decoding_bastion_gb300 import build
    build.build()
    bn.bastion_init(0)


@pytest.mark.parametrize("where", ["own", "prefix"])
@pytest.mark.parametrize("rows", [1, 8, 13, 40])
@pytest.mark.parametrize("gap,v_exp", [(90, 40), (24.5, 100), (8.5, 105), (7.5, 105)])
def test_a_late_key_of_a_large_value(where, rows, gap, v_exp):
    """bf16 caches: in every head a key `gap` binades above all others, late in some
    CTA's range, whose value is 2^v_exp.  The result is that value."""
    L, Hkv = 20000, 8
    own, pre = (L, 300) if where == "own" else (300, L)
    c = Case(60, [rows, 1], rows, Hkv, Hkv, 128, "bf16", False, 0, [own, 20], pre, 0, spread=0.0)
    cache = c.own if where == "own" else c.pre
    q = torch.nan_to_num(c.q.double())
    q[..., 1:] *= 2.0 ** -6                                  # the other scores: well below one binade
    q[..., 0] = gap * np.log(2.0) / (4.0 * c.scale)          # the key's: 4 q0 scale = gap binades
    c.q.copy_(q.to(torch.bfloat16))
    for one in (c.own, c.pre):
        one.t["k"][..., 0] = 0.0
    c.kt[..., 0] = 0.0
    for h in range(Hkv):
        key = 128 * (13 + 17 * h) + 100
        cache.t["k"][0, h, key] = 0.0
        cache.t["k"][0, h, key, 0] = 4.0
        cache.t["v"][0, h, key] = 2.0 ** v_exp
    for one in (c.own, c.pre):
        for b, n in enumerate(one.lens):
            one.k64[b], one.v64[b] = (one.t[x][b, :, :n].double() for x in "kv")
    for b, m in enumerate(c.n):                               # (rows behind the last node hold NaN again)
        c.q[b, m:] = float("nan")
    c.call()
    torch.cuda.synchronize()
    assert int(c.err) == 0
    c.check()
    assert float(c.out[0, 0].min()) > 2.0 ** (v_exp - 8)
