"""Attention over the 8-bit cache and behind a shared prefix at the ends of its
range: values and scales of every size, rows of very different sizes, long tails
of small weights; element by element against the 64-bit reference."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from tree_speculative_decoding_bastion_gb300 import binding as bn  # noqa: E402

from .context_cases import Case, scale_exponents  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def built():
    from tree_speculative_decoding_bastion_gb300 import build
    build.build()
    bn.bastion_init(0)


@pytest.mark.parametrize("where", ["own", "prefix"])
@pytest.mark.parametrize("rows", [1, 20, 70])
@pytest.mark.parametrize("gap,v_exp", [(90, 40), (24.5, 100), (8.5, 105)])
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


def tight(c, contexts=None):
    """(want, bound) of a Case over an 8-bit cache with bf16 inputs.  Besides the output's
    half step and the scores' error (context_cases): a weight that meets codes is an f16
    (2^-11 relative) in three e5m2 parts (2^-9 of it, or 2^-24 of its row's largest
    weight, both times the keys' V scales; test_context_parts_cpu), 1.25 2^-9 together;
    one that meets a tree's value is a bf16 (2^-8)."""
    want = torch.full(c.q.shape, float("nan"), dtype=torch.float64, device="cuda")
    bound = torch.zeros_like(want)
    g, d = c.Hq // c.Hkv, c.d
    for b, parts in enumerate(contexts or c.contexts()):
        m = c.n[b]
        ctx = sum(k.shape[1] for k, _ in parts)
        see = torch.ones(m, ctx + m, dtype=torch.bool)
        for i in range(m):
            for j in range(m):
                see[i, ctx + j] = bool((int(c.words[b, i, j // 64]) >> (j % 64)) & 1)
        see = see.cuda()
        for h in range(c.Hkv):
            keys = torch.cat([k[h] for k, _ in parts] + [c.kt[b, :m, h].double()])
            vals = torch.cat([v[h] for _, v in parts] + [c.vt[b, :m, h].double()])
            x = c.q[b, :m, h * g:(h + 1) * g].double()
            z = (torch.einsum("igd,jd->igj", x, keys) * c.scale).masked_fill(~see[:, None], float("-inf"))
            wt = torch.softmax(z, -1)
            ev = scale_exponents(vals)
            ev[ctx:] = ev[ctx:].max()
            peak = (wt * 2.0 ** (ev + 1)).amax(-1, keepdim=True)   # (a row's scale may be one more than its values need)
            step = peak * 1.01 * 2.0 ** -24 / 2.0 ** ev
            werr = torch.maximum(wt * 2.0 ** -8, torch.minimum(wt, step))
            werr[..., :ctx] = torch.maximum(wt * 1.25 * 2.0 ** -9, step)[..., :ctx]
            amax = x.abs().amax(-1, keepdim=True)
            dz = x.norm(dim=-1)[..., None] * keys.norm(dim=-1) * c.scale * ((d + 4) * 2.0 ** -24)
            # elements of q below 2^-6.8 of their row's largest are off by up to 2^-14 of it
            small = (x.abs() < amax * 2.0 ** -6.8).double()
            dz = dz + torch.einsum("igd,jd->igj", small, keys.abs()) * amax * 2.0 ** -14 * c.scale
            # an error dz of the scores moves a weight and the sum that divides it
            move = 2.0 * dz.amax(-1, keepdim=True) + 2.0 ** -18
            o = torch.einsum("igj,jd->igd", wt, vals)
            want[b, :m, h * g:(h + 1) * g] = o
            bound[b, :m, h * g:(h + 1) * g] = (torch.einsum("igj,jd->igd", werr + wt * move, vals.abs())
                                               + o.abs() * (2.0 ** -8 * 1.01 + move))
    return want, bound


def check_tight(c, contexts=None, floor=0.0):
    want, bound = tight(c, contexts)
    idle = torch.isnan(want)
    got = c.out.double()
    assert bool((got[idle] == 5.0).all()), "rows behind the last node were written"
    off = (got - want).abs() - bound - floor
    bad = ~idle & ~(off <= 0)
    if bool(bad.any()):
        i = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{int(bad.sum())} of {int((~idle).sum())} elements off, first {i}: got {float(got[i])}, "
                             f"want {float(want[i])}, bound {float(bound[i])}")


def flat_context(c, scores, values):
    """Request 0's own 8-bit context: key j scores scores[j] (nats, in every row and KV head;
    held by the first element), all its values are values[j]; tree nodes score and hold 0."""
    L, t = c.own.lens[0], c.own.t
    t["k"][0, :, :L] = 0
    t["ks"][0, :, :L] = 127
    t["vs"][0, :, :L] = 127
    c.q[0] = 0.0
    c.q[0, ..., 0] = 1.0 / 16.0 / c.scale                    # a code of 16 x scores a nat
    code = lambda x: torch.as_tensor(x, dtype=torch.float32).to(torch.float8_e4m3fn).view(torch.uint8).cuda()  # noqa: E731
    t["k"][0, :, :L, 0] = code(scores * 16.0)
    t["v"][0, :, :L] = code(values)[:, None]
    for x, name in ((c.own.k64, "k"), (c.own.v64, "v")):
        x[0] = t[name][0, :, :L].view(torch.float8_e4m3fn).double()
    c.kt[:] = 0.0
    c.vt[:] = 0.0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows", [2, 15, 25, 40])
@pytest.mark.parametrize("gap", [8, 10])
def test_a_flat_tail_behind_a_sink(gap, rows, d):
    """Equal keys of e^-gap of the sink's weight each, most of them in the same CTA's range:
    their rounding has one sign and adds up."""
    L, Hkv = 6000, 96
    c = Case(61, [rows], rows, 2 * Hkv, Hkv, d, "bf16", True, 0, [L], None, spread=0.0)
    scores, values = np.zeros(L), np.ones(L)
    scores[::1000], values[::1000] = gap, -1.0               # (of the head's ranges each has one)
    flat_context(c, scores, values)
    c.call()
    torch.cuda.synchronize()
    check_tight(c)


@pytest.mark.parametrize("rows", [2, 25, 40])
def test_tails_of_every_size_behind_a_sink(rows):
    """Scores spread over 12 nats below the sink, values that cancel in the mean."""
    L, Hkv = 8000, 64
    c = Case(62, [rows], rows, 2 * Hkv, Hkv, 128, "bf16", True, 0, [L], None, spread=0.0)
    r = np.random.default_rng(62)
    scores, values = r.uniform(0, 8, L), np.where(r.random(L) < 0.5, 1.0, -0.9375)
    scores[::2000], values[::2000] = 12.0, 0.5
    flat_context(c, scores, values)
    c.call()
    torch.cuda.synchronize()
    check_tight(c)


@pytest.mark.parametrize("form", ["q8", "q8_prefix"])
@pytest.mark.parametrize("spread", [0.0, 1.0, 2.0])
@pytest.mark.parametrize("rows,Hq,Hkv,d,page", [(1, 8, 2, 128, 16), (5, 8, 2, 64, 0), (13, 8, 2, 128, 0), (30, 8, 2, 64, 8),
                                                (64, 8, 2, 128, 16)])
def test_weights_keep_more_bits_than_the_output(rows, Hq, Hkv, d, page, spread, form):
    c = Case(63, [rows, max(1, rows - 3)], rows, Hq, Hkv, d, "bf16", True, page, [1500, 333],
             None if form == "q8" else 700, page, spread=spread, room=3)
    c.call()
    torch.cuda.synchronize()
    assert int(c.err) == 0
    check_tight(c)


def rescale(c, cache, e):
    """V rows of a Case's 8-bit cache: exponents e (int64 [B, Hkv, L], -127 .. 127) for the scales
    that they have; a row of exponent -127 becomes zero."""
    e = torch.as_tensor(e).cuda()
    zero = e == -127
    L = e.shape[2]
    cache.t["vs"][:, :, :L] = (e + 127).to(torch.uint8)
    cache.t["v"][:, :, :L] = torch.where(zero[..., None], torch.zeros_like(cache.t["v"][:, :, :L]), cache.t["v"][:, :, :L])
    for b, n in enumerate(cache.lens):
        rows = cache.t["v"][b, :, :n].view(torch.float8_e4m3fn).double() * torch.exp2(e[b, :, :n].double())[..., None]
        cache.v64[b] = rows


def largest(c):
    return max(float(v.abs().max()) for parts in c.contexts() for _, v in parts if v.numel())


@pytest.mark.parametrize("rows", [1, 12, 40])
@pytest.mark.parametrize("e", [-90, 40, 64, 67, 90, 110])
def test_zero_values_before_large_ones(e, rows):
    """The first 32 (and the first 140) keys of every 512 hold zeros under the smallest scale."""
    c = Case(64, [rows], rows, 8, 2, 128, "bf16", True, 0, [3000], None)
    at = torch.arange(3000)
    ev = torch.full((1, 2, 3000), e, dtype=torch.int64)
    ev[0, 0, at % 512 < 32] = -127
    ev[0, 1, at % 512 < 140] = -127
    rescale(c, c.own, ev)
    c.vt[:] = 0.0
    c.call()
    torch.cuda.synchronize()
    check_tight(c)


@pytest.mark.parametrize("rows", [1, 12, 40])
@pytest.mark.parametrize("lo,hi", [(-60, 60), (-126, 110), (0, 100), (-120, -20)])
def test_value_scales_that_differ_within_a_context(lo, hi, rows):
    c = Case(65, [rows, 1], rows, 8, 2, 128, "bf16", True, 0, [1900, 300], 700, 0, spread=0.5)
    r = np.random.default_rng(65)
    for cache in (c.own, c.pre):
        rescale(c, cache, r.integers(lo, hi + 1, (len(cache.lens), 2, max(cache.lens))))
    c.call()
    torch.cuda.synchronize()
    check_tight(c, floor=largest(c) * 2.0 ** -70)


@pytest.mark.parametrize("rows", [1, 12, 40])
@pytest.mark.parametrize("v_exp,tree_exp", [(-90, -90), (-90, 0), (90, 90), (0, -90), (0, 90), (90, -60), (-50, 60)])
def test_values_of_contexts_and_trees_of_every_size(v_exp, tree_exp, rows):
    c = Case(66, [rows, 2], max(rows, 2), 8, 2, 64, "bf16", True, 16, [1900, 0], 300, 16, v_exp=v_exp)
    c.vt *= 2.0 ** tree_exp
    c.call()
    torch.cuda.synchronize()
    check_tight(c, floor=max(largest(c), float(torch.nan_to_num(c.vt.double()).abs().max())) * 2.0 ** -70)


@pytest.mark.parametrize("ctx", [100, 3000])
def test_a_dominating_key_of_a_tiny_value(ctx):
    """A key far above the others whose value is 2^140 times smaller than theirs: the row is
    that value, off by no more than may be left out."""
    c = Case(67, [2], 2, 4, 2, 128, "bf16", True, 0, [ctx], None)
    e = torch.randint(5, 20, (1, 2, ctx), generator=torch.Generator().manual_seed(67))
    e[:, :, 50] = -120
    rescale(c, c.own, e)
    t = c.own.t
    t["k"][0, :, 50] = 0
    t["k"][0, :, 50, 0] = 0x7E                               # 448
    t["ks"][0, :, 50] = 127
    c.own.k64[0][:, 50] = 0.0
    c.own.k64[0][:, 50, 0] = 448.0
    c.q[..., 0] = 4.0                                        # its score: 158 nats
    c.call()
    torch.cuda.synchronize()
    check_tight(c, floor=largest(c) * 2.0 ** -70)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("which", ["vs", "ks"])
@pytest.mark.parametrize("rows", [1, 12, 40])
@pytest.mark.parametrize("weight", [1.0, 0.0])
def test_a_scale_byte_of_255_is_nan(weight, rows, which, dtype):
    """A context key whose K or V scale is the format's NaN makes the rows of its KV head
    NaN, whatever its codes and its weight; the other heads stay as they were."""
    c = Case(68, [rows, 1], rows, 8, 2, 128, dtype, True, 16, [700, 40], 300, 16)
    c.call()
    torch.cuda.synchronize()
    clean = c.out.clone()
    at, slot = int(c.own.table[0, 600 // 16]), 600 % 16
    c.own.t[which][at, 1, slot] = 255
    c.own.t["v"][at, 1, slot] = 0
    if weight == 0.0:                                         # a score some 10^5 below the others'
        c.own.t["k"][at, 1, slot] = torch.where(c.q[0, 0, 4].float() > 0, 0xFE, 0x7E).to(torch.uint8)
        if which == "vs":
            c.own.t["ks"][at, 1, slot] = 127 + 8
    c.call()
    torch.cuda.synchronize()
    assert int(c.err) == 0
    assert torch.isnan(c.out[0, :rows, 4:]).all()
    assert torch.equal(c.out[0, :rows, :4], clean[0, :rows, :4]) and torch.equal(c.out[1, :1], clean[1, :1])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N,g", [(4, 4), (8, 4), (16, 4), (32, 4), (50, 4)])
@pytest.mark.parametrize("ctx", [37, 1500])
@pytest.mark.parametrize("lo,hi", [(-5, 3), (-20, 3), (-2, 0)])
def test_rows_of_q_of_different_sizes(lo, hi, ctx, N, g, d):
    """Sizes of 2^lo to 2^hi among the rows of one tile, and a row of zeros: rows whose 8-bit
    parts have scales of their own (and, for the last range, a common one)."""
    c = Case(69, [N, max(1, N - 3)], N, 2 * g, 2, d, "bf16", True, 16, [ctx, 20], None)
    r = torch.Generator().manual_seed(69)
    size = torch.exp2(torch.randint(lo, hi + 1, (2, N, 2 * g, 1), generator=r).float()).cuda()
    c.q.copy_((c.q.float() * size).to(torch.bfloat16))
    c.q[0, N // 2, 1] = 0.0
    c.call()
    torch.cuda.synchronize()
    check_tight(c)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("spread", [0.0, 2.0])
@pytest.mark.parametrize("rows", [1, 13, 40])
def test_equal_values_come_out_as_they_are(rows, spread, d):
    """bf16 caches: where every key holds the same value the result is that value, bit for bit:
    the weights are divided by the sum of what they were rounded to, and what is left,
    fp32 sums, is far below half a step of the output."""
    c = Case(70, [rows, 1], rows, 8, 2, d, "bf16", False, 16, [900, 3], 700, 16, spread=spread)
    value = torch.randn(2, d, generator=torch.Generator().manual_seed(70)).to(torch.bfloat16).cuda()
    for cache in (c.own, c.pre):
        cache.t["v"].copy_(torch.where(torch.isnan(cache.t["v"]), cache.t["v"], value[None, :, None].expand_as(cache.t["v"])))
    for b, m in enumerate(c.n):
        c.vt[b, :m] = value
    c.call()
    torch.cuda.synchronize()
    assert int(c.err) == 0
    for b, m in enumerate(c.n):
        assert torch.equal(c.out[b, :m], value.repeat_interleave(4, 0)[None].expand(m, -1, -1))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("page", [0, 8, 64])
@pytest.mark.parametrize("shift", [1, 4])
def test_scales_at_any_address(shift, page, dtype):
    """Scale bytes need no alignment: the same bits from a copy that begins `shift` bytes on,
    lengths of every remainder by eight among the requests."""
    ctx = [1000 + i for i in range(9)]
    c = Case(71, [2] * 9, 2, 4, 2, 64, dtype, True, page, ctx, 301, page, room=7, v_exp=20)
    c.call()
    torch.cuda.synchronize()
    assert int(c.err) == 0
    c.check()
    want = c.out.clone()
    for cache in (c.own, c.pre):
        moved = []
        for name in ("ks", "vs"):
            t = cache.t[name]
            room = torch.full((t.numel() + 16,), 254, dtype=torch.uint8, device="cuda")
            view = room[shift:shift + t.numel()].view(t.shape)
            view.copy_(t)
            moved.append(view.view(torch.float8_e8m0fnu))
        cache.kv = bn.KVQ8(cache.kv.k, cache.kv.v, *moved, cache.kv.block_table)
    c.out.fill_(5.0)
    c.call()
    torch.cuda.synchronize()
    assert int(c.err) == 0
    assert torch.equal(c.out, want)
