"""Long prompts into the 8-bit cache: stretches of several passes a CTA, block tables of
many pages and any alignment, and a time that grows with the prompt."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from tree_speculative_decoding_bastion_gb300 import binding as bn  # noqa: E402

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def built():
    from tree_speculative_decoding_bastion_gb300 import build
    build.build()
    bn.bastion_init(0)


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def paged(B, Hkv, d, page, tokens, shift=0):
    """A zeroed paged cache of B requests of `tokens` positions; the block table begins `shift`
    words behind an aligned address."""
    per = -(-tokens // page)
    gen = torch.Generator(device="cuda").manual_seed(1)
    ids = torch.randperm(B * per, generator=gen, device="cuda").to(torch.int32)
    room = torch.zeros(B * per + 4, dtype=torch.int32, device="cuda")
    table = room[shift:shift + B * per].view(B, per)
    table.copy_(ids.view(B, per))
    return bn.KVQ8.empty(B * per, Hkv, page, d, block_table=table)


def parts(kv):
    return [t.view(torch.uint8) for t in (kv.k, kv.v, kv.k_scale, kv.v_scale)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,Hkv,d,page,ctx,new,shift", [
    (1, 20011, 8, 128, 1, [3], [20011], 0), (1, 20011, 8, 128, 1, [2], [20008], 1),
    (3, 9000, 8, 128, 1, [0, 5, 1], [9000, 0, 8997], 3), (1, 70001, 4, 128, 8, [9], [70001], 2)])
def test_a_long_append_is_many_short_ones(B, T, Hkv, d, page, ctx, new, shift, dtype):
    gen = torch.Generator(device="cuda").manual_seed(2)
    k, v = (torch.randn(B, T, Hkv, d, generator=gen, device="cuda").to(DT[dtype]) for _ in range(2))
    one, many = (paged(B, Hkv, d, page, max(ctx) + T, shift) for _ in range(2))
    c, err = i32(ctx), torch.zeros(1, dtype=torch.int32, device="cuda")
    bn.bastion_kv_append_q8(k, v, one, i32(new), c, c, dev_err=err)
    assert int(err) == 0 and c.tolist() == [a + n for a, n in zip(ctx, new)]
    c = i32(ctx)
    for t in range(0, T, 500):
        n = min(500, T - t)
        bn.bastion_kv_append_q8(k[:, t:t + n].contiguous(), v[:, t:t + n].contiguous(), many,
                                i32([min(max(x - t, 0), n) for x in new]), c, c, dev_err=err)
    assert int(err) == 0 and c.tolist() == [a + n for a, n in zip(ctx, new)]
    for a, b in zip(parts(one), parts(many)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("shift", [0, 1, 2, 3])
@pytest.mark.parametrize("where", [0, 1, 5, 6000, 19998, 19999])
@pytest.mark.parametrize("page_id", [-1, 1 << 30])
def test_a_bad_page_anywhere_writes_nothing(where, shift, page_id):
    T, Hkv, d = 20000, 8, 128
    kv = paged(1, Hkv, d, 1, T + 2, shift)
    kv.block_table[0, 1 + where] = page_id
    x = torch.ones(1, T, Hkv, d, dtype=torch.bfloat16, device="cuda")
    c, err = i32([1]), torch.zeros(1, dtype=torch.int32, device="cuda")
    bn.bastion_kv_append_q8(x, x, kv, i32([T]), c, c, dev_err=err)
    assert int(err) == bn.DEVERR_PAGE and c.tolist() == [1]
    assert all(int(t.max()) == 0 for t in parts(kv))
    kv.block_table[0, 1 + where] = 0                          # pages before and behind the new tokens do not matter
    kv.block_table[0, 0] = kv.block_table[0, T + 1] = page_id
    err.zero_()
    bn.bastion_kv_append_q8(x, x, kv, i32([T]), c, c, dev_err=err)
    assert int(err) == 0 and c.tolist() == [T + 1]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_small_pages_cost_a_part_of_the_prompt_not_its_square(dtype):
    """131072 tokens in pages of 8 within 1.5 times the same without pages (when every CTA
    checked every page for a few tokens of its own: 1.9)."""
    T, Hkv, d = 131072, 8, 128
    x = torch.randn(1, T, Hkv, d, device="cuda").to(DT[dtype])
    n, zero, out = i32([T]), i32([0]), i32([0])

    def fastest(kv):
        run = bn.prepare_call(bn.bastion_kv_append_q8, x, x, kv, n, zero, out)
        times = []
        for _ in range(12):
            e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            e0.record()
            run()
            e1.record()
            torch.cuda.synchronize()
            times.append(e0.elapsed_time(e1))
        return min(times[2:])

    assert fastest(paged(1, Hkv, d, 8, T)) <= 1.5 * fastest(bn.KVQ8.empty(1, Hkv, T, d))
