"""What the verification attention's dispatch and the step refuse, without a GPU."""
import pytest

torch = pytest.importorskip("torch")

from tree_speculative_decoding_bastion_gb300 import binding as bn  # noqa: E402


class Calls:
    """Stands in for the library: no call may reach it."""

    def __getattr__(self, name):
        raise AssertionError(f"{name} was called")


def caches():
    x = torch.zeros(1, 1, 8, 64)
    return {"kv": bn.KV(x, x), "kvq8": bn.KVQ8.empty(1, 1, 8, 64, device="cpu")}


@pytest.mark.parametrize("kind", ["kv", "kvq8"])
@pytest.mark.parametrize("given", ["prefix", "prefix_len"])
def test_a_prefix_and_its_length_come_together(monkeypatch, kind, given):
    """A length without its prefix would be ignored, a prefix without a length has none."""
    monkeypatch.setattr(bn, "_lib", Calls())
    kv = caches()[kind]
    x = torch.zeros(1, 1, 1, 64)
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(bn.BastionError, match="come together"):
        bn.verify_attn(x, x, x, kv, i, i, i, x, 1.0, **{given: kv if given == "prefix" else i})


@pytest.mark.parametrize("made,given", [("kv", "kvq8"), ("kvq8", "kv")])
def test_a_step_keeps_to_its_kind_of_cache(monkeypatch, made, given):
    """The 8-bit attention leaves anything in the step's attention workspace, and the other
    kind's wants it as its own calls leave it."""
    class Tensors:
        @staticmethod
        def bastion_tree_attn_workspace_size(*args):
            return 16

        bastion_tree_attn_q8_workspace_size = bastion_accept_workspace_size = bastion_tree_attn_workspace_size

    c = caches()
    monkeypatch.setattr(bn, "_lib", Tensors())
    step = bn.SpecTreeStep(1, 2, 16, 2, 1, 4, 1, 1, 64, c[made], device="cpu")
    monkeypatch.setattr(bn, "_lib", Calls())
    x = torch.zeros(1, 4, 1, 64)
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(bn.BastionError, match="caches was given"):
        step.verify(x, x, x, c[given], i, 1.0, x)
    with pytest.raises(bn.BastionError, match="must be a CUDA tensor"):   # the right kind goes on to the call's checks
        step.verify(x, x, x, c[made], i, 1.0, x)


def test_workspace_sizes_want_one_kind_of_cache(monkeypatch):
    monkeypatch.setattr(bn, "_lib", Calls())
    c = caches()
    for kv, prefix in ((c["kv"], c["kvq8"]), (c["kvq8"], c["kv"])):
        with pytest.raises(bn.BastionError, match="takes KV"):
            bn.verify_workspace_size(1, 4, 1, 1, 64, kv, prefix)
    with pytest.raises(bn.BastionError, match="takes KVQ8"):
        bn.bastion_tree_attn_q8_workspace_size(1, 4, 1, 1, 64, c["kv"])
