"""Numbers that a C int does not hold are refused by the binding, which would otherwise pass on their low 32 bits; without a
GPU, with the stand-ins of test_streams_cpu.py."""

import os

import pytest
import torch

from rotation_bit_quantization_amd import spin

from .test_streams_cpu import calls, seen  # noqa: F401

BIG = [2 ** 32, 2 ** 32 + 16, 2 ** 31, -2 ** 32 + 4]


class Shaped:
    """What the binding asks of a tensor, of any shape."""
    is_cuda, device = True, torch.device("cuda", 0)

    def __init__(self, shape, dtype=torch.int32):
        self.shape, self.dtype = torch.Size(shape), dtype

    def dim(self):
        return len(self.shape)

    def get_device(self):
        return 0

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 4096


@pytest.mark.parametrize("x", BIG)
@pytest.mark.parametrize("at", range(7))
def test_workspace(x, at):
    if not os.path.exists(spin.library_path()):
        pytest.skip("libspin.so not built (python -m rotation_bit_quantization_amd.build)")
    args = [1, 8, 1, 1, 300, 16, 0]
    assert spin.spin_kv_attn_workspace(*args) > 0
    args[at] = x
    with pytest.raises((ValueError, spin.SpinError)) as e:
        spin.spin_kv_attn_workspace(*args)
    assert e.type is ValueError


@pytest.mark.parametrize("x", BIG)
@pytest.mark.parametrize("name,which", [
    ("spin_fold_rotation", "r_block"), ("spin_fwht_quant", "had_n"), ("spin_fwht_quant8", "had_n"), ("spin_fwht_quant_f6", "had_n"),
    ("spin_w4a4_gemm", "kernel"), ("spin_kv_quant", "rotate"), ("spin_kv_quant8", "rotate"), ("spin_rope_table", "n_pos"),
    ("spin_rope_table", "pos0"), ("spin_kv_append", "pos0"), ("spin_kv_append", "interleaved"), ("spin_kv_attn", "window"),
    ("spin_kv_attn", "causal"), ("spin_kv_attn_shared", "window"), ("spin_kv_attn_shared", "causal")])
def test_arguments(seen, name, which, x):  # noqa: F811
    args = dict(calls()[name], **{which: x})
    if which == "n_pos":
        args["table"] = Shaped((max(x, 0), 8), torch.float32)
    with pytest.raises(ValueError, match="32 bits"):
        getattr(spin, name)(**args)
    assert seen["launched"] == []


@pytest.mark.parametrize("x", BIG[:3])
def test_a_prefix(seen, x):  # noqa: F811
    """Behind a table that has the pages."""
    args = calls()["spin_kv_attn_shared"]
    page, cache = 1024, {"K_codes": (2, 1, 1024, 64), "K_scale": (2, 1, 1024), "V_codes": (2, 1, 256, 16, 4, 4), "V_scale": (2, 1, 1024)}
    args["cache"] = {k: Shaped(v, torch.uint8 if "codes" in k else torch.float16) for k, v in cache.items()}
    args.update(prefix_len=x, prefix_table=Shaped((-(-x // page),)))
    with pytest.raises(ValueError, match="32 bits"):
        spin.spin_kv_attn_shared(**args)
    assert seen["launched"] == []


@pytest.mark.parametrize("name", ["spin_kv_append", "spin_kv_attn", "spin_kv_attn_shared"])
@pytest.mark.parametrize("B,max_pages", [(1, 2 ** 32 + 1), (2 ** 32 + 1, 1), (2 ** 31, 2)])
def test_batches(seen, name, B, max_pages):  # noqa: F811
    args = dict(calls()[name], page_table=Shaped((B, max_pages)), q_start=Shaped((B + 1,)), kv_len=Shaped((B,)))
    with pytest.raises(ValueError, match="32 bits"):
        getattr(spin, name)(**args)
    assert seen["launched"] == []


@pytest.mark.parametrize("shape", [(2 ** 32 + 8, 16), (8, 2 ** 32 + 16)])
def test_tables_of_positions(seen, shape):  # noqa: F811
    with pytest.raises(ValueError, match="32 bits"):
        spin.spin_kv_append(**dict(calls()["spin_kv_append"], rope=Shaped(shape, torch.float32)))
    assert seen["launched"] == []


def test_the_names_that_the_binding_offers():
    assert [n for n in spin.__all__ if not hasattr(spin, n)] == [] and len(set(spin.__all__)) == len(spin.__all__)
