"""Calls around the paged cache's steps on a given stream: what test_streams_cpu.py shows of the others."""

import torch
import pytest

from rotation_bit_quantization_amd import paged, spin

from .test_streams_cpu import Stream, gpu, seen, tensors  # noqa: F401


@pytest.fixture(autouse=True)
def a_workspace(monkeypatch):
    monkeypatch.setattr(paged, "spin_kv_weights_workspace", lambda *a: 4096)
    monkeypatch.setattr(paged, "spin_kv_choose_workspace", lambda *a: 4096)


def calls():
    z = lambda *shape, dtype=torch.float32: gpu(torch.zeros(shape, dtype=dtype))  # noqa: E731
    u8, f16, i32 = torch.uint8, torch.float16, torch.int32
    cache = {"K_codes": z(2, 1, 16, 64, dtype=u8), "K_scale": z(2, 1, 16, dtype=f16), "V_codes": z(2, 1, 4, 16, 4, 4, dtype=u8),
             "V_scale": z(2, 1, 16, dtype=f16)}
    batch = dict(page_table=z(1, 1, dtype=i32), q_start=z(2, dtype=i32), kv_len=z(1, dtype=i32))
    return {
        "spin_kv_tree": dict(parent=z(2, dtype=i32), q_start=z(2, dtype=i32), kv_len=z(1, dtype=i32), words=1),
        "spin_kv_attn_tree": dict(batch, Q=z(2, 2, 128, dtype=f16), cache=cache, tree=z(2, 1, dtype=i32), positions=z(2, dtype=i32)),
        "spin_kv_weights": dict(batch, Q=z(2, 2, 128, dtype=f16), lse=z(2, 2), cache=cache),
        "spin_kv_choose": dict(W=z(2, 1, 16), page_table=z(1, 1, dtype=i32), kv_len=z(1, dtype=i32), keep=3),
        "spin_kv_move": dict(cache=cache, page_table=z(1, 1, dtype=i32), kept=z(1, 1, 2, dtype=i32)),
        "spin_kv_append": dict(batch, Q=z(2, 2, 128), K=z(2, 1, 128), V=z(2, 1, 128), cache=cache, positions=z(2, dtype=i32)),
        "spin_kv_attn": dict(batch, Q=z(2, 2, 128, dtype=f16), cache=cache, lse=z(2, 2)),
        "spin_kv_attn_shared": dict(batch, Q=z(2, 2, 128, dtype=f16), cache=cache, prefix_table=z(1, dtype=i32), prefix_len=3, lse=z(2, 2)),
    }


def test_every_call_is_here():
    assert spin._PAGED <= {*calls(), "spin_kv_weights_workspace", "spin_kv_choose_workspace"} and spin._PAGED <= set(spin.__all__) and spin._PAGED <= set(dir(spin))
    with pytest.raises(AttributeError):
        spin.spin_kv_forest


@pytest.mark.parametrize("name", sorted(calls()))
@pytest.mark.parametrize("handle", [False, True])
def test_memory_belongs_to_the_stream_of_the_call(seen, name, handle):  # noqa: F811
    args = calls()[name]
    seen["made"].clear()
    res = tensors(getattr(spin, name)(**args, stream=7 if handle else Stream(7)))
    assert seen["launched"] == [7]
    assert all(on.cuda_stream == 7 for _, on in seen["made"])
    own = [t for t, _ in seen["made"]]
    returned = [t for t in res if any(t is m for m in own)]
    assert returned or name == "spin_kv_move"
    for t in returned:
        assert t.recorded == [seen["here"]]
    for t in tensors(tuple(args.values())) + tensors(args.get("cache", {})):
        assert not hasattr(t, "recorded")


@pytest.mark.parametrize("name", sorted(calls()))
def test_without_a_stream_the_current_one_is_taken(seen, name):  # noqa: F811
    seen["made"].clear()
    res = tensors(getattr(spin, name)(**calls()[name]))
    assert seen["launched"] == [1] and all(on.cuda_stream == 1 for _, on in seen["made"])
    assert not any(hasattr(t, "recorded") for t in res)


def test_a_stream_of_another_gpu_is_refused(seen):  # noqa: F811
    s = Stream(7)
    s.device = torch.device("cuda", 1)
    for name, args in calls().items():
        with pytest.raises(ValueError):
            getattr(spin, name)(**args, stream=s)
    assert seen["launched"] == []
