"""Where the binding's calls take memory when they are given a stream, without a GPU: stand-ins for tensors, streams and
the library record it.  Everything made for a call belongs to the stream it runs on; what it returns is kept from
reuse for the caller's stream."""

import contextlib
import inspect

import pytest
import torch

from rotation_bit_quantization_amd import spin

GPU = torch.device("cuda", 0)


class Made(torch.Tensor):
    """A CPU tensor that says it lives on GPU 0."""
    is_cuda = property(lambda self: True)
    device = property(lambda self: GPU)

    def get_device(self):
        return 0

    def record_stream(self, stream):
        self.recorded = [*getattr(self, "recorded", []), stream]

    def new_empty(self, shape, dtype=None):
        return torch.empty(shape, dtype=dtype or self.dtype, device=GPU)


def gpu(t):
    return t.as_subclass(Made)


class Stream:
    device = GPU

    def __init__(self, handle, device=None):
        self.cuda_stream = handle


@pytest.fixture
def seen(monkeypatch):
    """What happens: "made" [(tensor, stream it was made on)], "launched" [stream handle]."""
    now = [Stream(1)]
    log = {"made": [], "launched": [], "here": now[0]}

    def make(empty):
        def f(shape, dtype=None, device=None):
            t = gpu(empty(tuple(shape) if not isinstance(shape, int) else shape, dtype=dtype))
            log["made"].append((t, now[-1]))
            return t
        return f

    @contextlib.contextmanager
    def use(s):
        now.append(s)
        yield
        now.pop()

    class Library:
        def __getattr__(self, name):
            def call(*args):
                log["launched"].append(args[-1])
                return spin.SPIN_OK
            return call

    monkeypatch.setattr(torch, "empty", make(torch.empty))
    monkeypatch.setattr(torch, "zeros", make(torch.zeros))
    monkeypatch.setattr(torch, "empty_like", lambda t: torch.empty(t.shape, dtype=t.dtype, device=GPU))
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    monkeypatch.setattr(torch.cuda, "stream", use)
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: now[-1])
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(spin, "_raw_stream", lambda d: now[-1].cuda_stream)
    monkeypatch.setattr(spin, "_cur_device", lambda: 0)
    monkeypatch.setattr(spin, "_workspaces", {})
    monkeypatch.setattr(spin, "load", Library)
    monkeypatch.setattr(spin, "_entry", lambda fn: getattr(Library(), fn))
    monkeypatch.setattr(spin, "spin_kv_attn_workspace", lambda *a: 4096)
    return log


def calls():
    """name -> (arguments of a call that makes its own outputs, arguments with those that the caller owns)"""
    z = lambda *shape, dtype=torch.float32: gpu(torch.zeros(shape, dtype=dtype))  # noqa: E731
    u8, i8, f16, i32 = torch.uint8, torch.int8, torch.float16, torch.int32
    cache = {"K_codes": z(2, 1, 16, 64, dtype=u8), "K_scale": z(2, 1, 16, dtype=f16), "V_codes": z(2, 1, 4, 16, 4, 4, dtype=u8),
             "V_scale": z(2, 1, 16, dtype=f16)}
    batch = dict(page_table=z(1, 1, dtype=i32), q_start=z(2, dtype=i32), kv_len=z(1, dtype=i32))
    gemm = dict(x_scale=z(32), w_scale=z(64))
    return {
        "spin_fold_rotation": dict(W=z(128, 64), R=None, r_block=1),
        "spin_fwht_quant": dict(X=z(4, 128), had_n=1, want_rot=True),
        "spin_fwht_quant8": dict(X=z(4, 128), had_n=1, want_rot=True),
        "spin_fwht_quant_f6": dict(X=z(32, 64), had_n=1),
        "spin_w4a4_gemm": dict(gemm, Xq=z(32, 32, dtype=u8), Wq=z(64, 32, dtype=u8), want_acc=True),
        "spin_w4a8_gemm": dict(gemm, Xq8=z(32, 64, dtype=i8), Wq=z(64, 32, dtype=u8), want_acc=True),
        "spin_w4a4_gemm_f6": dict(gemm, Xf6=z(1536, dtype=u8), x_sum=z(32, dtype=i32), Wq=z(64, 32, dtype=u8), want_acc=True),
        "spin_codes_f6": dict(Wq=z(96, 32, dtype=u8)),
        "spin_w4a4_gemm_f6f6": dict(Xf6=z(1536, dtype=u8), x_sum=z(32, dtype=i32), x_scale=z(32), Wf6=z(4608, dtype=u8),
                                    w_sum=z(96, dtype=i32), w_scale=z(96), K=64, want_acc=True),
        "spin_fwht_quant_gemm": dict(X=z(4, 12288, dtype=f16), Wq=z(64, 6144, dtype=u8), w_scale=z(64), want_acc=True),
        "spin_kv_quant": dict(X=z(2, 1, 128), rotate=1, want_rot=True),
        "spin_kv_quant8": dict(X=z(2, 1, 128), rotate=1, want_rot=True),
        "spin_kv_qkv": dict(K=z(2, 1, 128), V=z(2, 1, 128), Q=z(2, 2, 128), want_k_rot=True, out={"K_scale": z(2, 1, dtype=f16)}),
        "spin_rope_table": dict(inv_freq=z(4, dtype=torch.float64), n_pos=3),
        "spin_kv_append": dict(batch, Q=z(2, 2, 128), K=z(2, 1, 128), V=z(2, 1, 128), cache=cache),
        "spin_kv_attn": dict(batch, Q=z(2, 2, 128, dtype=f16), cache=cache),
        "spin_kv_attn_shared": dict(batch, Q=z(2, 2, 128, dtype=f16), cache=cache, prefix_table=z(1, dtype=i32), prefix_len=3),
    }


def tensors(x):
    if isinstance(x, dict):
        return tensors(tuple(x.values()))
    return [t for t in (x if isinstance(x, tuple) else (x,)) if isinstance(t, torch.Tensor)]


def test_every_call_is_here():
    named = [n for n, f in vars(spin).items() if n.startswith("spin_") and inspect.isfunction(f)
             and "stream" in inspect.signature(f).parameters]
    assert sorted(calls()) == sorted(n for n in named if n != "spin_fwht_quant_gemm_noalloc")      # makes nothing


@pytest.mark.parametrize("name", sorted(calls()))
@pytest.mark.parametrize("handle", [False, True])
def test_memory_belongs_to_the_stream_of_the_call(seen, name, handle):
    args, s = calls()[name], Stream(7)
    seen["made"].clear()
    res = tensors(getattr(spin, name)(**args, stream=7 if handle else s))
    assert seen["launched"] == [7]
    assert seen["made"] and all(on.cuda_stream == 7 for _, on in seen["made"])
    own = [t for t, _ in seen["made"]]
    returned = [t for t in res if any(t is m for m in own)]
    assert returned
    for t in returned:
        assert t.recorded == [seen["here"]]
    for t in tensors(tuple(args.values())) + tensors(args.get("out", {})) + tensors(args.get("cache", {})):
        assert not hasattr(t, "recorded")


@pytest.mark.parametrize("name", sorted(calls()))
def test_without_a_stream_the_current_one_is_taken(seen, name):
    args = calls()[name]
    seen["made"].clear()
    res = tensors(getattr(spin, name)(**args))
    assert seen["launched"] == [1] and all(on.cuda_stream == 1 for _, on in seen["made"])
    assert not any(hasattr(t, "recorded") for t in res)


def test_a_stream_of_another_gpu_is_refused(seen):
    s = Stream(7)
    s.device = torch.device("cuda", 1)
    for name, args in calls().items():
        with pytest.raises(ValueError):
            getattr(spin, name)(**args, stream=s)
    assert seen["launched"] == []
