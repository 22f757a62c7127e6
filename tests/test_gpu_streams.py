"""Calls on a stream that is not the current one: their memory is not what the current stream still works on, results are
those of the current stream, eager and captured."""

import numpy as np
import pytest
import torch

from rotation_bit_quantization_amd import spin

from .paged_case import DEV, dev, host, pool, starts, tables

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spin.load()


def decode(kv=5000):
    """Arguments of an attention call in shares, which takes a workspace."""
    rng = np.random.default_rng(1)
    n = -(-kv // 64) + 1
    q = dev(rng.standard_normal((2, 16, 128)).astype(np.float16))
    args = (q, dev(pool(rng, n, 2, 64, 4)), dev(tables(rng, [kv - 64, 1], 64, n, extra=1)), dev(starts([1, 1])),
            dev(np.array([kv - 64, 1], np.int32)))
    assert spin.spin_kv_attn_workspace(2, 16, 2, 2, args[2].shape[1], 64) > 0
    return args


def test_memory_that_the_current_stream_let_go_is_not_taken():
    x = torch.randn((512, 4096), device=DEV)
    s = torch.cuda.Stream()
    mine = spin.spin_fwht_quant(x, 128, want_rot=True)
    at = [t.data_ptr() for t in mine]
    want = [host(t) for t in mine]
    del mine
    torch.cuda.synchronize()
    s.wait_stream(torch.cuda.current_stream())
    other = spin.spin_fwht_quant(x, 128, want_rot=True, stream=s)
    again = spin.spin_fwht_quant(x, 128, want_rot=True)
    s.synchronize()
    assert not {t.data_ptr() for t in other} & set(at)
    assert [t.data_ptr() for t in again] == at
    for t in (other, again):
        assert all(np.array_equal(host(a), b) for a, b in zip(t, want))


def test_attention_on_two_streams_at_once():
    """The current stream is behind with long products and with calls whose workspaces it has let go."""
    args = decode()
    want = host(spin.spin_kv_attn(*args)).copy()
    a = torch.randn((4096, 4096), device=DEV, dtype=torch.float16)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    here, there = [], []
    for handle in (s, s.cuda_stream):
        for _ in range(20):
            a @ a
            here.append(spin.spin_kv_attn(*args))
            there.append(spin.spin_kv_attn(*args, stream=handle))
    torch.cuda.synchronize()
    assert all(np.array_equal(host(o), want) for o in here + there)


def test_a_captured_call_on_a_second_stream():
    args = decode()
    want = host(spin.spin_kv_attn(*args)).copy()
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        s.wait_stream(torch.cuda.current_stream())
        there = spin.spin_kv_attn(*args, stream=s)
        here = spin.spin_kv_attn(*args)
        torch.cuda.current_stream().wait_stream(s)
    for _ in range(3):
        here.fill_(5.0)
        there.fill_(5.0)
        g.replay()
        assert np.array_equal(host(here), want) and np.array_equal(host(there), want)
        assert np.array_equal(host(spin.spin_kv_attn(*args)), want)


def test_a_layer_on_a_second_stream():
    """qkv_proj's product to o_proj's codes, every call on the same second stream."""
    rng = np.random.default_rng(2)
    T, Hq, Hkv = 70, 8, 2
    x = dev(rng.standard_normal((T, Hq + 2 * Hkv, 128)).astype(np.float32))
    inv, batch = dev(1e4 ** (-np.arange(64) / 64)), (dev(np.arange(5, dtype=np.int32)[None]), dev(starts([T])), dev(np.array([T], np.int32)))

    def layer(cache, **on):
        rope = spin.spin_rope_table(inv, 128, **on)
        q, k, v = x.split([Hq, Hkv, Hkv], dim=1)
        Q = spin.spin_kv_append(q, k, v, cache, *batch, rope=rope, **on)
        O = spin.spin_kv_attn(Q, cache, *batch, **on)
        return [Q, O, *spin.spin_fwht_quant(O.reshape(T, Hq * 128), 1, **on)[:2]]

    want = [host(t) for t in layer(spin.kv_cache(5, Hkv, 16))]
    cache, s = spin.kv_cache(5, Hkv, 16), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = layer(cache, stream=s)
    s.synchronize()
    assert all(np.array_equal(host(a), b) for a, b in zip(got, want))
