"""Pins of oracle/paged.py that do not use its own code: rotations as complex products, attention against torch's
softmax on contiguous heads, the cache layouts by hand."""

import numpy as np
import pytest
import torch

import oracle
from oracle.paged import cache_tokens, turn_heads

rng = np.random.default_rng(31)


def test_rotation_is_a_complex_product_and_keeps_relative_positions():
    inv = 1e4 ** (-np.arange(32) / 32)
    table = oracle.rope_table(inv, 50, 3, 1.0)
    assert np.allclose(table[7, :32] + 1j * table[7, 32:], np.exp(1j * 10 * inv), atol=1e-15)
    x = rng.standard_normal((2, 1, 128))
    for inter in (False, True):
        a = turn_heads(np.stack([x[0], x[0]]), table[[4, 9]], inter)
        b = turn_heads(np.stack([x[1], x[1]]), table[[11, 16]], inter)
        assert np.allclose((a[0] * b[0]).sum(), (a[1] * b[1]).sum())      # the same distance
        assert np.allclose(np.linalg.norm(a[0]), np.linalg.norm(x[0]))


def test_norm_makes_the_mean_square_one():
    x = 5 * rng.standard_normal((3, 2, 128))
    y = turn_heads(x, weight=np.ones(128))
    assert np.allclose((y * y).mean(-1), 1)


def test_layouts():
    k, v = rng.standard_normal((2, 5, 1, 128)).astype(np.float32)
    empty = {"K_codes": np.zeros((3, 1, 16, 64), np.uint8), "K_scale": np.zeros((3, 1, 16), np.float16),
             "V_codes": np.zeros((3, 1, 4, 16, 4, 4), np.uint8), "V_scale": np.zeros((3, 1, 16), np.float16)}
    cache, q = oracle.kv_append(np.zeros((5, 1, 128)), k, v, empty, np.array([[2, 1]]), [0, 5], [18])
    codes, scale, _ = oracle.kv_quant(v, False)
    # token 3 is place 16: page 1, slot 0; token 1 place 14: page 2, slot 14 = quad 3, token 2 of it
    assert np.array_equal(cache["V_codes"][1, 0, 0, :, 0].reshape(64), codes[3, 0])
    assert np.array_equal(cache["V_codes"][2, 0, 3, :, 2].reshape(64), codes[1, 0])
    assert cache["V_scale"][2, 0, 14] == scale[1, 0]
    codes, scale, _ = oracle.kv_quant(k, True)
    assert np.array_equal(cache["K_codes"][2, 0, 13], codes[0, 0]) and cache["K_scale"][2, 0, 13] == scale[0, 0]
    kc, ks, vc, vs, there = cache_tokens(cache, [2, 1], 0, 18)
    assert there.all() and np.array_equal(vc[16], oracle.unpack_int4(cache["V_codes"][1, 0, 0, :, 0].reshape(64)))


@pytest.mark.parametrize("causal", [True, False])
def test_attention_is_softmax(causal):
    n, Hq, H = 21, 4, 2
    x = rng.standard_normal((n, H, 128)).astype(np.float32)
    q = rng.standard_normal((n, Hq, 128))
    cache = {"K_codes": np.zeros((2, H, 16, 128), np.uint8), "K_scale": np.zeros((2, H, 16), np.float16),
             "V_codes": np.zeros((2, H, 4, 16, 4, 8), np.uint8), "V_scale": np.zeros((2, H, 16), np.float16)}
    cache, _ = oracle.kv_append(q, x, x[::-1], cache, np.array([[0, 1]]), [0, n], [n])
    got, bound = oracle.kv_attend(q, cache, np.array([[0, 1]]), [0, n], [n], 0.05, causal=causal)
    codes, scale, _ = oracle.kv_quant8(x, True)
    k = torch.from_numpy(codes.astype(np.float64) * scale[..., None]).repeat_interleave(2, 1).transpose(0, 1)
    codes, scale, _ = oracle.kv_quant8(x[::-1], False)
    v = torch.from_numpy(codes.astype(np.float64) * scale[..., None]).repeat_interleave(2, 1).transpose(0, 1)
    z = torch.from_numpy(q).transpose(0, 1) @ k.transpose(1, 2) * 0.05
    if causal:
        z = z.masked_fill(torch.ones(n, n).triu(1).bool(), -np.inf)
    assert np.allclose(got, (z.softmax(-1) @ v).transpose(0, 1).numpy(), atol=1e-12)
    assert (bound > 0).all() and bound.max() < 0.01


def test_lengths_past_the_table():
    """Appended and attended tokens stand at the same places: a table with room for 32 of 34 tokens is one whose third
    page is none of the pool, and the new tokens that have a page see themselves."""
    n, H = 4, 1
    x, q = rng.standard_normal((n, H, 128)).astype(np.float32), rng.standard_normal((n, H, 128))
    empty = {"K_codes": np.zeros((2, H, 16, 128), np.uint8), "K_scale": np.zeros((2, H, 16), np.float16),
             "V_codes": np.zeros((2, H, 4, 16, 4, 8), np.uint8), "V_scale": np.zeros((2, H, 16), np.float16)}
    short, wide = np.array([[0, 1]]), np.array([[0, 1, -1]])
    a, qa = oracle.kv_append(q, x, x, empty, short, [0, n], [34])
    b, qb = oracle.kv_append(q, x, x, empty, wide, [0, n], [34])
    assert all(np.array_equal(a[k], b[k]) for k in a)
    assert np.array_equal(qa[:2], qb[:2]) and (qa[2:] == 0).all()
    assert (a["K_scale"][1, 0, 14:] > 0).all() and (a["K_scale"][0] == 0).all() and (a["K_scale"][1, 0, :14] == 0).all()
    for more in (dict(), dict(window=3), dict(slopes=np.array([0.3], np.float32)), dict(bidir_len=[5])):
        u, _ = oracle.kv_attend(q, a, short, [0, n], [34], 0.1, **more)
        v, _ = oracle.kv_attend(q, a, wide, [0, n], [34], 0.1, **more)
        assert np.array_equal(u, v)
    # of a window of one token each row sees the value that it appended itself, the last two nothing
    u, _ = oracle.kv_attend(q, a, short, [0, n], [34], 0.1, window=1)
    codes, scale, _ = oracle.kv_quant8(x, False)
    assert np.allclose(u[:2], (codes * scale[..., None].astype(np.float64))[:2]) and (u[2:] == 0).all()
