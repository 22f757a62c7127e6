"""GPU parity of append and attention where a sequence's length passes the room of its page table: both go by the same
places, those of the length.  Reference and bounds as in test_gpu_kv_attn.py and test_gpu_kv_append.py."""

import numpy as np
import pytest
import torch

import oracle
from rotation_bit_quantization_amd import spin

from . import test_gpu_kv_append
from .paged_case import close, dev, host, pool, starts, tables
from .test_gpu_kv_attn_tiles import check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spin.load()


MASKS = [dict(), dict(window=5), dict(alibi=True), dict(bidir=True), dict(causal=False, window=40), dict(causal=False)]


@pytest.mark.parametrize("more", MASKS)
@pytest.mark.parametrize("over", [1, 2, 9, 10 ** 6, 2 ** 30 - 64, 2 ** 31 - 65])
@pytest.mark.parametrize("prefix", [0, 40])
def test_attention_of_few_rows(more, over, prefix):
    rng = np.random.default_rng(1)
    first = -(-prefix // 16)
    cache, table = pool(rng, 12, 2, 16, 4), tables(rng, [64, 50], 16, 12, first=first, extra=0)
    check(rng, [4, 3], [64 + over, 50], 8, 2, 4, 16, cache=cache, table=table, before=1, behind=1, prefix_len=prefix, **more)


@pytest.mark.parametrize("more", MASKS[:4])
@pytest.mark.parametrize("Hq,Hkv,room", [(64, 8, 1024), (128, 16, 4096)])      # tiles of 128 rows, of 256
def test_attention_of_many_rows(Hq, Hkv, room, more):
    rng = np.random.default_rng(2)
    n = 2 * room // 64
    cache, table = pool(rng, n + 1, Hkv, 64, 4), tables(rng, [room] * 2, 64, n + 1, extra=0)
    check(rng, [500, 100], [room + 77, room + 9], Hq, Hkv, 4, 64, cache=cache, table=table, most=8, **more)


def test_attention_behind_a_prefix_on_tiles_of_its_own():
    rng = np.random.default_rng(3)
    first = 16500 // 64 + 1
    cache, table = pool(rng, first + 128, 4, 64, 8), first + np.arange(128, dtype=np.int32)[:, None]
    check(rng, [3] * 128, [64 + i % 5 for i in range(128)], 16, 4, 8, 64, cache=cache, table=table, prefix_len=16500, most=10,
          window=16502)


@pytest.mark.parametrize("bits", [4, 8])
def test_append(bits):
    rng = np.random.default_rng(4)
    table = np.array([[1, 0], [2, 3], [5, 4]], np.int32)
    for lens in ([34, 33, 32], [35, 2 ** 31 - 1, 40], [-1, 30, 2 ** 30 + 5]):
        cache = pool(rng, 6, 2, 16, bits)
        test_gpu_kv_append.check(rng, [4, 1, 3], lens, 4, 2, bits, 16, cache=cache, table=table)


@pytest.mark.parametrize("bits", [4, 8])
def test_append_then_attention(bits):
    """The rows that have a page see their own keys, at the positions that they were turned by."""
    rng = np.random.default_rng(5)
    T, Hq, Hkv, kv = 6, 4, 2, [34, 20]
    x = rng.standard_normal((T, Hq + 2 * Hkv, 128)).astype(np.float32)
    table, q_start = np.array([[1, 0], [2, 3]], np.int32), starts([4, 2])
    rope = spin.spin_rope_table(dev(1e4 ** (-np.arange(64) / 64)), 64)
    cache = pool(rng, 4, Hkv, 16, bits)
    d, args = dev(cache), (dev(table), dev(q_start), dev(np.array(kv, np.int32)))
    q, k, v = dev(x).split([Hq, Hkv, Hkv], dim=1)
    Q = spin.spin_kv_append(q, k, v, d, *args, rope=rope)
    mirror, _ = oracle.kv_append(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], cache, table, q_start, kv, rope=host(rope))
    assert all(np.array_equal(host(d[name]).view(np.uint8), mirror[name].view(np.uint8)) for name in mirror)
    for more in (dict(), dict(window=2), dict(window=1)):
        ref, bound = oracle.kv_attend(host(Q), mirror, table, q_start, kv, 128 ** -0.5, **more)
        close(host(spin.spin_kv_attn(Q, d, *args, **more)).astype(np.float64), ref, bound)


@pytest.mark.parametrize("bidir", [-1, -2 ** 31, -2 ** 31 + 40, 2 ** 31 - 1])
@pytest.mark.parametrize("work,q_len,kv_len", [(0, [5, 2], [64, 37]), (2 ** 25, [140, 9], [150, 70]), (2 ** 28, [140, 9], [150, 70])])
@pytest.mark.parametrize("prefix", [0, 40])
def test_prefixes_seen_both_ways_of_any_length(bidir, work, q_len, kv_len, prefix):
    check(np.random.default_rng(6), q_len, kv_len, 4, 2, 4, 16, work, prefix_len=prefix, bidir_len=np.array([bidir, 3], np.int32))
