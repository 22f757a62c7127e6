"""GPU parity of the attention kernels that work on tiles of 128 and 256 rows, and of batches of many sequences.

Which kernel runs goes by rows times the tokens that a page table has room for, so a wide table (-1 behind the pages
that are there) brings short sequences to the large tiles.  Reference and bounds as in test_gpu_kv_attn.py: the
float64 oracle, element by element, within the roundings that it counts."""

import numpy as np
import pytest
import torch

import oracle
from rotation_bit_quantization_amd import spin

from .paged_case import attend, close, dev, host, pool, starts, tables

pytestmark = pytest.mark.gpu
DEV = "cuda"
WORK = [2 ** 25, 2 ** 28]      # rows x tokens x key heads from which tiles of 128, of 256 rows are taken


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spin.load()


def widened(table, rows, Hkv, page, work):
    room = -(-work // (rows * Hkv * page))
    return np.pad(table, ((0, 0), (0, max(room - table.shape[1], 0))), constant_values=-1)


def check(rng, q_len, kv_len, Hq, Hkv, bits, page, work=0, before=0, behind=0, scales=(0.05, 0.5), loud=1.5, cache=None,
          table=None, prefix_len=0, scale=128 ** -0.5, most=10 ** 9, **more):
    """One call against the oracle; of batches with more rows than ``most``, the first and last rows of some sequences
    and random ones are compared (and all that are not written)."""
    q_start = starts(q_len, before)
    T = before + int(sum(q_len)) + behind
    q = (loud * rng.standard_normal((T, Hq, 128))).astype(np.float16)
    first = -(-prefix_len // page)
    n_pages = first + sum(-(-max(n, 0) // page) for n in kv_len) + 2
    cache = pool(rng, n_pages, Hkv, page, bits, scales) if cache is None else cache
    table = tables(rng, kv_len, page, n_pages, first=first) if table is None else table
    table = widened(table, T * Hq // Hkv, Hkv, page, work)
    shared = {}
    if prefix_len:
        shared = dict(prefix_table=rng.permutation(first).astype(np.int32), prefix_len=prefix_len)
    if more.pop("alibi", False):
        more["slopes"] = (2.0 ** (-8 * np.arange(1, Hq + 1) / Hq)).astype(np.float32)
    if more.pop("bidir", False):
        more["bidir_len"] = np.resize(np.array([1000, 0, 40], np.int32), len(q_len))
    rows = range(before, T - behind)
    if len(rows) > most:
        ends = rng.permutation([r for a, b in zip(q_start, q_start[1:]) if b > a for r in (int(a), int(b) - 1)])
        rows = sorted({*ends[:most // 2].tolist(), *rng.choice(rows, most // 2, replace=False).tolist()})
    ref, bound = oracle.kv_attend(q, cache, table, q_start, kv_len, scale, rows=set(rows), **shared, **more)
    got = attend(q, cache, table, q_start, kv_len, scale=scale, **shared, **more)
    rows = [*range(before), *rows, *range(T - behind, T)]
    close(got[rows], ref[rows], bound[rows])
    return got


@pytest.mark.parametrize("work", WORK)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("q_len,kv_len,Hq,Hkv,bits,page", [
    ([64], [64], 1, 1, 4, 16),
    ([70, 2], [200, 2], 8, 1, 4, 128),
    ([129], [129], 2, 2, 4, 32),
    ([131, 40, 1, 0], [300, 40, 65, 9], 8, 2, 8, 64),
    ([260, 33], [333, 700], 2, 1, 4, 16),
    ([37, 1, 18], [37, 80, 130], 36, 3, 8, 16),
    ([0, 300, 0], [7, 1500, 0], 5, 1, 8, 1024),
    ([700], [2500], 6, 2, 4, 32),
])
def test_shapes(work, causal, q_len, kv_len, Hq, Hkv, bits, page):
    rng = np.random.default_rng(len(q_len) * 100 + Hq + bits + page)
    check(rng, q_len, kv_len, Hq, Hkv, bits, page, work, before=2, behind=3, causal=causal, most=200)


@pytest.mark.parametrize("work", WORK)
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("mask", [
    dict(softcap=20.0),
    dict(window=1),
    dict(window=24),
    dict(window=100, softcap=5.0),
    dict(alibi=True),
    dict(bidir=True),
    dict(bidir=True, window=30, alibi=True, softcap=30.0),
    dict(causal=False, window=17),
    dict(causal=False, alibi=True),
])
def test_masks(mask, work, bits):
    rng = np.random.default_rng(7 + bits)
    check(rng, [140, 150, 9], [140, 400, 30], 4, 1, bits, 64, work, **mask)
    check(rng, [90, 0, 77], [500, 40, 70], 6, 2, bits, 16, work, **mask)      # rows before the first token


# the lengths of the page tables that decide over the sequences' own part: on 16 rows, and on the prefix's tiles
@pytest.mark.parametrize("work", [0, 2 ** 25])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("q_len,kv_len,Hq,Hkv,prefix,more", [
    ([40, 35, 70], [40, 60, 70], 16, 8, 16000, {}),
    ([40, 35, 70], [40, 60, 70], 16, 8, 15000, dict(window=14990, softcap=20.0)),
    ([100, 60], [100, 90], 8, 8, 32001, dict(window=300, alibi=True)),
    ([1] * 128, [1 + i % 37 for i in range(128)], 16, 4, 16500, {}),
    ([20, 130, 0, 50], [25, 130, 8, 60], 64, 16, 2600, dict(bidir=True)),
    ([120, 130, 6], [125, 130, 6], 64, 16, 8200, {}),        # on tiles of 256
])
def test_shared_prefix(work, bits, q_len, kv_len, Hq, Hkv, prefix, more):
    rng = np.random.default_rng(bits + prefix)
    check(rng, q_len, kv_len, Hq, Hkv, bits, 64, work, before=1, behind=2, prefix_len=prefix, most=10, **more)


@pytest.mark.parametrize("work", [0] + WORK)
@pytest.mark.parametrize("B,G", [(64, 4), (65, 1), (129, 16), (700, 2)])
def test_many_sequences(work, B, G):
    """More sequences than lanes of a wave, some without rows, some without tokens."""
    rng = np.random.default_rng(B)
    q_len = rng.integers(0, 2 * 70 // G + 2, B)
    q_len[[0, B // 2, B - 1]] = 0, 400 // G, 3
    kv_len = np.where(rng.random(B) < 0.1, 0, q_len + rng.integers(0, 20, B))
    check(rng, q_len.tolist(), kv_len.tolist(), G, 1, 4, 16, work, before=1, behind=1, most=600)


@pytest.mark.parametrize("B", [70, 300, 5000])
def test_many_single_tokens(B):
    rng = np.random.default_rng(B)
    check(rng, [1] * B, rng.integers(0, 60, B).tolist(), 6, 2, 4, 16)


def test_more_sequences_behind_a_prefix_than_a_workgroup_can_list():
    B = 28000
    rng = np.random.default_rng(B)
    check(rng, [1] * B, rng.integers(0, 4, B).tolist(), 1, 1, 4, 16, prefix_len=1300, most=60, before=1, behind=1)


@pytest.mark.parametrize("work", [0] + WORK)
def test_the_widest_window_is_none(work):
    rng = np.random.default_rng(4)
    cache, table = pool(rng, 40, 1, 16, 4), tables(rng, [90, 300], 16, 40)
    q, q_start = rng.standard_normal((160, 2, 128)).astype(np.float16), starts([80, 80])
    table = widened(table, 320, 1, 16, work)
    for causal in (True, False):
        a, b = (attend(q, cache, table, q_start, [90, 300], window=w, causal=causal) for w in (0, 2 ** 31 - 1))
        assert np.array_equal(a, b)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("more", [{}, dict(softcap=20.0), dict(alibi=True, window=2000), dict(bidir=True), dict(causal=False, window=40)])
def test_long_contexts_in_shares(bits, more):
    rng = np.random.default_rng(bits)
    check(rng, [1, 2, 0, 1, 5], [2500, 6000, 3000, 1, 300], 6, 2, bits, 32, **more)
    check(rng, [1, 1], [2048, 513], 20, 1, bits, 16, **more)                  # one share


@pytest.mark.parametrize("B", [8, 9, 33, 64])
@pytest.mark.parametrize("G,Hkv", [(4, 8), (16, 2), (3, 1)])
def test_sequences_taken_in_the_order_of_their_lengths(B, G, Hkv):
    """Equal lengths, lengths of zero, one far longer than the rest; one token each, then some with several tiles."""
    rng = np.random.default_rng(B + G)
    for q_len in (np.ones(B, int), rng.integers(0, 9, B)):
        for kv_len in (np.full(B, 70), q_len + rng.integers(0, 200, B), np.where(np.arange(B) == B // 2, 2600, q_len)):
            kv_len = kv_len * (rng.random(B) > 0.1)
            table = tables(rng, kv_len, 64, int((-(-kv_len // 64)).sum()) + 2)
            table = np.pad(table, ((0, 0), (0, max(0, 40 - table.shape[1]))), constant_values=-1)      # room for 2560 tokens
            check(rng, q_len.tolist(), kv_len.tolist(), G * Hkv, Hkv, 4, 64, table=table, before=1, behind=1, most=40)


def test_one_long_sequence_among_many():
    """Shares of one size for all, of which the others have one."""
    rng = np.random.default_rng(2)
    kv_len = rng.integers(0, 40, 260)
    kv_len[[3, 200]] = 17000, 8200
    check(rng, [1] * 260, kv_len.tolist(), 2, 1, 4, 64)
    check(rng, [1] * 260, kv_len.tolist(), 16, 1, 8, 64, most=60)


@pytest.mark.parametrize("work", WORK)
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("which", ["K_scale", "V_scale"])
def test_scales_that_are_not_finite(bits, bad, which, work):
    rng = np.random.default_rng(8)
    kv, q_len = 160, 150
    cache = pool(rng, 16, 2, 16, bits)
    table = tables(rng, [kv - 3], 16, 16)
    cache[which][table[0, (kv - 4) // 16], :, (kv - 3) % 16:] = bad
    cache[which][np.setdiff1d(np.arange(16), table[0])] = bad
    for more in (dict(), dict(softcap=10.0, alibi=True)):
        check(rng, [q_len], [kv - 3], 4, 2, bits, 16, work, cache=cache, table=table, **more)
    cache[which][table[0, 2], 1, 5] = bad                      # token 37 of head 1
    for more in (dict(), dict(softcap=10.0, alibi=True), dict(window=4)):
        check(rng, [q_len], [kv - 3], 4, 2, bits, 16, work, cache=cache, table=table, **more)


@pytest.mark.parametrize("work", WORK)
def test_scales_of_every_size(work):
    rng = np.random.default_rng(9)
    kv = 200
    cache = pool(rng, 14, 2, 16, 4)
    cache["V_scale"][:] = (2.0 ** rng.uniform(-24, 15.9, cache["V_scale"].shape)).astype(np.float16)
    check(rng, [150], [kv], 2, 2, 4, 16, work, cache=cache)
    cache["V_scale"][:] = 2.0 ** -24
    check(rng, [150], [kv], 2, 2, 4, 16, work, cache=cache)
    cache["V_scale"][:] = 0
    cache["V_codes"][:] = 0
    assert (check(rng, [150], [kv], 2, 2, 4, 16, work, cache=cache) == 0).all()
    some = pool(rng, 14, 2, 16, 4)
    some["K_scale"][:] = (2.0 ** rng.uniform(-24, 0, some["K_scale"].shape)).astype(np.float16)
    check(rng, [150], [kv], 2, 2, 4, 16, work, cache=some, loud=20.0)
    for loud in (0.0, 0.01, 30.0):
        check(rng, [140], [300], 4, 2, 8, 32, work, loud=loud)
    check(rng, [140], [300], 4, 2, 8, 32, work, scale=-0.3)
    check(rng, [140], [300], 4, 2, 8, 32, work, scale=0.0)


@pytest.mark.parametrize("work", WORK)
def test_pages_that_are_not_there(work):
    rng = np.random.default_rng(5)
    cache = pool(rng, 3, 2, 16, 4)
    for bad in (-1, 3, 2 ** 31 - 1, -2 ** 31):
        assert (check(rng, [70], [80], 2, 2, 4, 16, work, cache=cache, table=np.full((1, 5), bad, np.int32)) == 0).all()
    check(rng, [80, 90], [40, 48], 4, 2, 4, 16, work, cache=cache, table=np.array([[2, -1, 0], [1, 7, 2]], np.int32))


@pytest.mark.parametrize("work", WORK)
def test_offsets_that_pass_32_bits(work):
    """A pool of 5 GiB of key codes, with the sequence's pages at its end."""
    rng = np.random.default_rng(12)
    n_pages, Hkv, page, T = 40960, 8, 256, 130
    small = pool(rng, 3, Hkv, page, 4)
    used = np.array([n_pages - 1, n_pages - 3, n_pages - 2])
    big = spin.kv_cache(n_pages, Hkv, page, 4)
    for name, a in small.items():
        big[name][torch.from_numpy(used).to(DEV)] = dev(a)
    q = rng.standard_normal((T, 16, 128)).astype(np.float16)
    wide = lambda t: widened(np.asarray(t, np.int32)[None], T * 2, Hkv, page, work)  # noqa: E731
    want = attend(q, small, wide([0, 1, 2]), [0, T], [700])
    O = spin.spin_kv_attn(dev(q), big, dev(wide(used)), dev(np.array([0, T], np.int32)), dev(np.array([700], np.int32)))
    assert np.array_equal(host(O).astype(np.float64), want)


@pytest.mark.parametrize("work", WORK)
@pytest.mark.parametrize("q_start", [[0, 2 ** 31 - 1, -2 ** 31, 90], [90, 0, 90, 0], [5, 5, 5, 5], [-2 ** 31, 0, 0, 2 ** 31 - 1],
                                     [200, 300, 400, 500]])
@pytest.mark.parametrize("prefix", [0, 40])
def test_borders_that_do_not_ascend_stay_in_bounds(work, q_start, prefix):
    """What such a call writes is not defined; it writes rows of O only."""
    rng = np.random.default_rng(16)
    cache, table = pool(rng, 24, 1, 16, 4), tables(rng, [100] * 3, 16, 24, first=3)
    q = rng.standard_normal((100, 4, 128)).astype(np.float16)
    table = widened(np.maximum(table, 0), 400, 1, 16, work)
    guard = torch.full((3, 100, 4, 128), 77.0, dtype=torch.float16, device=DEV)
    args = (dev(table), dev(np.array(q_start, np.int32)), dev(np.array([100, 90, -4], np.int32)))
    if prefix:
        spin.spin_kv_attn_shared(dev(q), dev(cache), dev(np.arange(3, dtype=np.int32)), prefix, *args, O=guard[1])
    else:
        spin.spin_kv_attn(dev(q), dev(cache), *args, O=guard[1])
    assert (host(guard[::2]) == 77.0).all()


@pytest.mark.parametrize("work", WORK)
def test_captured_calls_replay(work):
    rng = np.random.default_rng(13)
    Hq, Hkv, page, kv, q_len = 8, 2, 16, [300, 410, 200], [40, 100, 3]
    cache = pool(rng, 80, Hkv, page, 4)
    table = dev(widened(tables(rng, kv, page, 80), sum(q_len) * 4, Hkv, page, work))
    q, q_start, kv_d = dev(rng.standard_normal((sum(q_len), Hq, 128)).astype(np.float16)), dev(starts(q_len)), dev(np.array(kv, np.int32))
    cache = dev(cache)
    O = torch.zeros_like(q)
    call = lambda: spin.spin_kv_attn(q, cache, table, q_start, kv_d, O=O)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        graphs.append(g)
    for rep, less in enumerate([0, 7, 100, 0]):
        kv_d.copy_(torch.tensor([n - less for n in kv], dtype=torch.int32))
        want = host(call()).copy()
        for g in graphs:
            O.fill_(5.0)
            g.replay()
            assert np.array_equal(host(O), want), rep


def test_numbers_beyond_32_bits_are_refused():
    rng = np.random.default_rng(15)
    cache, q = dev(pool(rng, 4, 2, 16, 4)), dev(rng.standard_normal((2, 4, 128)).astype(np.float16))
    batch = dev(np.zeros((1, 2), np.int32)), dev(np.array([0, 2], np.int32)), dev(np.array([20], np.int32))
    for bad in (dict(window=2 ** 32 + 5), dict(window=-2 ** 32 + 5), dict(causal=2 ** 32 + 1)):
        with pytest.raises(ValueError):
            spin.spin_kv_attn(q, cache, *batch, **bad)
    with pytest.raises(ValueError):
        spin.spin_kv_append(q, q[:, :2].contiguous(), q[:, :2].contiguous(), cache, *batch, pos0=2 ** 32)
    with pytest.raises(ValueError):
        spin.spin_rope_table(torch.ones(4, dtype=torch.float64, device=DEV), 8, pos0=2 ** 32)
