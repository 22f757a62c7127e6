"""GPU parity of spin_kv_attn and spin_kv_attn_shared with the float64 oracle (oracle.kv_attend), element by
element within the bound that the oracle derives from the roundings the operator makes.  No run of this file has
set a tolerance: they are counted in oracle/paged.py."""

import numpy as np
import pytest
import torch

import oracle
from rotation_bit_quantization_amd import spin

from .paged_case import attend, close, dev, host, pool, starts, tables

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spin.load()


def check(rng, q_len, kv_len, Hq, Hkv, bits, page, before=0, behind=0, scales=(0.05, 0.5), loud=1.5, cache=None, table=None,
          prefix_len=0, scale=128 ** -0.5, **more):
    """One call against the oracle; `before` / `behind`: rows of no sequence around the batch's."""
    q_start = starts(q_len, before)
    T = before + int(sum(q_len)) + behind
    q = (loud * rng.standard_normal((T, Hq, 128))).astype(np.float16)
    first = -(-prefix_len // page)
    n_pages = first + sum(-(-max(n, 0) // page) for n in kv_len) + 2
    cache = pool(rng, n_pages, Hkv, page, bits, scales) if cache is None else cache
    table = tables(rng, kv_len, page, n_pages, first=first) if table is None else table
    shared = {}
    if prefix_len:
        shared = dict(prefix_table=rng.permutation(first).astype(np.int32), prefix_len=prefix_len)
    ref, bound = oracle.kv_attend(q, cache, table, q_start, kv_len, scale, **shared, **more)
    got = attend(q, cache, table, q_start, kv_len, scale=scale, **shared, **more)
    close(got, ref, bound)
    return got


SHAPES = [
    # q_len, kv_len, Hq, Hkv, bits, page
    ([1], [1], 1, 1, 4, 16),
    ([1, 1, 1], [17, 1, 64], 4, 2, 4, 16),
    ([1, 1, 1, 1, 1], [33, 500, 31, 32, 257], 8, 2, 8, 32),
    ([1] * 4, [700, 3, 1029, 256], 5, 1, 4, 64),
    ([3, 1, 0, 6], [40, 9, 0, 6], 6, 2, 4, 16),
    ([0, 0], [5, 0], 2, 2, 4, 16),
    ([37, 1, 18], [37, 80, 130], 3, 3, 8, 16),
    ([70, 2], [200, 2], 8, 1, 4, 128),
    ([129], [129], 2, 2, 4, 32),
    ([131, 40, 1], [300, 40, 65], 4, 2, 8, 64),
    ([260, 33], [333, 700], 2, 1, 4, 16),
    ([1, 1], [40, 33], 80, 4, 4, 1024),
]


@pytest.mark.parametrize("q_len,kv_len,Hq,Hkv,bits,page", SHAPES)
@pytest.mark.parametrize("causal", [True, False])
def test_shapes(q_len, kv_len, Hq, Hkv, bits, page, causal):
    rng = np.random.default_rng(len(q_len) * 100 + Hq + bits + page)
    check(rng, q_len, kv_len, Hq, Hkv, bits, page, before=2, behind=3, causal=causal)


MASKS = [
    dict(softcap=20.0),
    dict(window=1),
    dict(window=24),
    dict(window=100, softcap=5.0),
    dict(alibi=True),
    dict(bidir=True),
    dict(bidir=True, window=30, alibi=True, softcap=30.0),
    dict(causal=False, window=17),
    dict(causal=False, alibi=True),
]


@pytest.mark.parametrize("mask", MASKS)
@pytest.mark.parametrize("q_len,kv_len,Hq,Hkv,bits,page", [
    ([1, 1, 1], [300, 5, 77], 8, 2, 4, 16), ([50, 1, 9], [120, 33, 9], 4, 2, 8, 32), ([140, 150], [140, 400], 4, 1, 4, 64)])
def test_masks(mask, q_len, kv_len, Hq, Hkv, bits, page):
    rng = np.random.default_rng(7 + Hq + bits)
    more = dict(mask)
    if more.pop("alibi", False):
        more["slopes"] = (2.0 ** (-8 * np.arange(1, Hq + 1) / Hq)).astype(np.float32)
    if more.pop("bidir", False):
        more["bidir_len"] = np.array([0, 40, 1000][:len(q_len)], np.int32)[::-1].copy()
    check(rng, q_len, kv_len, Hq, Hkv, bits, page, **more)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("q_len,kv_len,prefix,more", [
    ([1, 1, 1, 1], [3, 17, 1, 60], 100, {}),
    ([1, 1, 1, 1], [0, 17, 1, 60], 16, {}),
    ([1] * 9, [5] * 9, 1000, dict(softcap=15.0)),
    ([20, 1, 3], [25, 8, 3], 333, dict(window=50)),
    ([20, 1, 3], [25, 8, 3], 333, dict(window=350, alibi=True)),
    ([40, 35, 70], [40, 60, 70], 129, dict(bidir=True)),
    ([2, 2], [2, 5], 1, dict(causal=False)),
])
def test_shared_prefix(bits, q_len, kv_len, prefix, more):
    rng = np.random.default_rng(bits + prefix)
    more = dict(more)
    if more.pop("alibi", False):
        more["slopes"] = np.array([0.5, 0.1, 0.0, 0.02], np.float32)
    if more.pop("bidir", False):
        more["bidir_len"] = np.array([0, 160, 60], np.int32)
    check(rng, q_len, kv_len, 4, 2, bits, 16, before=1, behind=2, prefix_len=prefix, **more)


def test_shared_prefix_of_no_tokens_is_plain_attention():
    rng = np.random.default_rng(3)
    cache = pool(rng, 9, 2, 16, 4)
    q = rng.standard_normal((3, 4, 128)).astype(np.float16)
    table, q_start, kv = tables(rng, [40, 33], 16, 9), starts([1, 2]), [40, 33]
    a = attend(q, cache, table, q_start, kv)
    b = attend(q, cache, table, q_start, kv, prefix_table=np.zeros(1, np.int32), prefix_len=0)
    assert np.array_equal(a, b)


def test_rows_without_a_visible_token_are_zero():
    rng = np.random.default_rng(5)
    # fewer tokens than rows: the first rows stand before the first token
    got = check(rng, [6, 3], [2, 0], 2, 2, 4, 16)
    assert (got[:4] == 0).all() and (got[6:] == 0).all() and (got[4:6] != 0).any()
    # no page of the table is in the pool
    cache = pool(rng, 3, 2, 16, 4)
    for bad in (-1, 3, 2 ** 31 - 1, -2 ** 31):
        got = check(rng, [2], [30], 2, 2, 4, 16, cache=cache, table=np.full((1, 2), bad, np.int32))
        assert (got == 0).all()
    # one page of three is missing: its tokens are left out
    check(rng, [1, 20], [40, 48], 4, 2, 4, 16, cache=cache, table=np.array([[2, -1, 0], [1, 7, 2]], np.int32))


def test_lengths_beyond_the_table_count_as_its_room():
    rng = np.random.default_rng(6)
    cache = pool(rng, 4, 1, 16, 4)
    table = np.array([[1, 3]], np.int32)
    q = rng.standard_normal((1, 2, 128)).astype(np.float16)
    assert np.array_equal(attend(q, cache, table, [0, 1], [2 ** 31 - 1]), attend(q, cache, table, [0, 1], [32]))
    assert (attend(q, cache, table, [0, 1], [-5]) == 0).all()


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("which", ["K_scale", "V_scale"])
@pytest.mark.parametrize("q_len,kv", [(1, 50), (40, 50), (150, 160)])
def test_scales_that_are_not_finite(bits, bad, which, q_len, kv):
    """Unwritten slots, unused pages and masked tokens may hold anything; a row that sees such a token is NaN."""
    rng = np.random.default_rng(8)
    cache = pool(rng, 16, 2, 16, bits)
    table = tables(rng, [kv], 16, 16)
    last = table[0, (kv - 1) // 16]
    cache[which][last, :, kv % 16:] = bad                      # behind the last token of its page
    free = np.setdiff1d(np.arange(16), table[0])
    cache[which][free] = bad
    check(rng, [q_len], [kv], 4, 2, bits, 16, cache=cache, table=table)
    cache[which][table[0, 2], 1, 5] = bad                      # token 37 of head 1
    check(rng, [q_len], [kv], 4, 2, bits, 16, cache=cache, table=table)
    check(rng, [q_len], [kv], 4, 2, bits, 16, cache=cache, table=table, window=4)


@pytest.mark.parametrize("q_len", [1, 150])
def test_scales_of_every_size(q_len):
    rng = np.random.default_rng(9)
    kv = 200
    cache = pool(rng, 14, 2, 16, 4)
    cache["V_scale"][:] = (2.0 ** rng.uniform(-24, 15.9, cache["V_scale"].shape)).astype(np.float16)
    check(rng, [q_len], [kv], 2, 2, 4, 16, cache=cache)
    cache["V_scale"][:] = 2.0 ** -24                           # the smallest fp16
    check(rng, [q_len], [kv], 2, 2, 4, 16, cache=cache)
    cache["V_scale"][:] = 0                                    # codes of a zero scale are zeros
    cache["V_codes"][:] = 0
    assert (check(rng, [q_len], [kv], 2, 2, 4, 16, cache=cache) == 0).all()
    some = pool(rng, 14, 2, 16, 4)
    zero = rng.random((14, 2, 4, 4)) < 0.5
    some["V_scale"][zero.reshape(14, 2, 16)] = 0
    some["V_codes"].transpose(0, 1, 2, 4, 3, 5)[zero] = 0
    check(rng, [q_len], [kv], 2, 2, 4, 16, cache=some)
    some["K_scale"][:] = (2.0 ** rng.uniform(-24, 0, some["K_scale"].shape)).astype(np.float16)
    check(rng, [q_len], [kv], 2, 2, 4, 16, cache=some, loud=20.0)


@pytest.mark.parametrize("q_len", [1, 140])
def test_peaked_and_flat_scores(q_len):
    rng = np.random.default_rng(10)
    for loud in (0.0, 0.01, 30.0):
        check(rng, [q_len], [300], 4, 2, 8, 32, loud=loud)
    check(rng, [q_len], [300], 4, 2, 8, 32, scale=-0.3)
    check(rng, [q_len], [300], 4, 2, 8, 32, scale=0.0)


@pytest.mark.parametrize("kv", [2047, 2048, 2049, 5000])
def test_long_contexts_split_over_workgroups(kv):
    check(np.random.default_rng(kv), [1, 1], [kv, kv // 3], 4, 1, 4, 16)
    check(np.random.default_rng(kv), [2], [kv], 8, 1, 8, 64, window=kv // 2)


def test_offsets_that_pass_32_bits():
    """A pool of 5 GiB of key codes, with the sequence's pages at its end."""
    rng = np.random.default_rng(12)
    n_pages, Hkv, page = 40960, 8, 256
    small = pool(rng, 3, Hkv, page, 4)
    used = np.array([n_pages - 1, n_pages - 3, n_pages - 2])
    big = spin.kv_cache(n_pages, Hkv, page, 4)
    for name, a in small.items():
        big[name][torch.from_numpy(used).to(DEV)] = dev(a)
    q = rng.standard_normal((130, 16, 128)).astype(np.float16)
    for q_len in (1, 130):
        want = attend(q[:q_len], small, np.array([[0, 1, 2]], np.int32), [0, q_len], [700])
        O = spin.spin_kv_attn(dev(q[:q_len]), big, dev(used[None].astype(np.int32)), dev(np.array([0, q_len], np.int32)),
                              dev(np.array([700], np.int32)))
        assert np.array_equal(host(O).astype(np.float64), want)


@pytest.mark.parametrize("q_len,prefix", [([1, 1, 1], 0), ([1, 1, 1], 600), ([40, 100, 3], 0)])
def test_captured_calls_replay(q_len, prefix):
    """Two graphs of the same call, replayed in turn with eager work between: the lengths they read are the
    device's at replay."""
    rng = np.random.default_rng(13)
    Hq, Hkv, page = 8, 2, 16
    kv = [300, 410, 200]
    first = -(-prefix // page)
    cache = pool(rng, 80 + first, Hkv, page, 4)
    table = dev(tables(rng, kv, page, 80 + first, first=first))
    q, q_start, kv_d = dev(rng.standard_normal((sum(q_len), Hq, 128)).astype(np.float16)), dev(starts(q_len)), dev(np.array(kv, np.int32))
    cache, front = dev(cache), dev(np.arange(max(first, 1), dtype=np.int32))
    O = torch.zeros_like(q)

    def call():
        if prefix:
            return spin.spin_kv_attn_shared(q, cache, front, prefix, table, q_start, kv_d, O=O)
        return spin.spin_kv_attn(q, cache, table, q_start, kv_d, O=O)

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


def test_on_another_stream_and_with_a_workspace():
    rng = np.random.default_rng(14)
    cache, kv = dev(pool(rng, 200, 1, 16, 4)), [3000]
    q = dev(rng.standard_normal((1, 8, 128)).astype(np.float16))
    args = (q, cache, dev(tables(rng, kv, 16, 200)), dev(starts([1])), dev(np.array(kv, np.int32)))
    want = host(spin.spin_kv_attn(*args))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = spin.spin_kv_attn(*args, stream=s)
    s.synchronize()
    assert np.array_equal(host(got), want)
    got = spin.spin_kv_attn(*args, stream=s.cuda_stream)
    s.synchronize()
    assert np.array_equal(host(got), want)
    need = spin.spin_kv_attn_workspace(1, 8, 1, 1, args[2].shape[1], 16)
    assert need > 0
    ws = torch.full((need + 64,), 255, dtype=torch.uint8, device=DEV)
    assert np.array_equal(host(spin.spin_kv_attn(*args, workspace=ws)), want)
    assert (host(ws)[need:] == 255).all()
    with pytest.raises(spin.SpinError):
        spin.spin_kv_attn(*args, workspace=ws[:need - 16])


def test_the_binding_refuses():
    rng = np.random.default_rng(15)
    cache = dev(pool(rng, 4, 2, 16, 4))
    q, table = dev(rng.standard_normal((2, 4, 128)).astype(np.float16)), dev(np.zeros((1, 2), np.int32))
    q_start, kv = dev(np.array([0, 2], np.int32)), dev(np.array([20], np.int32))
    ok = dict(Q=q, cache=cache, page_table=table, q_start=q_start, kv_len=kv)
    spin.spin_kv_attn(**ok)
    for bad in (dict(Q=q.float()), dict(Q=q[:, :, ::2]), dict(Q=q.cpu()), dict(kv_len=kv.long()), dict(kv_len=kv.repeat(2)),
                dict(q_start=q_start[:1]), dict(page_table=table[0]), dict(cache=dict(cache, V_codes=cache["V_codes"][:3])),
                dict(cache=dict(cache, K_scale=cache["K_scale"].float())), dict(Q=q[:, :3].contiguous()),
                dict(slopes=torch.ones(3, device=DEV)), dict(window=-1), dict(softcap=float("nan")), dict(scale=float("inf")),
                dict(bidir_len=torch.ones(2, dtype=torch.int32, device=DEV)), dict(O=torch.empty_like(q.float()))):
        with pytest.raises((ValueError, TypeError, spin.SpinError)):
            spin.spin_kv_attn(**dict(ok, **bad))
    with pytest.raises(ValueError):
        spin.spin_kv_attn_shared(q, cache, table[0], 33, table, q_start, kv)
