"""Eviction from the paged cache: the weight that tokens draw, the choice of those that stay, their move.  Weights against
the float64 oracle within the roundings that it counts, choices and bytes equal."""

import numpy as np
import pytest
import torch

import oracle
from rotation_bit_quantization_amd import spin

from .paged_case import DEV, dev, host, pool, starts, tables

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spin.load()


def weigh(q, lse, cache, table, q_start, kv_len, W, prior=None, **more):
    more = {k: dev(v) if isinstance(v, np.ndarray) else v for k, v in more.items()}
    spin.spin_kv_weights(dev(q), dev(lse), dev(cache), dev(table), dev(q_start), dev(np.asarray(kv_len, np.int32)), W=W,
                         prior=dev(prior), **more)
    return host(W).astype(np.float64)


def check(rng, q_len, kv_len, Hq, Hkv, bits, page, before=0, behind=0, prior=False, decay=1.0, cache=None, table=None, pos0=0,
          q=None, exact_logs=True, room=0, **more):
    q_start = starts(q_len, before)
    T = before + int(sum(q_len)) + behind
    q = (1.5 * rng.standard_normal((T, Hq, 128))).astype(np.float16) if q is None else q
    n_pages = sum(-(-max(n, 0) // page) for n in kv_len) + 2
    cache = pool(rng, n_pages, Hkv, page, bits) if cache is None else cache
    n_pages = len(cache["K_scale"])
    table = tables(rng, kv_len, page, n_pages) if table is None else table
    table = np.pad(table, ((0, 0), (0, max(room // page - table.shape[1], 0))), constant_values=-1)
    if more.pop("alibi", False):
        more["slopes"] = (2.0 ** (-8 * np.arange(1, Hq + 1) / Hq)).astype(np.float32)
    if more.pop("bidir", False):
        more["bidir_len"] = np.resize(np.array([pos0 + 100, 0, pos0 + 40], np.int32), len(q_len))
    if exact_logs:
        rows = dict(more, bidir_len=np.maximum(more["bidir_len"] - pos0, 0)) if "bidir_len" in more else more
        _, _, lse, _ = oracle.kv_attend(q, cache, table, q_start, kv_len, 128 ** -0.5, sums=True, **rows)
    else:
        lse = rng.uniform(0, 9, (T, Hq))
    lse = np.where(np.isnan(lse), 1.0, lse).astype(np.float32)
    old = rng.random((n_pages, Hkv, page)).astype(np.float32) if prior else None
    ref, bound = oracle.kv_weights(q, lse, cache, table, q_start, kv_len, 128 ** -0.5, prior=old, decay=decay, pos0=pos0, **more)
    got = weigh(q, lse, cache, table, q_start, kv_len, torch.full((n_pages, Hkv, page), 77.0, device=DEV), old, decay=decay, pos0=pos0,
                **more)
    written = ~np.isnan(ref)
    assert (got[~written] == 77.0).all()
    off = np.abs(got - ref)[written] - bound[written]
    assert off.size == 0 or off.max() <= 0, (off.max(), ref[written].max())
    again = weigh(q, lse, cache, table, q_start, kv_len, torch.full((n_pages, Hkv, page), 77.0, device=DEV), old, decay=decay, pos0=pos0,
                  **more)
    assert np.array_equal(got, again)
    return np.where(written, got, 0.0), lse


@pytest.mark.parametrize("q_len,kv_len,Hq,Hkv,bits,page", [
    ([1], [1], 1, 1, 4, 16),
    ([1, 1, 1], [64, 65, 300], 8, 2, 8, 16),
    ([1, 0, 1], [700, 20, 1], 5, 1, 4, 128),
    ([16, 17], [80, 17], 3, 3, 4, 32),
    ([130, 2, 0], [300, 2, 40], 8, 2, 8, 64),
    ([33, 1, 70], [600, 257, 255], 36, 3, 4, 16),
    ([300], [300], 5, 1, 8, 1024),
    ([1] * 70, [1 + 9 * i for i in range(70)], 16, 2, 4, 16),
    ([90, 0, 77], [50, 40, 70], 6, 2, 4, 16),                 # rows before the first token
    ([700], [2300], 6, 2, 4, 64),
])
@pytest.mark.parametrize("causal", [True, False])
def test_weights(q_len, kv_len, Hq, Hkv, bits, page, causal):
    rng = np.random.default_rng(len(q_len) * 100 + Hq + bits)
    check(rng, q_len, kv_len, Hq, Hkv, bits, page, before=1, behind=2, causal=causal)
    check(rng, q_len, kv_len, Hq, Hkv, bits, page, causal=causal, prior=True, decay=0.75)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("more", [
    dict(softcap=20.0),
    dict(softcap=1e4),
    dict(window=1),
    dict(window=24),
    dict(window=100, softcap=5.0),
    dict(alibi=True),
    dict(bidir=True),
    dict(bidir=True, window=30, alibi=True, softcap=30.0),
    dict(causal=False, window=17),
    dict(causal=False, alibi=True),
    dict(window=2 ** 31 - 1),
    dict(window=2 ** 31 - 1, causal=False),
])
@pytest.mark.parametrize("pos0", [0, 1000])
def test_masks(more, bits, pos0):
    rng = np.random.default_rng(7 + bits)
    check(rng, [140, 150, 9], [140, 400, 30], 4, 1, bits, 64, pos0=pos0, **more)
    check(rng, [1, 90, 0, 77], [333, 500, 40, 170], 6, 2, bits, 16, pos0=pos0, prior=True, decay=0.0, **more)


# Which kernel runs goes by rows, heads and the tables' room: one group of 64 tokens a wave or several in turn, 32 or 64
# tokens a wave with all rows or a share of them.
@pytest.mark.parametrize("q_len,kv_len,Hq,Hkv,page,room", [
    ([1, 3, 0, 2, 1, 1, 1, 1], [900, 70, 33, 2000, 64, 65, 1, 513], 32, 8, 16, 16384),
    ([1] * 8, [900, 70, 33, 2000, 64, 5000, 1, 513], 16, 8, 64, 131072 + 1024),
    ([20] * 8, [900, 70, 33, 2000, 64, 65, 20, 513], 8, 8, 64, 16384),
    ([300], [1100], 4, 1, 16, 66000),
    ([300, 17], [300, 400], 5, 1, 64, 40000),
    ([40, 0, 90], [600, 300, 90], 96, 32, 64, 1500),
    ([1, 2] * 140, [(37 * i) % 300 + 2 for i in range(280)], 2, 1, 16, 0),
])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("more", [{}, dict(softcap=20.0, alibi=True, bidir=True), dict(window=100)])
def test_kernels(q_len, kv_len, Hq, Hkv, page, room, bits, more):
    rng = np.random.default_rng(Hq + room)
    check(rng, q_len, kv_len, Hq, Hkv, bits, page, before=1, behind=1, prior=True, decay=0.5, room=room, **more)


def test_shares_in_a_workspace_of_the_callers():
    rng = np.random.default_rng(9)
    q, lse = rng.standard_normal((700, 8, 128)).astype(np.float16), rng.uniform(5, 9, (700, 8)).astype(np.float32)
    cache, table = pool(rng, 60, 2, 16, 4), tables(rng, [900], 16, 60)
    need = spin.spin_kv_weights_workspace(700, 8, 2, 1, table.shape[1], 16)
    assert need > 0
    W = lambda: torch.zeros((60, 2, 16), device=DEV)  # noqa: E731
    a = weigh(q, lse, cache, table, starts([700]), [900], W())
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)            # NaN wherever it is read unwritten
    b = weigh(q, lse, cache, table, starts([700]), [900], W(), workspace=ws)
    assert np.array_equal(a, b) and np.isfinite(a).all()
    with pytest.raises(spin.SpinError):
        weigh(q, lse, cache, table, starts([700]), [900], W(), workspace=ws[:need - 16])


def test_every_row_gives_a_weight_of_one_a_head():
    """With the logarithms that attention leaves.  Attention's logarithm is off by 2^-12 at most here (132 roundings of 2^-24
    of sums below 20, and its own), a weight by as much again."""
    rng = np.random.default_rng(1)
    for q_len, kv_len, Hq, Hkv, more in (([1] * 20, [3 + 111 * i for i in range(20)], 32, 8, {}), ([200, 64], [900, 64], 8, 2, {}),
                                         ([60, 1], [500, 4000], 4, 4, dict(softcap=30.0, window=300))):
        n = sum(-(-k // 16) for k in kv_len)
        cache, table = dev(pool(rng, n, Hkv, 16, 4)), tables(rng, kv_len, 16, n)
        q = dev(rng.standard_normal((sum(q_len), Hq, 128)).astype(np.float16))
        lse = torch.empty(q.shape[:2], device=DEV)
        args = (cache, dev(table), dev(starts(q_len)), dev(np.array(kv_len, np.int32)))
        spin.spin_kv_attn(q, *args, lse=lse, **more)
        W = host(spin.spin_kv_weights(q, lse, *args, **more)).astype(np.float64)
        for b, (m, k) in enumerate(zip(q_len, kv_len)):
            total = W[table[b, :-(-k // 16)]].sum((0, 2))
            assert np.abs(total - m * Hq // Hkv).max() <= 2.0 ** -11 * m * Hq / Hkv


def test_prior_may_be_the_weights_themselves():
    rng = np.random.default_rng(2)
    cache, table, q_start, kv_len = pool(rng, 30, 2, 16, 4), tables(rng, [200, 70], 16, 30), starts([1, 3]), [200, 70]
    q, lse = rng.standard_normal((4, 8, 128)).astype(np.float16), rng.uniform(3, 6, (4, 8)).astype(np.float32)
    W0 = rng.random((30, 2, 16)).astype(np.float32)
    apart = weigh(q, lse, cache, table, q_start, kv_len, dev(W0), prior=W0, decay=0.5)
    W = dev(W0)
    args = (dev(q), dev(lse), dev(cache), dev(table), dev(q_start), dev(np.array(kv_len, np.int32)))
    assert spin.spin_kv_weights(*args, prior=W, decay=0.5, W=W) is W
    assert np.array_equal(host(W), apart)
    fresh = host(spin.spin_kv_weights(*args))
    ref, _ = oracle.kv_weights(q, lse, cache, table, q_start, kv_len, 128 ** -0.5)
    assert (fresh[np.isnan(ref)] == 0).all() and (fresh[~np.isnan(ref)] > 0).any()


def test_no_rows_and_no_tokens():
    rng = np.random.default_rng(3)
    cache, table = pool(rng, 9, 2, 16, 4), tables(rng, [40, 0], 16, 9)
    q, lse = np.zeros((0, 4, 128), np.float16), np.zeros((0, 4), np.float32)
    prior = rng.random((9, 2, 16)).astype(np.float32)
    got = weigh(q, lse, cache, table, starts([0, 0]), [40, 0], torch.full((9, 2, 16), 77.0, device=DEV), prior, decay=0.5)
    ref, _ = oracle.kv_weights(q, lse, cache, table, starts([0, 0]), [40, 0], 1.0, prior=prior, decay=0.5)
    assert np.array_equal(got, np.where(np.isnan(ref), 77.0, ref))


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_numbers_that_are_not_finite(bad):
    """A row whose logarithm is not finite adds nothing, whatever it holds; a token whose scale is not finite draws nothing."""
    rng = np.random.default_rng(4)
    for more in ({}, dict(softcap=20.0), dict(softcap=1e3, alibi=True)):
        q_len, kv_len = [40, 1], [100, 300]
        cache, table = pool(rng, 40, 2, 16, 8), tables(rng, kv_len, 16, 40)
        cache["K_scale"][table[0, 2], 1, 3] = cache["K_scale"][table[1, 0], 0, 0] = bad
        cache["K_scale"][np.setdiff1d(np.arange(40), table)] = bad
        q = rng.standard_normal((41, 8, 128)).astype(np.float16)
        q[7, 2, 5] = q[30] = bad
        slopes = dict(slopes=(2.0 ** -np.arange(1, 9)).astype(np.float32)) if more.pop("alibi", False) else {}
        more.update(slopes)
        lse = rng.uniform(0, 5, (41, 8)).astype(np.float32)
        lse[7, 2] = lse[30] = bad
        lse[12, 4:] = bad
        prior = rng.random((40, 2, 16)).astype(np.float32)
        ref, bound = oracle.kv_weights(q, lse, cache, table, starts(q_len), kv_len, 128 ** -0.5, prior=prior, **more)
        got = weigh(q, lse, cache, table, starts(q_len), kv_len, torch.full((40, 2, 16), 77.0, device=DEV), prior, **more)
        written = ~np.isnan(ref)
        assert np.isfinite(got[written]).all() and (got[~written] == 77.0).all()
        assert (np.abs(got - ref)[written] <= bound[written]).all()
        assert got[table[0, 2], 1, 3] == prior[table[0, 2], 1, 3]


def test_attention_and_weights_of_a_batch_with_a_bad_row():
    """The logarithms as attention leaves them: a bad query or scale spoils no weight."""
    rng = np.random.default_rng(5)
    kv_len, q_len = [200, 90], [1, 30]
    cache, table = pool(rng, 30, 2, 16, 4), tables(rng, kv_len, 16, 30)
    cache["K_scale"][table[0, 5], 0, 1] = np.nan
    cache["V_scale"][table[1, 1], 1, 9] = np.inf
    q = rng.standard_normal((31, 8, 128)).astype(np.float16)
    q[9, 1] = np.inf
    q[10, 6, 3] = np.nan
    args = (dev(cache), dev(table), dev(starts(q_len)), dev(np.array(kv_len, np.int32)))
    lse = torch.empty((31, 8), device=DEV)
    spin.spin_kv_attn(dev(q), *args, lse=lse)
    logs = host(lse)
    assert not np.isfinite(logs[0, :4]).any() and np.isfinite(logs[0, 4:]).all()
    assert not np.isfinite(logs[9, 1]) and not np.isfinite(logs[10, 6])
    W = host(spin.spin_kv_weights(dev(q), lse, *args))
    assert np.isfinite(W).all() and (W[table[0, :12], 0] == 0).all() and (W[table[0, :12], 1] > 0).any()


def test_pages_that_are_not_there_and_lengths_past_the_table():
    rng = np.random.default_rng(6)
    table = tables(rng, [300, 80], 16, 30, extra=0)
    table[0, 3], table[1, 4] = -1, 1000
    for kv_len in ([300, 80], [2 ** 31 - 1, -3], [400, 90]):
        check(rng, [4, 20], kv_len, 4, 2, 4, 16, table=table, cache=pool(rng, 30, 2, 16, 4), exact_logs=False)


# ---------------------------------------------------------------------------------------------- the choice

def choose(W, table, kv_len, keep, first=0, recent=0):
    kept, lens = spin.spin_kv_choose(dev(W), dev(table), dev(np.asarray(kv_len, np.int32)), keep, first=first, recent=recent)
    ref, n = oracle.kv_choose(W, table, kv_len, keep, first, recent)
    assert np.array_equal(host(kept), ref) and np.array_equal(host(lens), n)
    return host(kept)


@pytest.mark.parametrize("kv_len,Hkv,page,keep,first,recent", [
    ([1], 1, 16, 1, 0, 0),
    ([0, 5, 6, 7], 2, 16, 6, 1, 2),
    ([100, 3, 64, 65], 3, 16, 1, 0, 0),
    ([100, 3, 64, 65], 3, 32, 64, 64, 0),
    ([100, 300, 64, 65], 2, 16, 64, 0, 64),
    ([1025, 1024, 1023, 2049], 2, 64, 1000, 4, 100),
    ([5000, 40, 20000], 4, 128, 2048, 16, 256),
    ([70000], 2, 1024, 69999, 1, 1),
    ([70000, 33000], 1, 64, 512, 0, 0),
    ([140000], 1, 64, 4096, 4, 64),
    ([9000, 10000, 300], 2, 16, 2048, 7, 9),                                        # 16 tokens a thread in the registers
    ([33000, 100, 8192, 8193, 40000, 0], 2, 64, 4000, 4, 1000),                     # several workgroups a head
    ([33000, 100, 8192, 8193, 40000, 0], 2, 64, 50000, 4, 1000),
    ([60000, 50], 1, 16, 20000, 9000, 11000),
    ([33000, 500] * 32, 4, 16, 4000, 4, 1000),                                      # more of each for a workgroup
    ([70000] + [500] * 30, 4, 64, 40000, 4, 1000),
    ([60000, 17000], 1, 16, 8193, 0, 0),
])
def test_choice(kv_len, Hkv, page, keep, first, recent):
    rng = np.random.default_rng(sum(kv_len))
    n = sum(-(-k // page) for k in kv_len) + 2
    table = tables(rng, kv_len, page, n)
    W = np.exp(3 * rng.standard_normal((n, Hkv, page))).astype(np.float32)
    choose(W, table, kv_len, keep, first, recent)
    choose(np.round(W), table, kv_len, keep, first, recent)                         # many ties
    choose(np.zeros_like(W), table, kv_len, keep, first, recent)                    # nothing else


def test_choice_of_any_numbers():
    rng = np.random.default_rng(1)
    table = tables(rng, [900, 500], 16, 100)
    W = rng.standard_normal((100, 2, 16)).astype(np.float32)
    W[rng.random(W.shape) < 0.2] = np.nan
    W[rng.random(W.shape) < 0.1] = np.inf
    W[rng.random(W.shape) < 0.1] = -np.inf
    W[rng.random(W.shape) < 0.1] = 0.0
    W[rng.random(W.shape) < 0.1] = -0.0
    W[rng.random(W.shape) < 0.1] *= 1e-42                                           # subnormal
    table[0, 7] = -1
    table[1, 3] = 100
    for keep in (1, 60, 333, 480, 499, 870, 899, 1000):
        choose(W, table, [900, 500], keep)
        choose(W, table, [900, 2 ** 31 - 1], keep, keep // 5, keep // 3)
        choose(W, table, [-9, 500], keep, 0, keep)
    W[:] = np.nan
    choose(W, table, [900, 500], 100, 3, 5)


@pytest.mark.parametrize("B", [300])
def test_choice_of_many_sequences(B):
    rng = np.random.default_rng(B)
    kv_len = rng.integers(0, 200, B)
    table = tables(rng, kv_len, 16, int((-(-kv_len // 16)).sum()) + 1)
    W = rng.random((int((-(-kv_len // 16)).sum()) + 1, 2, 16)).astype(np.float32)
    choose(W, table, kv_len, 50, 2, 10)


def test_choice_in_a_workspace_of_the_callers():
    rng = np.random.default_rng(3)
    table, W = tables(rng, [50000, 33000], 64, 1400), rng.random((1400, 2, 64)).astype(np.float32)
    kv = dev(np.array([50000, 33000], np.int32))
    need = spin.spin_kv_choose_workspace(2, 2, table.shape[1], 64)
    assert need > 0
    ref, _ = oracle.kv_choose(W, table, [50000, 33000], 3000, 10, 20)
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)
    for _ in range(2):
        kept, _ = spin.spin_kv_choose(dev(W), dev(table), kv, 3000, first=10, recent=20, workspace=ws)
        assert np.array_equal(host(kept), ref)
    with pytest.raises(spin.SpinError):
        spin.spin_kv_choose(dev(W), dev(table), kv, 3000, workspace=ws[:need - 16])


# ------------------------------------------------------------------------------------------------ the move

def move(cache, table, kept, at=None, to_table=None, W=None):
    c, w = dev(cache), dev(W)
    spin.spin_kv_move(c, dev(table), dev(kept), at=dev(at), to_table=dev(to_table), W=w)
    ref, w_ref = oracle.kv_move(cache, table, kept, at, to_table, W)
    for name in ref:
        assert np.array_equal(host(c[name]).view(np.uint8), ref[name].view(np.uint8)), name
    assert W is None or np.array_equal(host(w).view(np.uint32), w_ref.view(np.uint32))


def lists(rng, kv_len, heads, n, density=None):
    kept = np.full((len(kv_len), heads, n), -1, np.int32)
    for b, kv in enumerate(kv_len):
        for h in range(heads):
            m = min(n, kv)
            kept[b, h, :m] = np.sort(rng.permutation(kv)[:m])
    return kept


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("kv_len,Hkv,heads,page,n", [
    ([1], 1, 1, 16, 1),
    ([50, 0, 200], 2, 2, 16, 30),
    ([300, 64, 65, 63], 3, 1, 32, 64),
    ([700, 129], 2, 2, 64, 129),
    ([2000], 4, 4, 128, 1000),
    ([900, 20] * 20, 2, 2, 16, 200),
])
def test_move(bits, weights, kv_len, Hkv, heads, page, n):
    rng = np.random.default_rng(sum(kv_len) + bits)
    used = sum(-(-k // page) for k in kv_len)
    to = -(-n // page)
    pages = used + len(kv_len) * to + 2
    cache = pool(rng, pages, Hkv, page, bits)
    order = rng.permutation(pages)
    table = tables(rng, kv_len, page, used)
    table = np.where(table >= 0, order[table], -1).astype(np.int32)
    W = rng.standard_normal((pages, Hkv, page)).astype(np.float32) if weights else None
    kept = lists(rng, kv_len, heads, n)
    move(cache, table, kept, W=W)                                                   # to the front of their own pages
    to_table = order[used:used + len(kv_len) * to].reshape(len(kv_len), to).astype(np.int32)
    move(cache, table, kept, to_table=to_table, W=W)
    c = dev(cache)
    spin.spin_kv_move(c, dev(table), dev(kept), W=dev(W))
    again, same = dev(cache), dev(table)
    spin.spin_kv_move(again, same, dev(kept), to_table=same, W=dev(W))              # its own table: in place
    assert all(np.array_equal(host(c[k]).view(np.uint8), host(again[k]).view(np.uint8)) for k in c)
    shuffled = kept[:, :, rng.permutation(n)]                                       # any order into other pages
    move(cache, table, shuffled, to_table=to_table, W=W)


def test_accepted_paths():
    """Behind contexts of odd lengths, in place: paths of no, one and all tokens, entries that are passed over."""
    rng = np.random.default_rng(2)
    at, page = np.array([0, 5, 16, 33, 100, 63, 2], np.int32), 16
    table = tables(rng, at + 70, page, 80)
    cache, W = pool(rng, 80, 2, page, 4), rng.random((80, 2, 16)).astype(np.float32)
    kept = np.full((7, 1, 66), -1, np.int32)
    kept[1, 0, :1], kept[2, 0, :4], kept[3, 0, :66] = 69, [0, 2, 30, 66], np.arange(66)
    kept[4, 0, :5], kept[5, 0, :66], kept[6, 0, 0:9:2] = [0, 1, 2, 3, 69], np.arange(66) + 4, [1, 9, 10, 40, 41]
    move(cache, table, kept, at=at, W=W)
    move(cache, table, kept[:, :, :8].copy(), at=at)


def test_moves_from_and_to_nowhere():
    rng = np.random.default_rng(3)
    table = tables(rng, [200, 100], 16, 30)
    table[0, 2], table[1, 0] = -1, 30
    cache = pool(rng, 30, 2, 16, 8)
    kept = lists(rng, [200, 100], 2, 60)
    move(cache, table, kept)
    move(cache, table, kept, at=np.array([150, -20], np.int32))
    move(cache, table, np.minimum(kept * 4, 2 ** 31 - 1).astype(np.int32), at=np.array([0, 2 ** 31 - 1], np.int32))
    free = np.setdiff1d(np.arange(30), table)[:6].reshape(2, 3).astype(np.int32)
    free[0, 1], free[1, 2] = -1, 30
    move(cache, table, kept, to_table=free)
