"""The paged cache's calls on the paths between kernels: scales that are not finite behind a prefix, captured calls of two
launches, borders that do not ascend on tiles of 16 rows and in the append.  Reference and bounds as in
test_gpu_kv_attn.py."""

import numpy as np
import pytest
import torch

import oracle
from rotation_bit_quantization_amd import spin

from .paged_case import DEV, attend, close, dev, host, pool, starts, tables
from .test_gpu_kv_attn_tiles import check, widened

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spin.load()


# q_len, kv_len, Hq, Hkv, prefix, the own tokens' room as rows x tokens x key heads
PLANS = {
    "16 rows, one launch": ([2, 1, 9], [3, 17, 60], 8, 2, 300, 0),
    "prefix on 128 rows, joined by the own part": ([1] * 128, [1 + i % 37 for i in range(128)], 16, 2, 16500, 0),
    "prefix on 256 rows, joined by the own part": ([120, 130, 6], [125, 130, 6], 32, 2, 16500, 0),
    "both on 128 rows": ([40, 35, 70], [40, 60, 70], 16, 2, 16000, 2 ** 25),
    "prefix on 16 rows, own on 128": ([70, 80], [70, 95], 8, 2, 40, 2 ** 25),
    "prefix on 16 rows, own on 256": ([70, 80], [70, 95], 8, 2, 40, 2 ** 28),
}


@pytest.mark.parametrize("plan", sorted(PLANS))
@pytest.mark.parametrize("which,bad,bits", [("K_scale", np.nan, 4), ("K_scale", np.inf, 8), ("V_scale", np.nan, 8),
                                            ("V_scale", np.inf, 4), ("V_scale", -np.inf, 8)])
def test_scales_that_are_not_finite_behind_a_prefix(plan, which, bad, bits):
    q_len, kv_len, Hq, Hkv, prefix, work = PLANS[plan]
    rng = np.random.default_rng(8)
    page, first, G = 64, -(-prefix // 64), Hq // Hkv
    n = first + sum(-(-k // page) for k in kv_len) + 2
    cache = pool(rng, n, Hkv, page, bits)
    table = tables(rng, kv_len, page, n, first=first)
    for b, k in enumerate(kv_len):                                          # behind each sequence's last token
        if k % page:
            cache[which][table[b, k // page], :, k % page:] = bad
    cache[which][np.setdiff1d(np.arange(first, n), table)] = bad            # pages of no sequence
    go = lambda **more: check(rng, q_len, kv_len, Hq, Hkv, bits, page, work, cache=cache, table=table, prefix_len=prefix,  # noqa: E731
                              before=1, behind=1, most=2, **more)
    assert np.isfinite(go()[1:-1]).all()
    cache[which][table[1, 0], Hkv - 1, 0] = bad                             # the second sequence's first token, one head
    got = go()
    at = 1 + q_len[0]
    assert np.isnan(got[at:at + q_len[1], Hq - G:]).all() and np.isfinite(got[at:at + q_len[1], :Hq - G]).all()
    assert np.isfinite(np.delete(got[1:-1], np.arange(q_len[0], q_len[0] + q_len[1]), axis=0)).all()
    cache[which][0, 0, 5] = bad                                             # a token of the prefix, one head
    got = go(softcap=20.0, alibi=True)
    assert np.isnan(got[1:-1, :G]).all() and np.isfinite(got[1:at, G:]).all()
    go(window=kv_len[0] + 20)                                               # sees it or not, by the place of that page


@pytest.mark.parametrize("plan", ["prefix on 128 rows, joined by the own part", "prefix on 256 rows, joined by the own part",
                                  "prefix on 16 rows, own on 128", "both on 128 rows"])
def test_captured_calls_of_two_launches(plan):
    """Replayed in turn with eager calls, with other lengths each time; of the second graph the workspace is the
    caller's."""
    q_len, kv_len, Hq, Hkv, prefix, work = PLANS[plan]
    rng = np.random.default_rng(9)
    page, first, T = 64, -(-prefix // 64), sum(q_len)
    n = first + sum(-(-k // page) for k in kv_len)
    cache = dev(pool(rng, n, Hkv, page, 4))
    table = dev(widened(tables(rng, kv_len, page, n, first=first), T * Hq // Hkv, Hkv, page, work))
    front, q = dev(np.arange(first, dtype=np.int32)), dev(rng.standard_normal((T, Hq, 128)).astype(np.float16))
    q_start, kv = dev(starts(q_len)), dev(np.array(kv_len, np.int32))
    need = spin.spin_kv_attn_workspace(T, Hq, Hkv, len(q_len), table.shape[1], page, prefix)
    assert need > 0
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)           # NaN wherever it is read unwritten
    O = torch.zeros_like(q)
    call = lambda **more: spin.spin_kv_attn_shared(q, cache, front, prefix, table, q_start, kv, O=O, **more)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graphs = []
    for more in ({}, dict(workspace=ws)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(**more)
        graphs.append(g)
    seen = []
    for rep, less in enumerate([0, 5, 1000, 1, 0]):
        kv.copy_(torch.tensor([max(k - less, 0) for k in kv_len], dtype=torch.int32))
        want = host(call()).copy()
        assert np.isfinite(want).all()
        seen.append(want)
        for g in graphs:
            O.fill_(5.0)
            g.replay()
            assert np.array_equal(host(O), want), rep
    assert np.array_equal(seen[0], seen[-1]) and not np.array_equal(seen[0], seen[1])


@pytest.mark.parametrize("plan", sorted(PLANS))
@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_queries_that_are_not_finite(plan, bad):
    """Such a row is NaN or zero; of its token's others each is within its bound, and those of other tokens are those of the
    call without it, up to the bounds of both.  Not to the bit: rows of a wave move their maxima together, and a weight's
    rounding goes by where its row's maximum stands.  Of values up to v a bound is at most twice (2^-11 + e) v, with e
    below 2^-12 for the exponents here (132 roundings of 2^-24 of sums of 12): 2^-8 v for two."""
    q_len, kv_len, Hq, Hkv, prefix, work = PLANS[plan]
    rng = np.random.default_rng(10)
    page, first, T = 64, -(-prefix // 64), sum(q_len)
    n = first + sum(-(-k // page) for k in kv_len)
    cache, q = pool(rng, n, Hkv, page, 4), rng.standard_normal((T, Hq, 128)).astype(np.float16)
    table = widened(tables(rng, kv_len, page, n, first=first), T * Hq // Hkv, Hkv, page, work)
    args = (cache, table, starts(q_len), kv_len, np.arange(max(first, 1), dtype=np.int32), prefix)
    for more in (dict(), dict(softcap=20.0), dict(softcap=1e4, window=50)):
        want = attend(q, *args, **more)
        odd = q.copy()
        rows = [(0, 0), (T - 1, Hq - 1), (T // 2, 1)]
        tokens = sorted({t for t, _ in rows})
        ref, bound = oracle.kv_attend(q, cache, table, starts(q_len), kv_len, 128 ** -0.5, prefix_table=args[4],
                                      prefix_len=prefix, rows=set(tokens), **more)
        for i, (t, h) in enumerate(rows):
            odd[t, h, 5 + 40 * i] = bad
        got = attend(odd, *args, **more)
        for t, h in rows:
            assert (np.isnan(got[t, h]) | (got[t, h] == 0)).all()
            got[t, h] = want[t, h]
        close(got[tokens], ref[tokens], bound[tokens])
        assert np.abs(got - want).max() <= 2.0 ** -8 * 7 * float(cache["V_scale"].max())


@pytest.mark.parametrize("plan", sorted(PLANS))
@pytest.mark.parametrize("missing", ["some", "all"])
def test_pages_of_a_prefix_that_are_not_there(plan, missing):
    q_len, kv_len, Hq, Hkv, prefix, work = PLANS[plan]
    rng = np.random.default_rng(11)
    page, first, T = 64, -(-prefix // 64), sum(q_len)
    n = first + sum(-(-k // page) for k in kv_len)
    cache, q = pool(rng, n, Hkv, page, 8), rng.standard_normal((T, Hq, 128)).astype(np.float16)
    table = widened(tables(rng, kv_len, page, n, first=first), T * Hq // Hkv, Hkv, page, work)
    front = rng.permutation(first).astype(np.int32)
    front[rng.random(first) < (0.4 if missing == "some" else 2)] = -1
    front[0], front[first // 2] = n, -2 ** 31
    rows = {0, T // 2, T - 1}
    for more in (dict(), dict(window=prefix + 3)):
        ref, bound = oracle.kv_attend(q, cache, table, starts(q_len), kv_len, 0.1, prefix_table=front, prefix_len=prefix, rows=rows, **more)
        got = attend(q, cache, table, starts(q_len), kv_len, front, prefix, scale=0.1, **more)
        close(got[sorted(rows)], ref[sorted(rows)], bound[sorted(rows)])


def borders(kind, B, T):
    rng = np.random.default_rng(B)
    return {"wild": np.resize([0, 2 ** 31 - 1, -2 ** 31, 90], B + 1), "falling": np.linspace(T, 0, B + 1),
            "to and fro": np.resize([0, T, 0, T // 2], B + 1), "equal": np.full(B + 1, 5),
            "all rows in the last": np.append(np.full(B, -2 ** 31), 2 ** 31 - 1), "beyond": T + 100 * np.arange(B + 1),
            "random": rng.integers(-2 * T, 3 * T, B + 1)}[kind].astype(np.int32)


KINDS = ["wild", "falling", "to and fro", "equal", "all rows in the last", "beyond", "random"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("B,T,Hkv,room,prefix", [
    (3, 100, 1, 128, 0), (3, 100, 1, 128, 40), (12, 100, 2, 2560, 0), (64, 90, 1, 4096, 0), (100, 100, 1, 128, 0), (100, 100, 1, 128, 40),
    (300, 100, 1, 128, 0), (300, 400, 2, 64, 70), (128, 128, 4, 64, 16500)])
def test_borders_that_do_not_ascend_on_tiles_of_16_rows(kind, B, T, Hkv, room, prefix):
    """What such a call writes is not defined; it writes rows of O and its workspace only."""
    rng = np.random.default_rng(16)
    page, first = 64, -(-prefix // 64)
    n = first + 9
    cache = dev(pool(rng, n, Hkv, page, 4))
    before = {k: v.clone() for k, v in cache.items()}
    table = dev(rng.integers(-1, n + 1, (B, room // page)).astype(np.int32))
    kv = dev(rng.integers(-5, room + 9, B).astype(np.int32))
    q = dev(rng.standard_normal((T, 4 * Hkv, 128)).astype(np.float16))
    guard = torch.full((3, T, 4 * Hkv, 128), 77.0, dtype=torch.float16, device=DEV)
    need = spin.spin_kv_attn_workspace(T, 4 * Hkv, Hkv, B, room // page, page, prefix)
    ws = torch.full((need + 8192,), 171, dtype=torch.uint8, device=DEV)
    args = (table, dev(borders(kind, B, T)), kv)
    more = dict(O=guard[1], workspace=ws[4096:4096 + need])
    if prefix:
        spin.spin_kv_attn_shared(q, cache, dev(np.arange(first, dtype=np.int32)), prefix, *args, **more)
    else:
        spin.spin_kv_attn(q, cache, *args, **more)
    assert (host(guard[::2]) == 77.0).all()
    assert (host(ws[:4096]) == 171).all() and (host(ws[4096 + need:]) == 171).all()
    assert all(torch.equal(cache[k].view(torch.uint8), before[k].view(torch.uint8)) for k in cache)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("B,T,bits,queries", [(3, 100, 4, True), (17, 60, 8, True), (300, 700, 4, True), (300, 700, 8, False)])
def test_borders_that_do_not_ascend_in_the_append(kind, B, T, bits, queries):
    """It writes slots of the pool and rows of Q_out only."""
    rng = np.random.default_rng(17)
    Hq, Hkv, page, n, room = 8, 4, 16, 40, 48
    whole = {k: dev(v) for k, v in pool(rng, n + 2, Hkv, page, bits).items()}
    before = {k: v.clone() for k, v in whole.items()}
    cache = {k: v[1:-1] for k, v in whole.items()}
    table = dev(rng.integers(-1, n + 1, (B, room // page)).astype(np.int32))
    kv = dev(rng.integers(-5, room + 9, B).astype(np.int32))
    x = dev(rng.standard_normal((T, Hq + 2 * Hkv, 128)).astype(np.float16))
    q, k, v = x.split([Hq, Hkv, Hkv], dim=1)
    guard = torch.full((3, T, Hq, 128), 77.0, dtype=torch.float16, device=DEV)
    rope = spin.spin_rope_table(dev(1e4 ** (-np.arange(32) / 32)), 40)
    spin.spin_kv_append(q if queries else None, k, v, cache, table, dev(borders(kind, B, T)), kv, rope=rope,
                        Q_out=guard[1] if queries else None)
    assert (host(guard[::2]) == 77.0).all()
    for name in whole:
        assert all(torch.equal(whole[name][i].view(torch.uint8), before[name][i].view(torch.uint8)) for i in (0, -1)), name
