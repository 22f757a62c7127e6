"""Weights that are added up from step to step: tokens that are new have no prior, whatever their slots held before."""

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


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("q_len,kv_len,known,Hq,Hkv,page", [
    ([1, 1, 1, 1], [300, 65, 1, 64], [299, 64, 0, 64], 8, 2, 16),                # single tokens
    ([3, 1], [700, 20], [0, 19], 4, 4, 64),
    ([1] * 300, [1 + 2 * i for i in range(300)], [2 * i for i in range(300)], 4, 2, 16),
    ([40, 90, 0], [200, 90, 50], [160, 0, 30], 8, 2, 32),                        # tiles
    ([700], [2300], [1600], 6, 2, 64),                                           # shares of the rows
    ([50, 60], [400, 500], [-5, 2 ** 31 - 1], 8, 1, 16),                         # none, all
])
@pytest.mark.parametrize("more", [{}, dict(softcap=20.0, window=50)])
def test_tokens_without_a_prior(q_len, kv_len, known, Hq, Hkv, bits, page, more):
    rng = np.random.default_rng(Hq + page)
    n = sum(-(-k // page) for k in kv_len) + 1
    cache, table, T = pool(rng, n, Hkv, page, bits), tables(rng, kv_len, page, n), sum(q_len)
    q, lse = rng.standard_normal((T, Hq, 128)).astype(np.float16), rng.uniform(0, 5, (T, Hq)).astype(np.float32)
    prior = rng.random((n, Hkv, page)).astype(np.float32)
    for b, (k, m) in enumerate(zip(kv_len, known)):                              # what is behind is not read
        for j in range(max(m, 0), k):
            prior[table[b, j // page], :, j % page] = np.nan
    ref, bound = oracle.kv_weights(q, lse, cache, table, starts(q_len), kv_len, 128 ** -0.5, prior=prior, decay=0.75, prior_len=known, **more)
    args = (dev(q), dev(lse), dev(cache), dev(table), dev(starts(q_len)), dev(np.array(kv_len, np.int32)))
    written = ~np.isnan(ref)
    for alias in (False, True):
        old = dev(prior)
        W = old if alias else torch.full((n, Hkv, page), 77.0, device=DEV)
        spin.spin_kv_weights(*args, prior=old, decay=0.75, W=W, prior_len=dev(np.array(known, np.int32)), **more)
        got = host(W).astype(np.float64)
        assert (np.abs(got - ref)[written] <= bound[written]).all()
        assert alias or (got[~written] == 77.0).all()


def test_a_loop_that_evicts():
    """Prompts, then tokens one by one, thinned every few steps; one sequence ends and another takes its pages.  Every step's
    sums against the oracle's, where a token starts at 0 when it comes."""
    rng = np.random.default_rng(5)
    B, Hq, Hkv, page, bits, keep, most = 3, 8, 2, 16, 4, 48, 64
    width = 8
    n_pages = B * width
    table = rng.permutation(n_pages).reshape(B, width).astype(np.int32)
    cache, pages = dev(pool(rng, n_pages, Hkv, page, bits)), dev(table)
    W = torch.full((n_pages, Hkv, page), 1e6, device=DEV)                         # sums of sequences that are gone
    ref = np.zeros((B, Hkv, width * page))                                        # by place
    held, weighed = np.zeros(B, np.int32), np.zeros(B, np.int32)
    q_len = np.array([100, 7, 63])
    for step in range(14):
        if step == 9:                                                             # sequence 1 ends, another begins in its pages
            held[1] = weighed[1] = 0
            q_len = np.array([1, 30, 1])
        kv = (held + q_len).astype(np.int32)
        T = int(q_len.sum())
        x = dev(rng.standard_normal((T, Hq + 2 * Hkv, 128)).astype(np.float16))
        batch = (cache, pages, dev(starts(q_len)), dev(kv))
        Q = spin.spin_kv_append(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], *batch)
        lse = torch.empty((T, Hq), device=DEV)
        spin.spin_kv_attn(Q, *batch, lse=lse)
        spin.spin_kv_weights(Q, lse, *batch, prior=W, prior_len=dev(weighed), decay=0.9, W=W)
        add, off = oracle.kv_weights(host(Q), host(lse), {k: host(t) for k, t in cache.items()}, table, starts(q_len), kv, 128 ** -0.5)
        got = host(W).astype(np.float64)
        for b in range(B):
            n, j = kv[b], np.arange(kv[b])
            at = table[b, j // page]
            ref[b, :, held[b]:] = 0.0                                             # the new ones, and places behind
            ref[b, :, :n] = 0.9 * ref[b, :, :n] + add[at, :, j % page].T
            # this step's bound and two roundings of the sum; what earlier steps were off by is taken over below
            assert (np.abs(got[at, :, j % page].T - ref[b, :, :n]) <= off[at, :, j % page].T + 2.0 ** -22 * ref[b, :, :n]).all(), (step, b)
            ref[b, :, :n] = got[at, :, j % page].T
        weighed = kv
        if (kv > most).any():
            kept, lens = spin.spin_kv_choose(W, pages, dev(kv), keep, first=2, recent=8)
            spin.spin_kv_move(cache, pages, kept, W=W)
            kept, weighed = host(kept), host(lens)
            for b in range(B):
                order = [np.lexsort((np.arange(kv[b]), -np.where((np.arange(kv[b]) < 2) | (np.arange(kv[b]) >= kv[b] - 8), np.inf, ref[b, h, :kv[b]])))
                         for h in range(Hkv)]
                for h in range(Hkv):
                    stay = np.sort(order[h][:min(keep, kv[b])])
                    assert np.array_equal(kept[b, h, :weighed[b]], stay), (step, b, h)
                    ref[b, h, :len(stay)] = ref[b, h, stay]
        held, q_len = weighed.copy(), np.ones(B, np.int64)
