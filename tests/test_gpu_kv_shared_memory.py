"""Tensors of one call in the same memory, where the calls for trees and eviction allow it."""

import numpy as np
import pytest
import torch

import oracle
from rotation_bit_quantization_amd import spin

from .paged_case import dev, host, pool, tables
from .test_gpu_kv_evict import lists

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spin.load()


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("kv,Hkv,page,n,first,at", [
    (3000, 2, 16, 1000, 63, 0),              # the list's tokens fit the first pages, whole chunks and a rest
    (3000, 4, 16, 1000, 20, 0),              # they do not: those beyond stay where they are
    (700, 1, 64, 129, 3, 7),
    (200, 3, 128, 64, 1, 0),
    (500, 300, 16, 65, 5, 0),                # keys and values together
])
def test_a_sequence_moves_to_its_own_first_pages(bits, kv, Hkv, page, n, first, at):
    """A row of the page table cut short begins at the same address, and names pages that tokens come from: in place."""
    rng = np.random.default_rng(kv + bits)
    used = -(-kv // page)
    cache, W = pool(rng, used + 1, Hkv, page, bits), rng.random((used + 1, Hkv, page)).astype(np.float32)
    table = tables(rng, [kv], page, used + 1)
    kept, start = lists(rng, [kv - at], Hkv, n), np.array([at], np.int32)
    ref, w_ref = oracle.kv_move(cache, table, kept, start, table[:, :first], W)
    pages = dev(table)
    for given, to in ((pages, pages[:, :first]), (pages[:, :used], pages)):
        c, w = dev(cache), dev(W)
        spin.spin_kv_move(c, given, dev(kept), at=dev(start), to_table=to, W=w)
        if to is pages:
            ref, w_ref = oracle.kv_move(cache, table[:, :used], kept, start, table, W)
        assert all(np.array_equal(host(c[k]).view(np.uint8), ref[k].view(np.uint8)) for k in ref)
        assert np.array_equal(host(w).view(np.uint32), w_ref.view(np.uint32))


@pytest.mark.parametrize("kv_len,Hkv,page,keep,room", [
    ([300, 20, 0, 64, 65], 8, 16, 64, 0),
    ([5000, 900, 2000] * 30, 16, 64, 500, 0),             # more workgroups than run at once
    ([9000, 3000], 64, 64, 700, 0),
    ([3000, 40, 8192, 20000], 16, 64, 1000, 40000),       # tables in parts
    ([10, 2 ** 31 - 1, -5] * 400, 2, 16, 12, 0),          # a second workgroup of lengths, lengths past the table
])
def test_lengths_are_replaced_by_those_that_stay(kv_len, Hkv, page, keep, room):
    """lens in kv_len's memory: every head reads a sequence's length before it changes."""
    rng = np.random.default_rng(keep)
    held = [min(max(k, 0), 20000) if k < 2 ** 31 - 1 else 30 for k in kv_len]
    n = sum(-(-k // page) for k in held) + 1
    table = tables(rng, held, page, n)
    table = np.pad(table, ((0, 0), (0, max(room // page - table.shape[1], 0))), constant_values=-1)
    W = rng.random((n, Hkv, page)).astype(np.float32)
    ref, lens_ref = oracle.kv_choose(W, table, kv_len, keep, 2, 5)
    kv = dev(np.array(kv_len, np.int32))
    kept, lens = spin.spin_kv_choose(dev(W), dev(table), kv, keep, first=2, recent=5, lens=kv)
    assert lens is kv and np.array_equal(host(kept), ref) and np.array_equal(host(kv), lens_ref)


def test_a_captured_loop_with_one_buffer_of_lengths():
    rng = np.random.default_rng(8)
    kv_len, keep = np.array([400, 31, 200], np.int32), 100
    table, W = tables(rng, kv_len, 16, 50), dev(rng.random((50, 4, 16)).astype(np.float32))
    kv, pages = dev(kv_len), dev(table)
    spin.spin_kv_choose(W, pages, kv, keep, lens=kv)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kept, _ = spin.spin_kv_choose(W, pages, kv, keep, lens=kv)
    for less in (0, 7, 300, 0):
        now = np.maximum(kv_len - less, 0).astype(np.int32)
        W.copy_(torch.roll(W, 1, 0))
        kv.copy_(torch.from_numpy(now))
        g.replay()
        ref, lens = oracle.kv_choose(host(W), table, now, keep)
        assert np.array_equal(host(kept), ref) and np.array_equal(host(kv), lens)
