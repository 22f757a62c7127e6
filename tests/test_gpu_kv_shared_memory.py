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
