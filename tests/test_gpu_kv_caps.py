"""Capped weights, one product a score, so that nothing but the cap and the exponential rounds: as exact as fp32 weights
without a cap are, at scores small beside the cap too."""

import numpy as np
import pytest
import torch

from rotation_bit_quantization_amd import spin

from .paged_case import dev, host, pool, starts, tables

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spin.load()


def bound(z, cap):
    """How far e^(cap tanh(z / cap)) may be off, of itself, in counted roundings.

    Below 0.7 of the cap: the score in units of log2 1.7 U (the constant, a product), its ratio to the cap 5.4 U (the same, the
    cap's constant and product, a reciprocal, a product), of which the polynomial takes 0.27, its own fit and sums 1.5 U, the
    last multiply-add 1 U: 6 U of the capped score, held to 8.  Above: ten roundings of the cap's size, the score's 1.7 U at a
    slope below 0.46 and the last one, 13 U of the cap.  The exponential a unit in the last place, 2 U, held to 4."""
    z = np.abs(z)
    return np.where(z < 0.7 * cap, 8 * U * cap * np.tanh(z / cap), 13 * U * cap) + 4 * U


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("cap", [5.0, 20.0, 30.0, 50.0, 64.0, 65.0, 1e3, 1e5])
@pytest.mark.parametrize("rows,batch", [(1, 3), (2, 3), (4, 3), (16, 2), (40, 1), (300, 1)])     # 4, 8, 16 rows at a time, tiles, shares
@pytest.mark.parametrize("biased", [False, True])
def test_scores_of_one_product(bits, cap, rows, batch, biased):
    """Of each sequence's rows all but one have no logarithm, and add nothing; that one's query has one value."""
    rng = np.random.default_rng(rows + bits)
    n, page, H = 20, 64, 2
    kv_len = [1000 // batch] * batch
    cache, table = pool(rng, n, H, page, bits), tables(rng, kv_len, page, n)
    cache["K_scale"][:] = 2.0 ** rng.integers(-10, -2, (n, H, page)) * (16 if bits == 4 else 1)
    T = rows * batch
    q, lse = np.zeros((T, H, 128), np.float16), np.full((T, H), np.inf, np.float32)
    z, at = np.zeros((batch, H, kv_len[0])), np.arange(kv_len[0])
    for b in range(batch):
        for h in range(H):
            t, d = b * rows + rows - 1, int(rng.integers(128))
            q[t, h, d], lse[t, h] = rng.uniform(1, 4) * rng.choice([-1, 1]), 0.0
            raw = cache["K_codes"][table[b, at // page], h, at % page]
            if bits == 4:
                code = ((raw[:, d // 2] >> (4 * (d % 2))) & 15).astype(np.int64)
                code -= 16 * (code > 7)
            else:
                code = raw[:, d].view(np.int8).astype(np.int64)
            z[b, h] = float(q[t, h, d]) * code * cache["K_scale"][table[b, at // page], h, at % page].astype(np.float64)
    slopes = dict(slopes=dev(np.zeros(H, np.float32))) if biased else {}
    W = host(spin.spin_kv_weights(dev(q), dev(lse), dev(cache), dev(table), dev(starts([rows] * batch)), dev(np.array(kv_len, np.int32)),
                                  scale=1.0, softcap=cap, **slopes)).astype(np.float64)
    assert np.abs(z).max() > 20 and (np.abs(z) < 0.3).sum() > 10
    for b in range(batch):
        got = W[table[b, at // page], :, at % page].T
        ref = np.exp(cap * np.tanh(z[b] / cap))
        assert (np.abs(got - ref) <= ref * bound(z[b], cap)).all(), (np.abs(got / ref - 1) / bound(z[b], cap)).max()
