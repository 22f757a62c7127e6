"""Attention's logarithms and the weights taken with them, token by token against the float64 oracle alone."""

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
@pytest.mark.parametrize("q_len,kv_len,Hq,Hkv,more", [
    ([1] * 5, [1, 16, 300, 65, 900], 8, 2, {}),                        # single tokens
    ([1, 3], [4000, 20], 4, 4, dict(softcap=30.0)),                    # shares of the tokens, joined
    ([40, 1, 9], [200, 64, 90], 16, 2, dict(window=50)),
    ([300], [1100], 8, 1, {}),                                         # tiles
    ([300, 70], [300, 700], 4, 2, dict(softcap=90.0)),
])
def test_weights_by_attentions_logarithms(bits, q_len, kv_len, Hq, Hkv, more):
    """A weight is off by what the oracle counts for it and, of itself, by what it counts for the logarithm of its rows."""
    rng = np.random.default_rng(Hq + bits)
    n = sum(-(-k // 16) for k in kv_len)
    cache, table = pool(rng, n, Hkv, 16, bits), tables(rng, kv_len, 16, n)
    q = (2 * rng.standard_normal((sum(q_len), Hq, 128))).astype(np.float16)
    _, _, logs, off = oracle.kv_attend(q, cache, table, starts(q_len), kv_len, 128 ** -0.5, sums=True, **more)
    ref, bound = oracle.kv_weights(q, logs, cache, table, starts(q_len), kv_len, 128 ** -0.5, **more)
    lse = torch.empty(q.shape[:2], device=DEV)
    args = (dev(cache), dev(table), dev(starts(q_len)), dev(np.array(kv_len, np.int32)))
    spin.spin_kv_attn(dev(q), *args, lse=lse, **more)
    assert (np.abs(host(lse) - logs) <= off).all()
    got = host(spin.spin_kv_weights(dev(q), lse, *args, **more)).astype(np.float64)
    for b, (k, m) in enumerate(zip(kv_len, q_len)):
        at, slot = table[b, np.arange(k) // 16], np.arange(k) % 16
        rows = off[starts(q_len)[b]:starts(q_len)[b] + m].reshape(m, Hkv, -1).max((0, 2))
        # e^x - 1 is below 1.001 x at logarithms off by 2^-10 at most
        allowed = bound[at, :, slot] + 1.001 * rows * ref[at, :, slot]
        assert rows.max() < 2.0 ** -10 and (np.abs(got[at, :, slot] - ref[at, :, slot]) <= allowed).all()
