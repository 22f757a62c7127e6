"""Sums of weights over many rows of one sequence, whatever the rest of the batch makes the kernel: as exact as for few."""

import numpy as np
import pytest
import torch

from rotation_bit_quantization_amd import spin

from .paged_case import dev, host, pool, starts, tables

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spin.load()


# One long prompt among single tokens, rows on the mean 16.6 (16 at a time), 6 (8), 3.5 (4) and 300 (tiles of 32).
@pytest.mark.parametrize("singles,prompt", [(255, 4000), (599, 3000), (1199, 3000), (9, 3000)])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("more", [dict(), dict(softcap=30.0, slopes=0.0), dict(slopes=0.0), dict(window=700), dict(causal=False), dict(both=1000)])
def test_a_long_prompt_among_single_tokens(singles, prompt, bits, more):
    """Queries of zeros: every row that sees a token gives it e^-lse, here a third.

    That is off by 2^-23 of itself for the exponential and 2.2 x 2^-24 for the logarithm in units of log2; rows of one step
    are added in up to 15 additions of 2^-24 (four, one behind the other, in a lane; a tile's 16 as four of four, and two),
    the steps with what each has lost, 2^-23, and the lanes in three: 2^-19 covers them.  Added plainly, the 750 to 1000 steps
    of a lane are off by 2^-24 of the sum each, to one side."""
    more, rng = dict(more), np.random.default_rng(prompt)
    q_len, kv_len = [1] * singles + [prompt], [16] * singles + [prompt + 500]
    q_len[singles // 2], q_len[-1] = q_len[-1], q_len[singles // 2]
    kv_len[singles // 2], kv_len[-1] = kv_len[-1], kv_len[singles // 2]
    n, T, both = singles + -(-(prompt + 500) // 64), sum(q_len), more.pop("both", 0)
    cache, table = pool(rng, n, 1, 64, bits), tables(rng, kv_len, 64, n)
    if "slopes" in more:
        more["slopes"] = dev(np.zeros(1, np.float32))
    if both:
        more["bidir_len"] = dev(np.full(singles + 1, both, np.int32))
    lse = np.full((T, 1), np.log(3.0), np.float32)
    W = host(spin.spin_kv_weights(dev(np.zeros((T, 1, 128), np.float16)), dev(lse), dev(cache), dev(table), dev(starts(q_len)),
                                  dev(np.array(kv_len, np.int32)), **more)).astype(np.float64)
    b, j = singles // 2, np.arange(prompt + 500)
    p = np.arange(500, prompt + 500)[:, None]
    seen = np.ones((prompt, prompt + 500), bool)
    if more.get("causal", True):
        seen &= (j <= p) | (j < both)
    if "window" in more:
        seen &= np.abs(p - j) < more["window"]
    ref = seen.sum(0) * np.exp(-float(lse[0, 0]))
    got = W[table[b, j // 64], 0, j % 64]
    assert ref.max() > 200 and (np.abs(got - ref) <= 2.0 ** -19 * ref).all(), np.abs(got / np.maximum(ref, 1e-9) - 1).max()
    first = W[table[0, 0], 0, :16]
    assert (np.abs(first - np.exp(-float(lse[0, 0]))) <= 2.0 ** -21).all()
