"""GPU parity of the attention's scores at their ends: caps of every size against scores of every size, on every kernel.
Reference and bounds as in test_gpu_kv_attn.py: the float64 oracle, element by element, within the roundings that it
counts."""

import numpy as np
import pytest
import torch

from rotation_bit_quantization_amd import spin

from .test_gpu_kv_attn_tiles import WORK, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spin.load()


@pytest.mark.parametrize("work", [0] + WORK)
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("cap", [50.0, 64.0, 64.00001, 100.0, 1e3, 1e4, 1e6, 1e8, 1e30, 3e38])
def test_caps_of_every_size(cap, bits, work):
    """Scores of about -8 .. 8 whatever the cap: from some thousand on it changes nothing, and nothing may be lost."""
    rng = np.random.default_rng(bits)
    q_len, kv_len = ([1, 3], [300, 70]) if work == 0 else ([150, 9], [300, 30])
    check(rng, q_len, kv_len, 4, 2, bits, 16, work, softcap=cap)
    check(rng, q_len, kv_len, 4, 2, bits, 16, work, softcap=cap, alibi=True, window=90, bidir=True)


@pytest.mark.parametrize("work", [0] + WORK)
@pytest.mark.parametrize("cap", [60.0, 70.0, 200.0, 1e3])
@pytest.mark.parametrize("times", [0.05, 0.3, 1.0, 5.0, -1.0])
def test_scores_up_to_and_past_the_cap(cap, times, work):
    rng = np.random.default_rng(int(cap))
    check(rng, [2] if work == 0 else [140], [300], 4, 2, 8, 32, work, softcap=cap, scale=times * cap / 8 * 128 ** -0.5)


@pytest.mark.parametrize("work", [0] + WORK)
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("cap,scale", [(1e-20, 0.1), (1e-30, 0.1), (1e-38, -0.1), (1e-45, 0.1), (1e-45, 3e38), (5.0, 3e38),
                                       (100.0, -3e38), (3e38, 3e38), (0.0, 1e32), (0.0, 3e38), (0.0, -3e38)])
def test_caps_near_zero_and_scales_near_infinity(cap, scale, bits, work):
    """Scores of any size: queries of zeros weigh all tokens alike, others are finite."""
    rng = np.random.default_rng(bits)
    for loud in (0.0, 1.5):
        check(rng, [2, 1] if work == 0 else [140, 1], [300, 0], 4, 2, bits, 16, work, softcap=cap, scale=scale, loud=loud)
