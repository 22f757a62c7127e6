"""Batches on a paged KV cache for the tests: random pools, tables and lengths, on the host and on the GPU."""

import numpy as np
import torch

from rotation_bit_quantization_amd import spin

DEV = "cuda"


def pool(rng, n_pages, Hkv, page, bits, scales=(0.05, 0.5)):
    """A cache (numpy) of random codes and scales, every slot of it filled."""
    q = 7 if bits == 4 else 127
    codes = np.clip(np.rint(rng.standard_normal((2, n_pages, Hkv, page, 128)) * q / 2.7), -q, q).astype(np.int8)

    def raw(c):
        if bits == 8:
            return c.view(np.uint8)
        return ((c[..., 0::2] & 15) | ((c[..., 1::2] & 15) << 4)).astype(np.uint8)

    s = lambda: (rng.uniform(*scales, (n_pages, Hkv, page)) * 7 / q).astype(np.float16)  # noqa: E731
    v = raw(codes[1]).reshape(n_pages, Hkv, page // 4, 4, 16, bits).transpose(0, 1, 2, 4, 3, 5)
    return {"K_codes": raw(codes[0]), "K_scale": s(), "V_codes": np.ascontiguousarray(v), "V_scale": s()}


def tables(rng, kv_len, page, n_pages, extra=1, first=0):
    """Page tables of the sequences, their pages drawn without repetition from first .. n_pages - 1; -1 behind."""
    need = [-(-int(max(n, 0)) // page) for n in kv_len]
    width = max(need + [1]) + extra
    order = first + rng.permutation(n_pages - first)
    t = np.full((len(kv_len), width), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        t[b, :n] = order[at:at + n]
        at += n
    return t


def starts(q_len, before=0):
    return (before + np.concatenate([[0], np.cumsum(q_len)])).astype(np.int32)


def dev(a):
    if isinstance(a, dict):
        return {k: dev(v) for k, v in a.items()}
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def host(t):
    torch.cuda.synchronize()
    return t.cpu().numpy()


def attend(q, cache, table, q_start, kv_len, prefix_table=None, prefix_len=0, **more):
    """The framework's attention on host arrays; rows it does not write hold 77."""
    O = torch.full(q.shape, 77.0, dtype=torch.float16, device=DEV)
    more = {k: dev(v) if isinstance(v, np.ndarray) else v for k, v in more.items()}
    args = (dev(table), dev(np.asarray(q_start, np.int32)), dev(np.asarray(kv_len, np.int32)))
    if prefix_table is not None:
        spin.spin_kv_attn_shared(dev(q), dev(cache), dev(prefix_table), prefix_len, *args, O=O, **more)
    else:
        spin.spin_kv_attn(dev(q), dev(cache), *args, O=O, **more)
    return host(O).astype(np.float64)


def close(got, ref, bound):
    """Rows that are not written hold 77, rows that see a scale that is not finite hold NaN, the others are within
    the bound."""
    silent, bad = np.isnan(ref), np.isinf(ref)
    assert (got[silent] == 77.0).all()
    assert np.isnan(got[bad]).all()
    # 65520 lies half a step above the largest fp16, 65504: an exact value from there on rounds to infinity, and one
    # within the bound of 65520 may fall on either side
    big = ~silent & ~bad & (np.abs(np.where(bad, 0, ref)) + bound >= 65520)
    over = big & ~np.isfinite(got)
    assert (got[over] == np.sign(ref[over]) * np.inf).all()
    assert (np.abs(ref[big & ~over]) - bound[big & ~over] < 65520).all()
    fine = ~silent & ~bad & ~over
    off = np.abs(got - ref)[fine]
    assert np.isfinite(got[fine]).all()
    worst = (off - bound[fine]).max() if off.size else 0.0
    assert worst <= 0.0, (worst, off.max(), np.unravel_index(np.argmax(np.where(fine, np.abs(got - ref) - bound, -1)), got.shape))
