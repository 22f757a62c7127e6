"""The paged KV cache: position rotation, append and attention (oracle; test infrastructure).

Everything is float64 from the inputs on; codes are decided by
``quant.quantize_kv_groups`` on the float32 rounding of the exact value, as
everywhere.  Layouts (this library's reading; the pages fix none):

  K_codes  uint8 [pages][H][page][16 * bits]          a token's codes in order
  V_codes  uint8 [pages][H][page / 4][16][4][bits]    octets of four tokens beside each other
  scales   fp16  [pages][H][page]

Sequence b owns query rows q_start[b] .. q_start[b + 1] - 1, its i-th row stands
at place kv_len[b] - q_len + i of its table, whose place p lies in slot p % page
of page table[b][p // page]; places past the table have no page.
"""

import numpy as np

from .hadamard import rotate_rows
from .quant import pack_int4, quantize_kv_groups, unpack_int4

__all__ = ["rope_table", "turn_heads", "kv_append", "kv_attend", "cache_tokens"]

D = 128


def rope_table(inv_freq, P, pos0=0, scale=1.0):
    """[P, 2 n] float64: cosines, then sines, of (pos0 + p) * inv_freq."""
    a = np.arange(pos0, pos0 + P, dtype=np.float64)[:, None] * np.asarray(inv_freq, np.float64)[None]
    return np.concatenate([np.cos(a), np.sin(a)], axis=1) * scale


def turn_heads(x, rows=None, interleaved=False, weight=None, eps=0.0):
    """x [N, H, 128] -> float64: norm per head, rotation by ``rows`` [N, rot] (cos | sin), H_128 / sqrt(128)."""
    y = np.asarray(x, np.float64).copy()
    if weight is not None:
        y = y / np.sqrt(np.mean(y * y, axis=-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    if rows is not None:
        n = rows.shape[1] // 2
        for i in range(n):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
            c, s = np.asarray(rows[:, None, i], np.float64), np.asarray(rows[:, None, n + i], np.float64)
            u, v = y[..., a].copy(), y[..., b].copy()
            y[..., a], y[..., b] = u * c - v * s, v * c + u * s
    return rotate_rows(y, D)


def _length(n):
    """A sequence's length as its tokens' places go by it, past its table or not."""
    return min(max(int(n), 0), 1 << 30)


def _places(q_start, kv_len, T):
    """[(row, sequence, place)] of the rows that belong to a sequence."""
    for b in range(len(kv_len)):
        for t in range(q_start[b], min(q_start[b + 1], T)):
            yield t, b, _length(kv_len[b]) - int(q_start[b + 1]) + t


def kv_append(q, k, v, cache, table, q_start, kv_len, rope=None, interleaved=False, q_norm=None, k_norm=None, eps=1e-6,
              pos0=0):
    """The cache (a dict of numpy arrays, a changed copy) and the queries in float64 (NaN rows: not written)."""
    cache = {name: a.copy() for name, a in cache.items()}
    pages, H, page, width = cache["K_codes"].shape
    bits = width // 16
    T = k.shape[0]
    q_out = np.full(q.shape, np.nan)
    for t, b, p in _places(q_start, kv_len, T):
        if p < 0 or p >= table.shape[1] * page or (rope is not None and p + pos0 >= len(rope)):
            q_out[t] = 0.0
            continue
        row = None if rope is None else rope[p + pos0][None]
        q_out[t] = turn_heads(q[t:t + 1], row, interleaved, q_norm, eps)[0]
        at = table[b, p // page]
        if at < 0 or at >= pages:
            continue
        slot = p % page
        for name, y in (("K", turn_heads(k[t:t + 1], row, interleaved, k_norm, eps)[0]), ("V", v[t].astype(np.float64))):
            codes, scale = quantize_kv_groups(y.astype(np.float32)[None], 7 if bits == 4 else 127)
            raw = (pack_int4(codes[0]) if bits == 4 else codes[0].view(np.uint8)).reshape(H, 16, bits)
            if name == "K":
                cache["K_codes"][at, :, slot] = raw.reshape(H, width)
            else:
                cache["V_codes"][at, :, slot // 4, :, slot % 4] = raw
            cache[name + "_scale"][at, :, slot] = scale[0]
    return cache, q_out


def cache_tokens(cache, pages, h, n):
    """Codes [n, 128] and scales [n] (float64) of head h's first n tokens in ``pages``, keys then values.
    A page outside the pool has scale NaN and codes 0, and there = False."""
    n_pages, _, page, width = cache["K_codes"].shape
    bits = width // 16
    out = []
    there = np.zeros(n, bool)
    at = np.arange(n) // page
    ids = np.asarray(pages)[at] if n else np.zeros(0, int)
    there[:] = (ids >= 0) & (ids < n_pages)
    safe = np.where(there, ids, 0)
    slot = np.arange(n) % page
    for name in "KV":
        if name == "K":
            raw = cache["K_codes"][safe, h, slot]
        else:
            raw = cache["V_codes"][safe, h, slot // 4, :, slot % 4].reshape(n, width)
        codes = unpack_int4(raw) if bits == 4 else raw.view(np.int8)
        out += [codes.reshape(n, D).astype(np.float64), cache[name + "_scale"][safe, h, slot].astype(np.float64)]
    return (*out, there)


def kv_attend(q, cache, table, q_start, kv_len, scale, softcap=0.0, slopes=None, window=0, causal=True, bidir_len=None,
              prefix_table=None, prefix_len=0, rows=None):
    """(O [T, Hq, 128] float64, NaN rows where nothing is written, bound [T, Hq, 128]).  ``rows``: those of T to
    compute, all by default; what is returned for others means nothing.

    ``bound`` is how far a result may be that holds scores in float32, rounds softmax weights (times the value's
    scale, relative to the row's largest) to fp16 and the result to fp16:

      z      128 products and their sum, the key's scale, the softmax scale, bias and cap: 132 roundings of at most
             2^-24 of sum |terms|, and the exponentials' own errors, 2^-16 in all at the sizes here
      cap    2^-18 of the capped score (the tanh's argument, exponential, reciprocal and sums, 36 roundings of 2^-24
             where the score is a quarter of the cap, fewer below); at caps up to 64 2^-22 of the cap instead
      w      half a step, 2^-11 relative; below 2^-14 of the largest half a subnormal step, 2^-25
      O      half a step, 2^-11 relative; below 2^-14 half a subnormal step, 2^-25
    """
    T, Hq, _ = q.shape
    n_pages, H, page, _ = cache["K_codes"].shape
    G = Hq // H
    out, bound = np.full(q.shape, np.nan), np.zeros(q.shape)
    for h in range(H):
        if prefix_len:
            front = cache_tokens(cache, prefix_table, h, prefix_len)
        for b in range(len(kv_len)):
            if rows is not None and not any(t in rows for t in range(q_start[b], q_start[b + 1])):
                continue
            kv = min(_length(kv_len[b]), table.shape[1] * page)
            parts = cache_tokens(cache, table[b], h, kv)
            if prefix_len:
                parts = tuple(np.concatenate([f, p]) for f, p in zip(front, parts))
            kc, ks, vc, vs, there = parts
            j = np.arange(prefix_len + kv)
            for t in range(q_start[b], min(q_start[b + 1], T)):
                if rows is not None and t not in rows:
                    continue
                p = prefix_len + _length(kv_len[b]) - int(q_start[b + 1]) + t
                seen = there.copy()
                if causal:
                    seen &= (j <= p) | (j < (bidir_len[b] if bidir_len is not None else 0))
                if window:
                    seen &= np.abs(p - j) < window
                for g in range(h * G, (h + 1) * G):
                    x = q[t, g].astype(np.float64)
                    if not seen.any():
                        out[t, g] = 0.0
                        continue
                    if not (np.isfinite(ks[seen]).all() and np.isfinite(vs[seen]).all()):
                        out[t, g] = np.inf     # stands for "has to be NaN"
                        continue
                    kd, sc, vd, vsc = kc[seen], ks[seen], vc[seen], vs[seen]
                    z = scale * (kd @ x) * sc
                    ez = 132 * 2.0 ** -24 * abs(scale) * (np.abs(kd) @ np.abs(x)) * sc + 2.0 ** -16
                    if softcap:
                        z = softcap * np.tanh(z / softcap)
                        ez += softcap * 2.0 ** -22 if softcap <= 64 else np.abs(z) * 2.0 ** -18
                    if slopes is not None:
                        bias = float(slopes[g]) * np.abs(p - j[seen])
                        z = z - bias
                        ez += np.abs(bias) * 2.0 ** -22
                    w = np.exp(z - z.max())
                    l = w.sum()
                    v = vd * vsc[:, None]
                    o = (w @ v) / l
                    spread = ((w * (2.0 ** -11 + ez)) @ np.abs(v)) / l
                    top = (w * np.maximum(vsc, 2.0 ** -24)).max()
                    tiny = 2.0 ** -25 * top * np.abs(vd).sum(axis=0) / l
                    out[t, g] = o
                    bound[t, g] = spread + tiny + np.abs(o) * (2.0 ** -11 + (w * ez).sum() / l) + 2.0 ** -25
    return out, bound
