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

__all__ = ["rope_table", "turn_heads", "kv_append", "kv_attend", "cache_tokens", "kv_tree", "kv_weights", "kv_choose", "kv_move"]

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
              pos0=0, positions=None):
    """The cache (a dict of numpy arrays, a changed copy) and the queries in float64 (NaN rows: not written).
    ``positions`` [T]: what rows are turned by, in place of pos0 + place."""
    cache = {name: a.copy() for name, a in cache.items()}
    pages, H, page, width = cache["K_codes"].shape
    bits = width // 16
    T = k.shape[0]
    q_out = np.full(q.shape, np.nan)
    for t, b, p in _places(q_start, kv_len, T):
        turn = p + pos0 if positions is None else int(positions[t])
        if p < 0 or p >= table.shape[1] * page or (rope is not None and not 0 <= turn < len(rope)):
            q_out[t] = 0.0
            continue
        row = None if rope is None else rope[turn][None]
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
              prefix_table=None, prefix_len=0, rows=None, tree=None, positions=None, sums=False):
    """(O [T, Hq, 128] float64, NaN rows where nothing is written, bound [T, Hq, 128]).  ``rows``: those of T to
    compute, all by default; what is returned for others means nothing.

    ``tree`` [T, words] uint32: rows see the context and, of their sequence's new tokens, those whose bits are set;
    distances of new tokens go by ``positions`` [T].  With ``sums`` also (log sum e^z [T, Hq], bound): errors of the
    scores, weighted, a rounding of the sum for every token and 2^-22 of the logarithm.

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
    logs, log_bound = np.full((T, Hq), np.nan), np.zeros((T, Hq))
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
                seen, at = there.copy(), j
                if tree is not None:
                    names, at, p = _tree_row(tree, positions, t, q_start, b, prefix_len, _length(kv_len[b]), j)
                    seen &= names
                elif causal:
                    seen &= (j <= p) | (j < (bidir_len[b] if bidir_len is not None else 0))
                if window:
                    seen &= np.abs(p - at) < window
                for g in range(h * G, (h + 1) * G):
                    x = q[t, g].astype(np.float64)
                    if not seen.any():
                        out[t, g], logs[t, g] = 0.0, -np.inf
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
                        bias = float(slopes[g]) * np.abs(p - at[seen])
                        z = z - bias
                        ez += np.abs(bias) * 2.0 ** -22
                    w = np.exp(z - z.max())
                    l = w.sum()
                    logs[t, g] = z.max() + np.log(l)
                    log_bound[t, g] = (w * ez).sum() / l + 2.0 ** -24 * len(z) + 2.0 ** -22 * (abs(logs[t, g]) + 24)
                    v = vd * vsc[:, None]
                    o = (w @ v) / l
                    spread = ((w * (2.0 ** -11 + ez)) @ np.abs(v)) / l
                    top = (w * np.maximum(vsc, 2.0 ** -24)).max()
                    tiny = 2.0 ** -25 * top * np.abs(vd).sum(axis=0) / l
                    out[t, g] = o
                    bound[t, g] = spread + tiny + np.abs(o) * (2.0 ** -11 + (w * ez).sum() / l) + 2.0 ** -25
    return (out, bound, logs, log_bound) if sums else (out, bound)


def _tree_row(tree, positions, t, q_start, b, prefix_len, kv, j):
    """Which of the tokens j, a prefix and the kv of sequence b behind it, row t names, their positions and its own.
    A prefix's tokens are context, also where the sequence has fewer tokens than rows."""
    news = int(q_start[b + 1]) - int(q_start[b])
    i = np.where(j < prefix_len, -1, j - (prefix_len + kv - news))
    bits = np.unpackbits(np.ascontiguousarray(tree[t]).view(np.uint8), bitorder="little").astype(bool)
    names = i < 0
    inside = (i >= 0) & (i < min(len(bits), news))
    names[inside] = bits[i[inside]]
    if positions is None:
        return names, j, 0
    held = lambda rows: np.clip(np.asarray(positions)[rows], 0, 1 << 30)  # noqa: E731
    at = np.array(j)
    fresh = (i >= 0) & (i < news)
    at[fresh] = held(int(q_start[b]) + i[fresh])
    return names, at, int(held(t))


def kv_tree(parent, q_start, kv_len, words, pos0=0):
    """(tree [T, words] uint32, positions [T]) of drafted tokens, by walking up from each."""
    tree, positions = np.zeros((len(parent), words), np.uint32), np.zeros(len(parent), np.int32)
    for b in range(len(kv_len)):
        lo, hi = int(q_start[b]), int(q_start[b + 1])
        for t in range(lo, hi):
            i, depth = t - lo, -1
            while i >= 0 and t - lo < 32 * words:
                tree[t, i // 32] |= np.uint32(1 << (i % 32))
                p = int(parent[lo + i])
                i, depth = p if p < i else -1, depth + 1
            positions[t] = pos0 + _length(kv_len[b]) - (hi - lo) + max(depth, 0)
    return tree, positions


def kv_weights(q, lse, cache, table, q_start, kv_len, scale, softcap=0.0, slopes=None, window=0, causal=True, bidir_len=None,
               pos0=0, prior=None, decay=1.0, prior_len=None):
    """(W [n_pages, Hkv, page] float64, NaN where nothing is written, bound): decay * prior + the attention weight that
    each token draws; of a sequence's tokens from prior_len[b] on the prior is 0.

    A weight is off by the score's error (128 products of the query with codes and their sum, its scale, bias and
    cap: 132 roundings of 2^-24 of the terms; the cap as in ``kv_attend``, below 0.7 of it 2^-22 of the score), that of
    the difference to lse in units of log2 (2^-22 of both) and the exponential's 2^-22 (numbers below 2^-126 may be 0); the sum by a rounding of itself for
    every row, and two for the prior."""
    T, Hq, _ = q.shape
    n_pages, H, page, _ = cache["K_codes"].shape
    G = Hq // H
    W, bound = np.full((n_pages, H, page), np.nan), np.zeros((n_pages, H, page))
    for b in range(len(kv_len)):
        kv = min(_length(kv_len[b]), table.shape[1] * page)
        j = np.arange(kv)
        lo, hi = int(q_start[b]), min(int(q_start[b + 1]), T)
        p = pos0 + _length(kv_len[b]) - int(q_start[b + 1]) + np.arange(lo, hi)[:, None]
        far = p - (pos0 + j)[None]
        seen = np.ones(far.shape, bool)
        if causal:
            seen &= (far >= 0) | (pos0 + j < (bidir_len[b] if bidir_len is not None else 0))[None]
        if window:
            seen &= np.abs(far) < window
        for h in range(H):
            kd, ks, _, _, there = cache_tokens(cache, table[b], h, kv)
            fine = there & np.isfinite(ks)
            ks = np.where(fine, ks, 0.0)
            w, e = np.zeros(kv), np.zeros(kv)
            for g in range(h * G, (h + 1) * G):
                counts = np.isfinite(lse[lo:hi, g])
                x = np.where(counts[:, None], q[lo:hi, g].astype(np.float64), 0.0)
                log = np.where(counts, lse[lo:hi, g].astype(np.float64), 0.0)[:, None]
                z = scale * (x @ kd.T) * ks
                ez = 132 * 2.0 ** -24 * abs(scale) * (np.abs(x) @ np.abs(kd).T) * ks
                if softcap:
                    near = np.abs(z) < 0.7 * softcap
                    z = softcap * np.tanh(z / softcap)
                    ez += np.where(near, np.abs(z) * 2.0 ** -22, softcap * 2.0 ** -22 if softcap <= 64 else np.abs(z) * 2.0 ** -18)
                if slopes is not None:
                    z = z - float(slopes[g]) * np.abs(far)
                    ez += np.abs(float(slopes[g]) * far) * 2.0 ** -22
                ez += 2.0 ** -22 * (np.abs(z) + np.abs(log) + 1)
                weight = np.where(seen & counts[:, None] & fine[None], np.exp(np.minimum(z - log, 700.0)), 0.0)
                w += weight.sum(0)
                e += (weight * ez).sum(0)
            e += 2.0 ** -24 * ((hi - lo) * G + 8) * w
            at, slot = np.where(there, table[b][j // page], 0)[there], (j % page)[there]
            if prior is not None:
                old = decay * prior[at, h, slot].astype(np.float64)
                if prior_len is not None:
                    old = np.where(j[there] < prior_len[b], old, 0.0)
                w[there] += old
                e[there] += 2.0 ** -23 * (np.abs(old) + np.abs(w[there]))
            W[at, h, slot], bound[at, h, slot] = w[there], e[there] + 2.0 ** -110
    return W, bound


def kv_choose(W, table, kv_len, keep, first=0, recent=0):
    """(kept [B, Hkv, keep] int32, lens [B]): by sorting."""
    n_pages, H, page = W.shape
    kept, lens = np.full((len(kv_len), H, keep), -1, np.int32), np.zeros(len(kv_len), np.int32)
    for b in range(len(kv_len)):
        n = min(max(int(kv_len[b]), 0), table.shape[1] * page)
        j = np.arange(n)
        ids = table[b][j // page]
        there = (ids >= 0) & (ids < n_pages)
        must = (j < first) | (j >= n - recent)
        lens[b] = m = min(n, keep)
        for h in range(H):
            w = W[np.where(there, ids, 0), h, j % page].astype(np.float64)
            none = ~there | np.isnan(w)
            order = np.lexsort((j, -np.where(none, 0.0, w), none, ~must))
            kept[b, h, :m] = np.sort(order[:m])
    return kept, lens


def kv_move(cache, table, kept, at=None, to_table=None, W=None):
    """(the changed cache, the changed W): every token is read before any is written."""
    n_pages, H, page, _ = cache["K_codes"].shape
    old = dict(cache) if W is None else dict(cache, W=W)
    new = {k: v.copy() for k, v in old.items()}
    to_table = table if to_table is None else to_table

    def slot(rows, place):
        if place < 0 or place >= len(rows) * page or not 0 <= rows[place // page] < n_pages:
            return None
        return int(rows[place // page]), place % page

    for b in range(len(table)):
        start = 0 if at is None else int(at[b])
        for h in range(H):
            for i, src in enumerate(kept[b, h % kept.shape[1]]):
                here, there = slot(table[b], start + int(src)), slot(to_table[b], start + i)
                if src < 0 or here is None or there is None:
                    continue
                (p, s), (q, d) = here, there
                for name in old:
                    if name == "V_codes":
                        new[name][q, h, d // 4, :, d % 4] = old[name][p, h, s // 4, :, s % 4]
                    else:
                        new[name][q, h, d] = old[name][p, h, s]
    return {k: v for k, v in new.items() if k != "W"}, new.get("W")
