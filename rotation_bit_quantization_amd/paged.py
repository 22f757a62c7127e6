"""Binding of the libspin calls around a paged cache's steps: trees of drafted tokens (ancestors, attention, the accepted
path's move) and eviction (the weight that tokens draw, the choice of those that stay, their move).

They are reached as spin.spin_kv_tree and so on, and are made as the calls in spin.py are: checks of the tensors, outputs
on the stream of the call, the C entry of the same name (spin_kv_attn_ex for spin_kv_attn_tree).

Declarations and contracts: include/libspin.h.
"""

import ctypes
import functools

import torch

from .spin import _attn, _batch, _cache, _check, _gpu, _int, _launch, _on_stream, _prefix, _ptr, _raise, _want, load

__all__ = ["spin_kv_tree", "spin_kv_attn_tree", "spin_kv_weights", "spin_kv_weights_workspace", "spin_kv_choose",
           "spin_kv_choose_workspace", "spin_kv_move"]


def _all(dev, *given):
    """Raise unless every (tensor, name, dtype, shape) is contiguous, of that type and shape, on GPU `dev`."""
    for t, name, dtype, shape in given:
        if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous()):
            _want(t, name, dtype, shape, dev) if isinstance(t, torch.Tensor) else _check(t, name, (dtype,), shape)


def spin_kv_tree(parent, q_start, kv_len, words, pos0=0, tree=None, positions=None, stream=None):
    """parent [T] int32 (of each new token of a sequence, the number of the one before it, -1: the context's last)
    -> (tree [T, words] int32: bits of each token's ancestors and itself, positions [T] int32)."""
    if stream is not None:
        return _on_stream(stream, parent, spin_kv_tree, parent, q_start, kv_len, words, pos0, tree, positions)
    dev = _gpu(parent, "parent")
    if parent.dim() != 1 or kv_len.dim() != 1:
        raise ValueError(f"parent and kv_len have shapes {tuple(parent.shape)} and {tuple(kv_len.shape)}, expected [T] and [B]")
    T, B, words = _int(parent.shape[0], "T"), _int(kv_len.shape[0], "B"), _int(words, "words")
    if words < 1:
        raise ValueError(f"words is {words}, expected 1 or more")
    _all(dev, (parent, "parent", torch.int32, (T,)), (q_start, "q_start", torch.int32, (B + 1,)), (kv_len, "kv_len", torch.int32, (B,)))
    if tree is None:
        tree = torch.empty((T, words), dtype=torch.int32, device=parent.device)
    else:
        _want(tree, "tree", torch.int32, (T, words), dev)
    if positions is None:
        positions = torch.empty_like(parent)
    else:
        _want(positions, "positions", torch.int32, (T,), dev)
    if T != 0 and B != 0:           # an empty tensor has no address to pass
        _launch("spin_kv_tree", dev, (parent.data_ptr(), T, B, q_start.data_ptr(), kv_len.data_ptr(), _int(pos0, "pos0"), words,
                                      tree.data_ptr(), positions.data_ptr()))
    return tree, positions


def spin_kv_attn_tree(Q, cache, page_table, q_start, kv_len, tree, positions=None, scale=None, softcap=0.0, slopes=None,
                      window=0, prefix_table=None, prefix_len=0, O=None, workspace=None, stream=None, lse=None):
    """spin_kv_attn (spin_kv_attn_shared behind a prefix) where ``tree`` [T, words] int32 says which of its sequence's
    new tokens a row sees beside the context, as spin_kv_tree writes it; ``positions`` [T] int32 are needed with a
    window or slopes."""
    if stream is not None:
        return _on_stream(stream, Q, spin_kv_attn_tree, Q, cache, page_table, q_start, kv_len, tree, positions, scale,
                          softcap, slopes, window, prefix_table, prefix_len, O, workspace, lse=lse)
    if tree is None:
        raise TypeError("tree must be a torch.Tensor")
    if prefix_table is None and prefix_len:
        raise ValueError("prefix_len without prefix_table")
    prefix = None if prefix_table is None else _prefix(prefix_table, prefix_len, cache)
    return _attn("spin_kv_attn_ex", Q, cache, prefix, page_table, q_start, kv_len, scale, softcap, slopes, window, False, None,
                 O, workspace, lse, tree, positions)


def _weights(W, name, cache, dev):
    """Check an fp32 tensor of the cache's slots; returns its address."""
    return _want(W, name, torch.float32, cache["K_scale"].shape, dev)


@functools.lru_cache(4096)
def spin_kv_weights_workspace(T, Hq, Hkv, B, max_pages, page_size):
    """Bytes of workspace that spin_kv_weights takes at these sizes."""
    for name, x in dict(T=T, Hq=Hq, Hkv=Hkv, B=B, max_pages=max_pages, page_size=page_size).items():
        _int(x, name)
    n = ctypes.c_size_t(0)
    _raise("spin_kv_weights_workspace", load().spin_kv_weights_workspace(T, Hq, Hkv, B, max_pages, page_size, ctypes.byref(n)))
    return n.value


def _workspace(given, need, of, dev):
    """(the workspace of a call, its bytes): the caller's, or one of ``need`` bytes on ``of``'s GPU."""
    if given is not None:
        _want(given, "workspace", torch.uint8, (given.numel(),), dev)
        return given, given.numel()
    return (of.new_empty((need,), dtype=torch.uint8), need) if need else (None, 0)


def spin_kv_weights(Q, lse, cache, page_table, q_start, kv_len, scale=None, softcap=0.0, slopes=None, window=0, causal=True,
                    bidir_len=None, pos0=0, prior=None, decay=1.0, W=None, stream=None, workspace=None, prior_len=None):
    """Q [T, Hq, 128] fp16 and lse [T, Hq] fp32 (from spin_kv_attn, with the same scores and masks) -> W [n_pages, Hkv,
    page_size] fp32: at each cached token's slot decay * prior + the attention weight it draws from the rows.

    W is made, of zeros, if it is not given; it may be ``prior``.  ``prior_len`` [B] int32 (spin_kv_weights_ex): how many of
    each sequence's tokens have a prior; those behind them, whose slots may hold sums of tokens that are gone, start at 0.
    ``workspace`` (uint8, spin_kv_weights_workspace bytes)
    is allocated if it is not given."""
    if stream is not None:
        return _on_stream(stream, Q, spin_kv_weights, Q, lse, cache, page_table, q_start, kv_len, scale, softcap, slopes,
                          window, causal, bidir_len, pos0, prior, decay, W, workspace=workspace, prior_len=prior_len)
    dev = _gpu(Q, "Q")
    (kc, ks, _, _), n_pages, Hkv, page, bits = _cache(cache, dev)
    (starts, lens, table), B, max_pages = _batch(page_table, q_start, kv_len, dev)
    shape = Q.shape
    if len(shape) != 3 or shape[2] != 128:
        raise ValueError(f"Q has shape {tuple(shape)}, expected [T, Hq, 128]")
    T, Hq, _ = shape
    q = _want(Q, "Q", torch.float16, shape, dev)
    log = _want(lse, "lse", torch.float32, (T, Hq), dev)
    slope = None if slopes is None else _want(slopes, "slopes", torch.float32, (Hq,), dev)
    both = None if bidir_len is None else _want(bidir_len, "bidir_len", torch.int32, (B,), dev)
    old = None if prior is None else _weights(prior, "prior", cache, dev)
    fn, known = "spin_kv_weights", ()
    if prior_len is not None:
        if prior is None:
            raise ValueError("prior_len without prior")
        fn, known = "spin_kv_weights_ex", (_want(prior_len, "prior_len", torch.int32, (B,), dev),)
    if W is None:
        W = torch.zeros(cache["K_scale"].shape, dtype=torch.float32, device=Q.device)
    out = _weights(W, "W", cache, dev)
    if B != 0:                      # an empty tensor has no address to pass; no rows are no weights
        if T == 0:
            q = log = starts
        ws, ws_bytes = _workspace(workspace, spin_kv_weights_workspace(T, Hq, Hkv, B, max_pages, page), Q, dev)
        _launch(fn, dev,
                (q, log, T, Hq, Hkv, 128, bits, kc, ks, n_pages, page, B, starts, lens, table, max_pages, _int(pos0, "pos0"),
                 0.08838834764831845 if scale is None else scale, softcap, slope, _int(window, "window"), _int(causal, "causal"), both,
                 old, *known, decay, out, _ptr(ws), ws_bytes))
    return W


@functools.lru_cache(4096)
def spin_kv_choose_workspace(Hkv, B, max_pages, page_size):
    """Bytes of workspace that spin_kv_choose takes at these sizes."""
    for name, x in dict(Hkv=Hkv, B=B, max_pages=max_pages, page_size=page_size).items():
        _int(x, name)
    n = ctypes.c_size_t(0)
    _raise("spin_kv_choose_workspace", load().spin_kv_choose_workspace(Hkv, B, max_pages, page_size, ctypes.byref(n)))
    return n.value


def spin_kv_choose(W, page_table, kv_len, keep, first=0, recent=0, kept=None, lens=None, stream=None, workspace=None):
    """W [n_pages, Hkv, page_size] fp32 -> (kept [B, Hkv, keep] int32: the places of the tokens that stay, ascending, -1
    behind them, lens [B] int32): per sequence and head its first ``first`` and last ``recent`` tokens and those of
    greatest weight.  ``lens`` may be ``kv_len``, which it replaces.  ``workspace`` (uint8, spin_kv_choose_workspace bytes) is
    allocated if it is not given."""
    if stream is not None:
        return _on_stream(stream, W, spin_kv_choose, W, page_table, kv_len, keep, first, recent, kept, lens, workspace=workspace)
    dev = _gpu(W, "W")
    if W.dim() != 3 or page_table.dim() != 2:
        raise ValueError(f"W and page_table have shapes {tuple(W.shape)} and {tuple(page_table.shape)}, expected [n_pages, Hkv, page_size] "
                         "and [B, max_pages]")
    n_pages, Hkv, page = W.shape
    B, max_pages = page_table.shape
    keep = _int(keep, "keep")
    if keep < 1:
        raise ValueError(f"keep is {keep}, expected 1 or more")
    _all(dev, (W, "W", torch.float32, W.shape), (page_table, "page_table", torch.int32, (B, max_pages)), (kv_len, "kv_len", torch.int32, (B,)))
    if kept is None:
        kept = torch.empty((B, Hkv, keep), dtype=torch.int32, device=W.device)
    else:
        _want(kept, "kept", torch.int32, (B, Hkv, keep), dev)
    if lens is None:
        lens = torch.empty_like(kv_len)
    else:
        _want(lens, "lens", torch.int32, (B,), dev)
    if B != 0:                      # an empty tensor has no address to pass
        ws, ws_bytes = _workspace(workspace, spin_kv_choose_workspace(Hkv, B, max_pages, page), W, dev)
        _launch("spin_kv_choose", dev, (W.data_ptr(), Hkv, n_pages, page, B, kv_len.data_ptr(), page_table.data_ptr(), max_pages, keep,
                                        _int(first, "first"), _int(recent, "recent"), kept.data_ptr(), lens.data_ptr(), _ptr(ws), ws_bytes))
    return kept, lens


def spin_kv_move(cache, page_table, kept, at=None, to_table=None, W=None, stream=None):
    """The tokens at places ``at`` + ``kept`` [B, 1 or Hkv, n] int32 of each sequence go to places ``at`` + 0, 1, .. of its
    pages, or of those that ``to_table`` names, with their weights ``W`` if given; entries below 0 are passed over.
    ``to_table`` may be ``page_table`` itself, of one sequence also its first pages alone.  Returns ``cache``."""
    if stream is not None:
        return _on_stream(stream, kept, spin_kv_move, cache, page_table, kept, at, to_table, W)
    dev = _gpu(kept, "kept")
    addresses, n_pages, Hkv, page, bits = _cache(cache, dev)
    if kept.dim() != 3 or page_table.dim() != 2 or kept.shape[1] not in (1, Hkv):
        raise ValueError(f"kept and page_table have shapes {tuple(kept.shape)} and {tuple(page_table.shape)}, expected [B, 1 or {Hkv}, n] "
                         "and [B, max_pages]")
    B, max_pages = page_table.shape
    heads, n = kept.shape[1:]
    _all(dev, (page_table, "page_table", torch.int32, (B, max_pages)), (kept, "kept", torch.int32, (B, heads, n)))
    start = None if at is None else _want(at, "at", torch.int32, (B,), dev)
    to, to_pages = None, 0
    if to_table is not None:
        if to_table.dim() != 2:
            raise ValueError(f"to_table has shape {tuple(to_table.shape)}, expected [B, pages]")
        to_pages = _int(to_table.shape[1], "to_table's pages")
        to = _want(to_table, "to_table", torch.int32, (B, to_pages), dev)
    w = None if W is None else _weights(W, "W", cache, dev)
    if B != 0 and n != 0 and not (to_table is not None and to_pages == 0):      # an empty tensor has no address to pass
        _launch("spin_kv_move", dev, (*addresses, w, Hkv, 128, bits, n_pages, page, _int(B, "B"), page_table.data_ptr(), _int(max_pages, "max_pages"),
                                      kept.data_ptr(), heads, _int(n, "n"), start, to, to_pages))
    return cache
