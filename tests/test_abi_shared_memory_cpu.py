"""Tensors of one call in the same memory, without a GPU: what is refused, before any device call (fake, never dereferenced
pointers), also under the host sanitizers."""

import os
import sys

import pytest

from rotation_bit_quantization_amd import spin

from .test_abi_paged_cpu import A, ROOT, caller
from .test_abi_served_cpu import lib  # noqa: F401


def test_a_move_within_rows_of_another_length(lib):  # noqa: F811
    """Of several sequences rows of another length in page_table's memory are other pages, which may be those that tokens
    come from."""
    call = caller(lib.spin_kv_move, dict(kc=A, ks=A, vc=A, vs=A, W=A, Hkv=8, D=128, bits=4, n_pages=10, page=16, B=3, table=A, max_pages=5,
                                         kept=A, heads=8, n=100, at=A, to=A, to_pages=2, st=None))
    assert call() == call(to_pages=9) == call(heads=1, W=None) == spin.SPIN_ERR_BAD_SHAPE
    assert call(n=0) == call(B=0) == spin.SPIN_OK


def test_lengths_that_overlap_in_part(lib):  # noqa: F811
    """Of 100 sequences; lens may be kv_len itself or lie beside it."""
    call = caller(lib.spin_kv_choose, dict(W=A, Hkv=8, n_pages=10, page=16, B=100, kv_len=1 << 20, table=A, max_pages=5, keep=40, first=4,
                                           recent=30, kept=A, lens=(1 << 20) + 16, ws=A, ws_bytes=1 << 30, st=None))
    for lens in ((1 << 20) + 16, (1 << 20) + 384, (1 << 20) - 16, (1 << 20) - 384):
        assert call(lens=lens) == spin.SPIN_ERR_UNSUPPORTED
        assert call(lens=lens, B=0) == spin.SPIN_OK


def test_a_tree_in_its_parents_memory(lib):  # noqa: F811
    """Rows walk through other rows' parents."""
    at = 1 << 20
    call = caller(lib.spin_kv_tree, dict(parent=at, T=100, B=4, q_start=A, kv_len=A, pos0=0, words=2, tree=1 << 22, pos=1 << 23, st=None))
    for bad in (dict(pos=at), dict(pos=at + 384), dict(pos=at - 384), dict(tree=at), dict(tree=at + 384), dict(tree=at - 784)):
        assert call(**bad) == spin.SPIN_ERR_UNSUPPORTED, bad
        assert call(**bad, T=0) == call(**bad, B=0) == spin.SPIN_OK


def test_weights_that_overlap_their_prior_in_part(lib):  # noqa: F811
    """Of 10 x 8 x 16 slots; prior may be W itself."""
    at = 1 << 20
    call = caller(lib.spin_kv_weights, dict(Q=A, lse=A, T=5, Hq=32, Hkv=8, D=128, bits=4, kc=A, ks=A, n_pages=10, page=16, B=1, q_start=A,
                                            kv_len=A, table=A, max_pages=5, pos0=0, scale=0.1, cap=0.0, slopes=A, window=0, causal=1,
                                            bidir=A, prior=at, decay=1.0, W=at, ws=A, ws_bytes=1 << 30, st=None))
    for W in (at + 16, at - 16, at + 5104, at - 5104):
        assert call(W=W) == spin.SPIN_ERR_UNSUPPORTED
        assert call(W=W, B=0) == spin.SPIN_OK


def test_under_host_sanitizers():
    if os.environ.get("SPIN_LIBRARY"):
        pytest.skip("already the sanitized library")
    from rotation_bit_quantization_amd import build
    from .test_host_sanitizers import _run
    if not os.path.exists(os.path.join(ROOT, "rotation_bit_quantization_amd", "libspin.so")):
        pytest.skip("libspin.so not built")
    try:
        library, runtime = build.build_host_sanitized(), build.sanitizer_runtime()
    except RuntimeError as e:
        pytest.skip(f"host sanitizer build unavailable: {e}")
    out = _run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider", os.path.join("tests", "test_abi_shared_memory_cpu.py")],
               {"LD_PRELOAD": runtime, "SPIN_LIBRARY": library})
    assert " passed" in out and " failed" not in out
