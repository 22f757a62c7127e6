"""Argument validation of the calls for drafted trees and eviction, without a GPU: every error is returned before any
device call (fake, never dereferenced pointers), also under the host sanitizers."""

import ctypes
import os
import sys

import pytest

from rotation_bit_quantization_amd import spin

from .test_abi_paged_cpu import A, APPEND, ATTN, BIG, ROOT, U, caller

INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(spin.library_path()):
        pytest.skip("libspin.so not built (python -m rotation_bit_quantization_amd.build)")
    return spin.load()


def refusals(call, null, unsupported, shape, aligned):
    for name in null:
        assert call(**{name: None}) == spin.SPIN_ERR_NULL, name
    for bad in unsupported:
        assert call(**bad) == spin.SPIN_ERR_UNSUPPORTED, bad
    for bad in shape:
        assert call(**bad) == spin.SPIN_ERR_BAD_SHAPE, bad
    for name in aligned:
        assert call(**{name: U}) == spin.SPIN_ERR_MISALIGNED, name


PAGES = (dict(B=-1), dict(n_pages=0), dict(page=8), dict(page=48), dict(page=2048), dict(page=0), dict(max_pages=0), dict(max_pages=1 << 26))


def test_tree(lib):
    call = caller(lib.spin_kv_tree, dict(parent=A, T=0, B=4, q_start=A, kv_len=A, pos0=0, words=2, tree=A, pos=A, st=None))
    assert call() == call(T=9, B=0) == spin.SPIN_OK
    refusals(call, ("parent", "q_start", "kv_len", "tree", "pos"), (),
             (dict(T=-1), dict(T=(1 << 26) + 1), dict(B=-1), dict(pos0=-1), dict(pos0=BIG), dict(words=0), dict(words=-1), dict(words=129)),
             ("parent", "q_start", "kv_len", "tree", "pos"))


def test_append_at(lib):
    names = list(APPEND)
    ok = {("pos" if k == "pos0" else k): (A if k == "pos0" else APPEND[k]) for k in names}
    call = caller(lib.spin_kv_append_at, ok)
    assert call() == call(T=5, B=0) == spin.SPIN_OK
    refusals(call, ("pos", "K", "V", "kc", "table", "out"), (dict(dt=2), dict(bits=5), dict(inter=2), dict(eps=NAN)),
             (dict(T=-1), dict(D=64), dict(rot=24), dict(rope_len=0), dict(ks=1020), dict(T=1 << 27)), ("pos", "Q", "K", "rope", "out"))


def test_attention_with_more(lib):
    head = list(ATTN.items())
    ok = dict(head[:12] + [("prefix", A), ("prefix_len", 50)] + head[12:])
    ok = list(ok.items())
    at = [k for k, _ in ok].index("O")
    ok = dict(ok[:at] + [("tree", A), ("words", 2), ("pos", A), ("O", A), ("lse", A)] + ok[at + 1:])
    ok["bidir"] = None
    call = caller(lib.spin_kv_attn_ex, ok)
    assert call() == call(T=5, B=0) == call(lse=None) == call(tree=None, words=0, pos=None, bidir=A) == spin.SPIN_OK
    assert call(pos=None, slopes=None) == call(words=128) == call(prefix=None, prefix_len=0) == spin.SPIN_OK
    refusals(call, ("Q", "kc", "ks", "vc", "vs", "q_start", "kv_len", "table", "O", "prefix", "pos"),
             (dict(bits=6), dict(causal=2), dict(scale=NAN), dict(cap=-1.0), dict(bidir=A)),
             (dict(T=-1), dict(Hq=31), dict(window=-1), dict(words=0), dict(words=-3), dict(words=129), dict(prefix_len=-1)) + PAGES,
             ("Q", "tree", "pos", "lse", "O", "ws", "slopes"))
    assert call(pos=None, slopes=None, window=5) == spin.SPIN_ERR_NULL
    long = dict(T=1, B=1, max_pages=4096)
    assert call(**long, ws=None) == spin.SPIN_ERR_NULL
    assert call(**long, ws_bytes=16) == spin.SPIN_ERR_BAD_SHAPE


def test_weights(lib):
    call = caller(lib.spin_kv_weights, dict(Q=A, lse=A, T=5, Hq=32, Hkv=8, D=128, bits=4, kc=A, ks=A, n_pages=10, page=16, B=0, q_start=A,
                                            kv_len=A, table=A, max_pages=5, pos0=0, scale=0.1, cap=0.0, slopes=A, window=0, causal=1,
                                            bidir=A, prior=A, decay=1.0, W=A, ws=A, ws_bytes=1 << 30, st=None))
    assert call() == call(slopes=None, bidir=None, prior=None) == call(decay=-2.0) == spin.SPIN_OK
    refusals(call, ("Q", "lse", "kc", "ks", "q_start", "kv_len", "table", "W"),
             (dict(bits=5), dict(causal=2), dict(scale=NAN), dict(scale=INF), dict(cap=-1.0), dict(cap=INF), dict(decay=NAN), dict(decay=-INF)),
             (dict(T=-1), dict(D=64), dict(Hq=31), dict(Hq=0), dict(Hkv=0), dict(window=-1), dict(pos0=-1), dict(pos0=BIG), dict(T=BIG),
              dict(B=1 << 24), dict(B=BIG, max_pages=1 << 25), dict(Hq=1 << 17, Hkv=1 << 17)) + PAGES,
             ("Q", "lse", "kc", "ks", "q_start", "kv_len", "table", "slopes", "bidir", "prior", "W", "ws"))
    # many rows of few heads are dealt out in shares, which need their workspace
    long = dict(T=4096, B=1, max_pages=256)
    assert call(**long, ws=None) == spin.SPIN_ERR_NULL
    assert call(**long, ws_bytes=16) == spin.SPIN_ERR_BAD_SHAPE


def test_weights_workspace(lib):
    n = ctypes.c_size_t(7)
    call = caller(lib.spin_kv_weights_workspace, dict(T=4096, Hq=32, Hkv=8, B=1, max_pages=256, page=16, out=ctypes.byref(n)))
    assert call() == spin.SPIN_OK and n.value >= 2 * 8 * 4096 * 4
    assert call(T=1) == spin.SPIN_OK and n.value == 0
    assert call(B=0) == spin.SPIN_OK and n.value == 0
    assert call(out=None) == spin.SPIN_ERR_NULL
    for bad in (dict(T=-1), dict(Hq=31), dict(Hkv=0), dict(B=-1), dict(max_pages=0), dict(page=7), dict(T=BIG), dict(B=BIG)):
        assert call(**bad) == spin.SPIN_ERR_BAD_SHAPE, bad


def test_choose(lib):
    call = caller(lib.spin_kv_choose, dict(W=A, Hkv=8, n_pages=10, page=16, B=0, kv_len=A, table=A, max_pages=5, keep=40, first=4, recent=30,
                                           kept=A, lens=A, ws=A, ws_bytes=1 << 30, st=None))
    assert call() == call(first=40, recent=0) == call(first=0, recent=40) == spin.SPIN_OK
    refusals(call, ("W", "kv_len", "table", "kept", "lens"), (),
             (dict(keep=0, first=0, recent=0), dict(keep=-1), dict(first=-1), dict(recent=-1), dict(first=11), dict(first=41, recent=0),
              dict(first=BIG, recent=BIG), dict(keep=BIG), dict(B=1 << 20), dict(Hkv=0),
              dict(B=1 << 16, max_pages=1 << 12)) + PAGES, ("W", "kv_len", "table", "kept", "lens", "ws"))
    assert call(ws=None, ws_bytes=0) == spin.SPIN_OK
    # long tables are dealt out, which needs a workspace
    assert call(B=1, max_pages=4096, ws=None) == spin.SPIN_ERR_NULL
    assert call(B=1, max_pages=4096, ws_bytes=16) == spin.SPIN_ERR_BAD_SHAPE
    n = ctypes.c_size_t(7)
    need = caller(lib.spin_kv_choose_workspace, dict(Hkv=8, B=2, max_pages=4096, page=16, out=ctypes.byref(n)))
    assert need() == spin.SPIN_OK and n.value >= 16 * 4 * 6144
    assert need(max_pages=2048) == spin.SPIN_OK and n.value == 0
    assert need(B=0) == spin.SPIN_OK and n.value == 0
    assert need(out=None) == spin.SPIN_ERR_NULL
    for bad in (dict(Hkv=0), dict(B=-1), dict(max_pages=0), dict(page=7), dict(B=BIG)):
        assert need(**bad) == spin.SPIN_ERR_BAD_SHAPE, bad


def test_move(lib):
    call = caller(lib.spin_kv_move, dict(kc=A, ks=A, vc=A, vs=A, W=A, Hkv=8, D=128, bits=4, n_pages=10, page=16, B=0, table=A, max_pages=5,
                                         kept=A, heads=8, n=20, at=A, to=A, to_pages=2, st=None))
    assert call() == call(W=None, at=None, to=None, to_pages=0) == call(heads=1) == call(B=5, n=0) == spin.SPIN_OK
    refusals(call, ("kc", "ks", "vc", "vs", "table", "kept"), (dict(bits=6),),
             (dict(D=64), dict(Hkv=0), dict(n=-1), dict(heads=2), dict(heads=0), dict(to_pages=0), dict(to_pages=-1), dict(to_pages=1 << 26),
              dict(B=1 << 22), dict(B=4, n=BIG)) + PAGES, ("kc", "ks", "vc", "vs", "W"))
    for name in ("table", "kept", "at", "to"):
        assert call(**{name: U}) == spin.SPIN_OK and call(**{name: U + 2}) == spin.SPIN_ERR_MISALIGNED, name


def test_the_binding_checks_before_the_library(lib):
    torch = pytest.importorskip("torch")
    c = spin.kv_cache(4, 2, 16, 4, device="cpu")
    i = torch.zeros((3,), dtype=torch.int32)
    for call in (lambda: spin.spin_kv_tree(i, i, i, 1), lambda: spin.spin_kv_weights(c["K_scale"], None, c, None, None, None),
                 lambda: spin.spin_kv_choose(c["K_scale"], None, None, 4), lambda: spin.spin_kv_move(c, None, i)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    for call in (lambda: spin.spin_kv_tree(None, i, i, 1), lambda: spin.spin_kv_choose(None, None, None, 4),
                 lambda: spin.spin_kv_move(c, None, None), lambda: spin.spin_kv_attn_tree(c["K_scale"], c, None, None, None, None)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(ValueError, match="prefix_table"):
        spin.spin_kv_attn_tree(c["K_scale"], c, None, None, None, i, prefix_len=5)


def test_validation_under_host_sanitizers():
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
    out = _run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider", os.path.join("tests", "test_abi_served_cpu.py")],
               {"LD_PRELOAD": runtime, "SPIN_LIBRARY": library})
    assert " passed" in out and " failed" not in out
