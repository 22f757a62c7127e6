"""Argument validation of the paged-cache calls, without a GPU: every error is returned before any device call
(fake, never dereferenced pointers), also under the host sanitizers."""

import ctypes
import os
import sys

import pytest

from rotation_bit_quantization_amd import spin

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A, U = 4096, 4100      # a fake aligned and a misaligned device address
BIG = 2 ** 31 - 1


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(spin.library_path()):
        pytest.skip("libspin.so not built (python -m rotation_bit_quantization_amd.build)")
    return spin.load()


def caller(f, ok):
    def call(**kw):
        assert set(kw) <= set(ok)
        return f(*dict(ok, **kw).values())
    return call


def test_rope_table(lib):
    call = caller(lib.spin_rope_table, dict(inv=A, n=64, pos0=0, P=0, s=1.0, table=A, st=None))
    assert call() == spin.SPIN_OK
    assert call(inv=None) == call(table=None) == spin.SPIN_ERR_NULL
    for bad in (dict(n=0), dict(n=65), dict(n=-1), dict(pos0=-1), dict(P=-1), dict(pos0=1 << 29, P=1), dict(pos0=BIG, P=BIG)):
        assert call(**bad) == spin.SPIN_ERR_BAD_SHAPE, bad
    assert call(inv=U) == call(table=U) == spin.SPIN_ERR_MISALIGNED


APPEND = dict(Q=A, K=A, V=A, dt=spin.SPIN_F32, T=0, Hq=32, Hkv=8, D=128, qs=6144, ks=6144, vs=6144, qn=A, kn=A, eps=1e-6, rope=A,
              rope_len=100, rot=128, inter=0, pos0=0, bits=4, kc=A, ksc=A, vc=A, vsc=A, n_pages=10, page=16, B=4, q_start=A,
              kv_len=A, table=A, max_pages=5, out=A, st=None)


def test_append(lib):
    call = caller(lib.spin_kv_append, APPEND)
    assert call() == spin.SPIN_OK and call(T=5, B=0) == spin.SPIN_OK
    assert call(Q=None, out=None, Hq=0, qs=0) == spin.SPIN_OK
    assert call(rope=None, rot=0, rope_len=0) == spin.SPIN_OK
    assert call(qn=None, kn=None, eps=float("nan")) == spin.SPIN_OK
    for name in ("K", "V", "kc", "ksc", "vc", "vsc", "q_start", "kv_len", "table", "Q", "out", "rope"):
        assert call(**{name: None}) == spin.SPIN_ERR_NULL, name
    assert call(rot=0) == spin.SPIN_ERR_NULL
    for bad in (dict(dt=2), dict(bits=5), dict(bits=0), dict(inter=2), dict(eps=-1e-9), dict(eps=float("nan")), dict(eps=float("inf"))):
        assert call(**bad) == spin.SPIN_ERR_UNSUPPORTED, bad
    for bad in (dict(T=-1), dict(D=64), dict(Hq=0), dict(Hkv=0), dict(B=-1), dict(n_pages=0), dict(max_pages=0), dict(page=8),
                dict(page=24), dict(page=0), dict(page=-16), dict(page=2048), dict(max_pages=1 << 26), dict(rot=24), dict(rot=144),
                dict(rot=-16), dict(rope_len=0), dict(pos0=-1), dict(pos0=BIG), dict(ks=6146), dict(ks=1020), dict(vs=0),
                dict(qs=4092), dict(qs=-6144), dict(ks=1 << 41), dict(dt=spin.SPIN_F16, ks=6148), dict(T=1 << 27), dict(T=BIG, Hq=BIG, qs=1 << 39)):
        assert call(**bad) == spin.SPIN_ERR_BAD_SHAPE, bad
    for name in ("Q", "K", "V", "qn", "kn", "rope", "kc", "ksc", "vc", "vsc", "q_start", "kv_len", "table", "out"):
        assert call(**{name: U}) == spin.SPIN_ERR_MISALIGNED, name


ATTN = dict(Q=A, T=0, Hq=32, Hkv=8, D=128, bits=4, kc=A, ks=A, vc=A, vs=A, n_pages=10, page=16, B=4, q_start=A, kv_len=A, table=A,
            max_pages=5, scale=0.1, cap=0.0, slopes=A, window=0, causal=1, bidir=A, O=A, ws=A, ws_bytes=1 << 30, st=None)


@pytest.mark.parametrize("shared", [False, True])
def test_attention(lib, shared):
    ok, f = ATTN, lib.spin_kv_attn
    if shared:
        head = list(ATTN.items())
        ok, f = dict(head[:12] + [("prefix", A), ("prefix_len", 50)] + head[12:]), lib.spin_kv_attn_shared
    call = caller(f, ok)
    assert call() == spin.SPIN_OK and call(T=5, B=0) == spin.SPIN_OK
    assert call(slopes=None, bidir=None, ws=None, ws_bytes=0) == spin.SPIN_OK
    for name in ("Q", "kc", "ks", "vc", "vs", "q_start", "kv_len", "table", "O"):
        assert call(**{name: None}) == spin.SPIN_ERR_NULL, name
    for bad in (dict(bits=6), dict(causal=2), dict(causal=-1), dict(scale=float("nan")), dict(scale=float("-inf")), dict(cap=-1.0),
                dict(cap=float("inf")), dict(cap=float("nan"))):
        assert call(**bad) == spin.SPIN_ERR_UNSUPPORTED, bad
    for bad in (dict(T=-1), dict(D=127), dict(Hq=0), dict(Hq=31), dict(Hq=-8), dict(Hkv=0), dict(B=-1), dict(n_pages=0), dict(page=8),
                dict(page=48), dict(page=2048), dict(max_pages=0), dict(max_pages=1 << 26), dict(window=-1), dict(T=BIG),
                dict(T=4, B=1 << 24), dict(Hq=1 << 20, Hkv=1 << 17, T=1)):
        assert call(**bad) == spin.SPIN_ERR_BAD_SHAPE, bad
    for name in ("Q", "kc", "ks", "vc", "vs", "q_start", "kv_len", "table", "slopes", "bidir", "O", "ws"):
        assert call(**{name: U}) == spin.SPIN_ERR_MISALIGNED, name
    # a single token over a long table is split, and needs its workspace
    long = dict(T=1, B=1, max_pages=4096)
    assert call(**long, ws=None) == spin.SPIN_ERR_NULL
    assert call(**long, ws_bytes=16) == spin.SPIN_ERR_BAD_SHAPE
    if shared:
        assert call(prefix=None) == spin.SPIN_ERR_NULL
        assert call(prefix=None, prefix_len=0) == spin.SPIN_OK
        assert call(prefix=U) == spin.SPIN_ERR_MISALIGNED
        assert call(prefix_len=-1) == call(prefix_len=BIG) == spin.SPIN_ERR_BAD_SHAPE


def test_workspace(lib):
    n = ctypes.c_size_t(7)
    call = caller(lib.spin_kv_attn_workspace, dict(T=1, Hq=32, Hkv=8, B=1, max_pages=4096, page=16, prefix=0, out=ctypes.byref(n)))
    assert call() == spin.SPIN_OK and n.value >= 2 * 32 * 130 * 4
    split = n.value
    assert call(prefix=1 << 20) == spin.SPIN_OK and n.value > split
    assert call(max_pages=1) == spin.SPIN_OK and n.value == 0
    assert call(T=0) == spin.SPIN_OK and n.value == 0
    assert call(out=None) == spin.SPIN_ERR_NULL
    for bad in (dict(T=-1), dict(Hq=31), dict(Hkv=0), dict(B=-1), dict(max_pages=0), dict(page=7), dict(prefix=-1), dict(T=BIG)):
        assert call(**bad) == spin.SPIN_ERR_BAD_SHAPE, bad


def test_the_binding_checks_before_the_library(lib):
    with pytest.raises(ValueError):
        spin.kv_cache(4, 2, 16, 3, device="cpu")
    with pytest.raises(ValueError):
        spin.kv_cache(4, 2, 24, 4, device="cpu")
    c = spin.kv_cache(4, 2, 16, 8, device="cpu")
    assert c["K_codes"].shape == (4, 2, 16, 128) and c["V_codes"].shape == (4, 2, 4, 16, 4, 8)
    with pytest.raises(TypeError):
        spin.spin_kv_attn(None, c, None, None, None)
    with pytest.raises(ValueError):
        spin.spin_kv_attn(c["K_scale"], c, None, None, None)


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
    out = _run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider", os.path.join("tests", "test_abi_paged_cpu.py")],
               {"LD_PRELOAD": runtime, "SPIN_LIBRARY": library})
    assert " passed" in out and " failed" not in out
