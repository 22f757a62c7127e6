"""Weights of tokens some of which have no prior (spin_kv_weights_ex), without a GPU: its refusals, the binding's call."""

import pytest
import torch

from rotation_bit_quantization_amd import paged, spin

from .test_abi_paged_cpu import A, U, caller
from .test_abi_served_cpu import PAGES, lib, refusals  # noqa: F401
from .test_streams_cpu import seen  # noqa: F401
from .test_streams_served_cpu import calls, gpu


def test_refusals(lib):  # noqa: F811
    at = 1 << 20
    ok = dict(Q=A, lse=A, T=5, Hq=32, Hkv=8, D=128, bits=4, kc=A, ks=A, n_pages=10, page=16, B=0, q_start=A, kv_len=A, table=A, max_pages=5,
              pos0=0, scale=0.1, cap=0.0, slopes=A, window=0, causal=1, bidir=A, prior=A, known=A, decay=1.0, W=A, ws=A, ws_bytes=1 << 30, st=None)
    call = caller(lib.spin_kv_weights_ex, ok)
    assert call() == call(known=None) == call(prior=None) == call(prior=None, known=None) == spin.SPIN_OK
    refusals(call, ("Q", "lse", "kc", "ks", "q_start", "kv_len", "table", "W"), (dict(bits=5), dict(causal=2), dict(decay=float("nan"))),
             (dict(T=-1), dict(Hq=31), dict(pos0=-1)) + PAGES, ("Q", "lse", "prior", "known", "W", "ws"))
    assert call(B=1, prior=at, W=at + 16) == spin.SPIN_ERR_UNSUPPORTED
    assert call(known=U) == spin.SPIN_ERR_MISALIGNED


def test_the_binding_passes_it_on(seen, monkeypatch):  # noqa: F811
    """Behind the prior, and with a stream as without; not without a prior."""
    monkeypatch.setattr(paged, "spin_kv_weights_workspace", lambda *a: 0)
    given = []
    monkeypatch.setattr(paged, "_launch", lambda fn, dev, args: given.append((fn, args)))
    args = dict(calls()["spin_kv_weights"], prior=gpu(torch.zeros((2, 1, 16))))
    known = gpu(torch.zeros((1,), dtype=torch.int32))
    spin.spin_kv_weights(**args)
    spin.spin_kv_weights(**args, prior_len=known)
    spin.spin_kv_weights(**args, prior_len=known, stream=7)
    (fn0, a0), (fn1, a1), (fn2, a2) = given
    assert fn0 == "spin_kv_weights" and fn1 == fn2 == "spin_kv_weights_ex"
    at = [i for i, x in enumerate(a0) if x == args["prior"].data_ptr()][0] + 1
    assert a1[at] == a2[at] == known.data_ptr() and len(a1) == len(a0) + 1 and a1[:at] == a0[:at]
    for bad in (torch.zeros((2,), dtype=torch.int32), torch.zeros((1, 1), dtype=torch.int32)):
        with pytest.raises(ValueError):
            spin.spin_kv_weights(**args, prior_len=gpu(bad))
    with pytest.raises(TypeError):
        spin.spin_kv_weights(**args, prior_len=gpu(torch.zeros((1,))))
    with pytest.raises(ValueError, match="prior"):
        spin.spin_kv_weights(**calls()["spin_kv_weights"], prior_len=known)
