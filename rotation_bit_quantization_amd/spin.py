"""Thin Python binding of the libspin C ABI (ctypes; argument marshalling only).

Every function here checks tensor dtype / device / contiguity, allocates the
outputs it was not given (torch device memory), and calls the C entry point
of the same name on torch's current HIP stream, or on ``stream`` (a torch
stream, or a handle): what the call makes then belongs to that stream, and the
caller orders the stream behind the work on the arguments, and its own work
behind the stream.  All arithmetic happens in the HIP kernels of libspin.so; if
the library is missing this module raises instead of computing anything itself.

Declarations and contracts: include/libspin.h.
"""

import ctypes
import functools
import os

import torch

__all__ = ["SpinError", "load", "library_path", "SPIN_OK", "SPIN_ERR_NULL",
           "SPIN_ERR_BAD_SHAPE", "SPIN_ERR_MISALIGNED", "SPIN_ERR_UNSUPPORTED", "SPIN_ERR_HIP",
           "SPIN_F32", "SPIN_F16", "spin_status_string", "spin_fold_rotation", "spin_fwht_quant",
           "spin_w4a4_gemm", "spin_kv_quant", "spin_fwht_quant8", "spin_w4a8_gemm", "spin_kv_quant8",
           "spin_kv_qkv", "spin_fwht_quant_gemm", "spin_fwht_quant_gemm_noalloc", "spin_fwht_quant_f6", "spin_w4a4_gemm_f6",
           "spin_codes_f6", "spin_w4a4_gemm_f6f6", "f6_bytes", "kv_cache", "spin_rope_table", "spin_kv_append",
           "spin_kv_attn", "spin_kv_attn_shared", "spin_kv_attn_workspace", "SPIN_GEMM_AUTO", "SPIN_GEMM_INT8", "SPIN_GEMM_FP6", "SPIN_GEMM_FP6_SPLITK",
           "EXPORTED_SYMBOLS"]

SPIN_OK, SPIN_ERR_NULL, SPIN_ERR_BAD_SHAPE, SPIN_ERR_MISALIGNED, SPIN_ERR_UNSUPPORTED, \
    SPIN_ERR_HIP = range(6)
SPIN_F32, SPIN_F16 = 0, 1
SPIN_GEMM_AUTO, SPIN_GEMM_INT8, SPIN_GEMM_FP6, SPIN_GEMM_FP6_SPLITK = 0, 1, 2, 3
SPIN_FWHT_QUANT_GEMM_WORKSPACE_WORDS = 1025

EXPORTED_SYMBOLS = ("spin_fold_rotation", "spin_fwht_quant", "spin_w4a4_gemm", "spin_kv_quant",
                    "spin_fwht_quant8", "spin_w4a8_gemm", "spin_kv_quant8", "spin_kv_qkv", "spin_w4a4_gemm_ex",
                    "spin_fwht_quant_gemm", "spin_fwht_quant_gemm_noalloc", "spin_fwht_quant_f6",
                    "spin_w4a4_gemm_f6", "spin_codes_f6", "spin_w4a4_gemm_f6f6", "spin_rope_table", "spin_kv_append",
                    "spin_kv_attn", "spin_kv_attn_shared", "spin_kv_attn_workspace",
                    "spin_status_string", "spin_version")

_HERE = os.path.dirname(os.path.abspath(__file__))
_lib = None


def library_path() -> str:
    """The in-tree libspin.so, or the build SPIN_LIBRARY names (the
    host-sanitized one of the sanitizer tests); there is no other fallback."""
    return os.environ.get("SPIN_LIBRARY") or os.path.join(_HERE, "libspin.so")


class SpinError(RuntimeError):
    """A libspin call returned a non-zero spin_status."""

    def __init__(self, fn, status):
        self.status = status
        super().__init__(f"{fn}: {spin_status_string(status)}")


def load():
    """Load libspin.so (raises OSError with a build hint if it is absent)."""
    global _lib
    if _lib is not None:
        return _lib
    path = library_path()
    if not os.path.exists(path):
        raise OSError(f"{path} is missing: build it with `python -m rotation_bit_quantization_amd.build`")
    lib = ctypes.CDLL(path)
    vp, i = ctypes.c_void_p, ctypes.c_int
    lib.spin_fold_rotation.argtypes = [vp, i, i, vp, i, vp, vp, vp, vp]
    lib.spin_fwht_quant.argtypes = [vp, i, i, i, i, vp, vp, vp, vp]
    lib.spin_w4a4_gemm.argtypes = [vp, vp, vp, vp, i, i, i, vp, vp, vp]
    lib.spin_w4a4_gemm_ex.argtypes = [vp, vp, vp, vp, i, i, i, vp, vp, i, vp]
    lib.spin_fwht_quant_gemm.argtypes = [vp, i, i, i, i, vp, vp, i, vp, vp, vp, vp, vp, vp]
    lib.spin_fwht_quant_gemm_noalloc.argtypes = [vp, i, i, i, i, vp, vp, i, vp, vp, vp, vp, vp]
    lib.spin_fwht_quant_f6.argtypes = [vp, i, i, i, i, vp, vp, vp, vp]
    lib.spin_w4a4_gemm_f6.argtypes = [vp, vp, vp, vp, vp, i, i, i, vp, vp, vp]
    lib.spin_codes_f6.argtypes = [vp, i, i, vp, vp, vp]
    lib.spin_w4a4_gemm_f6f6.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, vp, vp, vp]
    lib.spin_kv_quant.argtypes = [vp, i, i, i, i, i, vp, vp, vp, vp]
    lib.spin_fwht_quant8.argtypes = [vp, i, i, i, i, vp, vp, vp, vp]
    lib.spin_w4a8_gemm.argtypes = [vp, vp, vp, vp, i, i, i, vp, vp, vp]
    lib.spin_kv_quant8.argtypes = [vp, i, i, i, i, i, vp, vp, vp, vp]
    lib.spin_kv_qkv.argtypes = [vp, vp, vp, i, i, i, i, i, i, vp, vp, vp, vp, vp, vp, vp]
    f, q, d, z = ctypes.c_float, ctypes.c_int64, ctypes.c_double, ctypes.c_size_t
    lib.spin_rope_table.argtypes = [vp, i, i, i, d, vp, vp]
    lib.spin_kv_append.argtypes = [vp, vp, vp, i, i, i, i, i, q, q, q, vp, vp, f, vp, i, i, i, i, i, vp, vp, vp, vp, i, i,
                                   i, vp, vp, vp, i, vp, vp]
    cache = [vp, i, i, i, i, i, vp, vp, vp, vp, i, i]
    mask = [f, f, vp, i, i, vp, vp, vp, z, vp]
    lib.spin_kv_attn.argtypes = cache + [i, vp, vp, vp, i] + mask
    lib.spin_kv_attn_shared.argtypes = cache + [vp, i, i, vp, vp, vp, i] + mask
    lib.spin_kv_attn_workspace.argtypes = [i, i, i, i, i, i, i, ctypes.POINTER(z)]
    for name in ("spin_rope_table", "spin_kv_append", "spin_kv_attn", "spin_kv_attn_shared", "spin_kv_attn_workspace"):
        getattr(lib, name).restype = ctypes.c_int
    for name in ("spin_fold_rotation", "spin_fwht_quant", "spin_w4a4_gemm", "spin_kv_quant",
                 "spin_fwht_quant8", "spin_w4a8_gemm", "spin_kv_quant8", "spin_kv_qkv", "spin_w4a4_gemm_ex", "spin_fwht_quant_gemm",
                 "spin_fwht_quant_gemm_noalloc", "spin_fwht_quant_f6", "spin_w4a4_gemm_f6"):
        getattr(lib, name).restype = ctypes.c_int
    lib.spin_status_string.argtypes = [ctypes.c_int]
    lib.spin_status_string.restype = ctypes.c_char_p
    lib.spin_version.argtypes = []
    lib.spin_version.restype = ctypes.c_int
    _lib = lib
    return lib


def spin_status_string(status: int) -> str:
    return load().spin_status_string(int(status)).decode()


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_cur_device = getattr(torch._C, "_cuda_getDevice", None)


def _stream(stream=None):
    """The hipStream_t to launch on, as an integer: torch's current stream on the
    current device unless one is given."""
    if stream is None:
        if _raw_stream is not None and _cur_device is not None:
            return _raw_stream(_cur_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _on_stream(stream, of, call, *args, **kw):
    """call(*args, **kw) with ``stream`` (a torch stream, or a handle) as torch's current one, on the GPU that ``of`` lives
    on.  Tensors made for the call then come from memory of that stream: memory of the stream that was current may
    still be in use by work queued there, which nothing orders ``stream`` behind.  Those that the call returns are kept
    from reuse until what the caller's stream has queued on them is done."""
    if not (isinstance(of, torch.Tensor) and of.is_cuda):
        return call(*args, **kw)              # raises, and names what is wrong
    dev = of.get_device()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=dev)
    if stream.device.index != dev:
        raise ValueError(f"{call.__name__}: a stream of {stream.device} for tensors on GPU {dev}")
    here = torch.cuda.current_stream(dev)
    with torch.cuda.stream(stream):
        res = call(*args, **kw)
    given = {id(t) for a in (*args, *kw.values()) for t in (a.values() if isinstance(a, dict) else (a,))}
    for t in res.values() if isinstance(res, dict) else res if isinstance(res, tuple) else (res,):
        if isinstance(t, torch.Tensor) and id(t) not in given:
            t.record_stream(here)
    return res


def _int(x, name):
    """x as a C int takes it; ctypes would drop the bits above."""
    x = int(x)
    if not -2 ** 31 <= x < 2 ** 31:
        raise ValueError(f"{name} is {x}, beyond 32 bits")
    return x


def _ptr(t):
    return None if t is None else t.data_ptr()


def _check(t, name, dtypes, shape=None):
    """Raise unless t is a contiguous GPU tensor of one of `dtypes` (and `shape`)."""
    try:
        if t.is_cuda and t.dtype in dtypes and (shape is None or t.shape == shape) and t.is_contiguous():
            return
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must live on the GPU (got {t.device})")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _raise(fn, status):
    if status != SPIN_OK:
        raise SpinError(fn, status)


def _dtype_code(t):
    return SPIN_F16 if t.dtype == torch.float16 else SPIN_F32


def spin_fold_rotation(W, R, r_block, W_rot=None, Wq=None, w_scale=None, stream=None):
    """W [K, N] fp32, R [r, r] fp32 or None -> (W_rot [K, N] fp32, Wq [N, K/2] u8, w_scale [N] fp32)."""
    if stream is not None:
        return _on_stream(stream, W, spin_fold_rotation, W, R, r_block, W_rot, Wq, w_scale)
    _check(W, "W", (torch.float32,))
    K, N = W.shape
    if R is not None:
        _check(R, "R", (torch.float32,), (r_block, r_block))
    dev = W.device
    W_rot = torch.empty((K, N), dtype=torch.float32, device=dev) if W_rot is None else W_rot
    Wq = torch.empty((N, K // 2), dtype=torch.uint8, device=dev) if Wq is None else Wq
    w_scale = torch.empty((N,), dtype=torch.float32, device=dev) if w_scale is None else w_scale
    _check(W_rot, "W_rot", (torch.float32,), (K, N))
    _check(Wq, "Wq", (torch.uint8,), (N, K // 2))
    _check(w_scale, "w_scale", (torch.float32,), (N,))
    st = load().spin_fold_rotation(_ptr(W), K, N, _ptr(R), _int(r_block, "r_block"), _ptr(W_rot), _ptr(Wq),
                                   _ptr(w_scale), _stream())
    _raise("spin_fold_rotation", st)
    return W_rot, Wq, w_scale


def spin_fwht_quant(X, had_n, Xq=None, x_scale=None, X_rot=None, want_rot=False, stream=None):
    """X [M, K] fp16/fp32 -> (Xq [M, K/2] u8, x_scale [M] fp32, X_rot [M, K] fp32 or None)."""
    if stream is not None:
        return _on_stream(stream, X, spin_fwht_quant, X, had_n, Xq, x_scale, X_rot, want_rot)
    _check(X, "X", (torch.float16, torch.float32))
    M, K = X.shape
    dev = X.device
    Xq = torch.empty((M, K // 2), dtype=torch.uint8, device=dev) if Xq is None else Xq
    x_scale = torch.empty((M,), dtype=torch.float32, device=dev) if x_scale is None else x_scale
    if X_rot is None and want_rot:
        X_rot = torch.empty((M, K), dtype=torch.float32, device=dev)
    _check(Xq, "Xq", (torch.uint8,), (M, K // 2))
    _check(x_scale, "x_scale", (torch.float32,), (M,))
    if X_rot is not None:
        _check(X_rot, "X_rot", (torch.float32,), (M, K))
    st = load().spin_fwht_quant(_ptr(X), _dtype_code(X), M, K, _int(had_n, "had_n"), _ptr(Xq), _ptr(x_scale),
                                _ptr(X_rot), _stream())
    _raise("spin_fwht_quant", st)
    return Xq, x_scale, X_rot


def spin_w4a4_gemm(Xq, x_scale, Wq, w_scale, Y=None, acc_out=None, want_acc=False, kernel=None,
                   stream=None):
    """Packed Xq [M, K/2], Wq [N, K/2] + scales -> (Y [M, N] fp32, acc [M, N] int32 or None).

    ``kernel`` (SPIN_GEMM_INT8 / SPIN_GEMM_FP6 / SPIN_GEMM_FP6_SPLITK) names the kernel family through
    spin_w4a4_gemm_ex; None leaves the choice to the library."""
    if stream is not None:
        return _on_stream(stream, Xq, spin_w4a4_gemm, Xq, x_scale, Wq, w_scale, Y, acc_out, want_acc, kernel)
    _check(Xq, "Xq", (torch.uint8,))
    _check(Wq, "Wq", (torch.uint8,))
    M, Kh = Xq.shape
    N, Kh2 = Wq.shape
    if Kh != Kh2:
        raise ValueError("Xq and Wq disagree on K")
    _check(x_scale, "x_scale", (torch.float32,), (M,))
    _check(w_scale, "w_scale", (torch.float32,), (N,))
    dev = Xq.device
    Y = torch.empty((M, N), dtype=torch.float32, device=dev) if Y is None else Y
    if acc_out is None and want_acc:
        acc_out = torch.empty((M, N), dtype=torch.int32, device=dev)
    _check(Y, "Y", (torch.float32,), (M, N))
    if acc_out is not None:
        _check(acc_out, "acc_out", (torch.int32,), (M, N))
    if kernel is None:
        st = load().spin_w4a4_gemm(_ptr(Xq), _ptr(x_scale), _ptr(Wq), _ptr(w_scale), M, N, 2 * Kh,
                                   _ptr(Y), _ptr(acc_out), _stream())
        _raise("spin_w4a4_gemm", st)
    else:
        st = load().spin_w4a4_gemm_ex(_ptr(Xq), _ptr(x_scale), _ptr(Wq), _ptr(w_scale), M, N, 2 * Kh,
                                      _ptr(Y), _ptr(acc_out), _int(kernel, "kernel"), _stream())
        _raise("spin_w4a4_gemm_ex", st)
    return Y, acc_out


def f6_bytes(M, K):
    """Bytes of an [M][K] activation code matrix in the FP6 operand layout."""
    return ((M + 31) // 32) * (K // 64) * 1536


def spin_fwht_quant_f6(X, Xf6=None, x_sum=None, x_scale=None, stream=None, had_n=12288):
    """X [M, K] -> (Xf6 uint8 [f6_bytes(M, K)], x_sum [M] int32, x_scale [M] fp32).

    had_n = 12288: X fp16 [M, 12288], the R4 Hadamard first; had_n = 1: X fp16 / fp32, quantized as given."""
    if stream is not None:
        return _on_stream(stream, X, spin_fwht_quant_f6, X, Xf6, x_sum, x_scale, had_n=had_n)
    _check(X, "X", (torch.float16,) if had_n == 12288 else (torch.float16, torch.float32))
    M, K = X.shape
    dev = X.device
    Xf6 = torch.empty((f6_bytes(M, K),), dtype=torch.uint8, device=dev) if Xf6 is None else Xf6
    x_sum = torch.empty((M,), dtype=torch.int32, device=dev) if x_sum is None else x_sum
    x_scale = torch.empty((M,), dtype=torch.float32, device=dev) if x_scale is None else x_scale
    _check(Xf6, "Xf6", (torch.uint8,), (f6_bytes(M, K),))
    _check(x_sum, "x_sum", (torch.int32,), (M,))
    _check(x_scale, "x_scale", (torch.float32,), (M,))
    st = load().spin_fwht_quant_f6(_ptr(X), _dtype_code(X), M, K, _int(had_n, "had_n"), _ptr(Xf6), _ptr(x_sum),
                                   _ptr(x_scale), _stream())
    _raise("spin_fwht_quant_f6", st)
    return Xf6, x_sum, x_scale


def spin_w4a4_gemm_f6(Xf6, x_sum, x_scale, Wq, w_scale, Y=None, acc_out=None, want_acc=False, stream=None):
    """Activation codes in the FP6 operand layout (+ row sums, scales) x packed Wq [N, K/2]
    -> (Y [M, N] fp32, acc [M, N] int32 or None)."""
    if stream is not None:
        return _on_stream(stream, x_sum, spin_w4a4_gemm_f6, Xf6, x_sum, x_scale, Wq, w_scale, Y, acc_out,
                          want_acc)
    _check(x_sum, "x_sum", (torch.int32,))
    M = x_sum.shape[0]
    _check(Wq, "Wq", (torch.uint8,))
    N, Kh = Wq.shape
    K = 2 * Kh
    _check(Xf6, "Xf6", (torch.uint8,), (f6_bytes(M, K),))
    _check(x_scale, "x_scale", (torch.float32,), (M,))
    _check(w_scale, "w_scale", (torch.float32,), (N,))
    dev = Wq.device
    Y = torch.empty((M, N), dtype=torch.float32, device=dev) if Y is None else Y
    if acc_out is None and want_acc:
        acc_out = torch.empty((M, N), dtype=torch.int32, device=dev)
    _check(Y, "Y", (torch.float32,), (M, N))
    if acc_out is not None:
        _check(acc_out, "acc_out", (torch.int32,), (M, N))
    st = load().spin_w4a4_gemm_f6(_ptr(Xf6), _ptr(x_sum), _ptr(x_scale), _ptr(Wq), _ptr(w_scale), M, N, K,
                                  _ptr(Y), _ptr(acc_out), _stream())
    _raise("spin_w4a4_gemm_f6", st)
    return Y, acc_out


def spin_codes_f6(Wq, Wf6=None, w_sum=None, stream=None):
    """Packed codes [N, K/2] (weights, or activations) -> (uint8 [f6_bytes(N, K)], row sums [N] int32):
    the codes in the FP6 operand layout, for spin_w4a4_gemm_f6f6."""
    if stream is not None:
        return _on_stream(stream, Wq, spin_codes_f6, Wq, Wf6, w_sum)
    _check(Wq, "Wq", (torch.uint8,))
    N, Kh = Wq.shape
    K = 2 * Kh
    dev = Wq.device
    Wf6 = torch.empty((f6_bytes(N, K),), dtype=torch.uint8, device=dev) if Wf6 is None else Wf6
    w_sum = torch.empty((N,), dtype=torch.int32, device=dev) if w_sum is None else w_sum
    _check(Wf6, "Wf6", (torch.uint8,), (f6_bytes(N, K),))
    _check(w_sum, "w_sum", (torch.int32,), (N,))
    st = load().spin_codes_f6(_ptr(Wq), N, K, _ptr(Wf6), _ptr(w_sum), _stream())
    _raise("spin_codes_f6", st)
    return Wf6, w_sum


def spin_w4a4_gemm_f6f6(Xf6, x_sum, x_scale, Wf6, w_sum, w_scale, K, Y=None, acc_out=None, want_acc=False,
                        stream=None):
    """Both operands in the FP6 operand layout (+ code sums, scales) -> (Y [M, N] fp32, acc [M, N] int32
    or None).  K is the reduction length (the layouts do not carry it)."""
    if stream is not None:
        return _on_stream(stream, x_sum, spin_w4a4_gemm_f6f6, Xf6, x_sum, x_scale, Wf6, w_sum, w_scale, K, Y,
                          acc_out, want_acc)
    _check(x_sum, "x_sum", (torch.int32,))
    _check(w_sum, "w_sum", (torch.int32,))
    M, N = x_sum.shape[0], w_sum.shape[0]
    _check(Xf6, "Xf6", (torch.uint8,), (f6_bytes(M, K),))
    _check(Wf6, "Wf6", (torch.uint8,), (f6_bytes(N, K),))
    _check(x_scale, "x_scale", (torch.float32,), (M,))
    _check(w_scale, "w_scale", (torch.float32,), (N,))
    dev = Wf6.device
    Y = torch.empty((M, N), dtype=torch.float32, device=dev) if Y is None else Y
    if acc_out is None and want_acc:
        acc_out = torch.empty((M, N), dtype=torch.int32, device=dev)
    _check(Y, "Y", (torch.float32,), (M, N))
    if acc_out is not None:
        _check(acc_out, "acc_out", (torch.int32,), (M, N))
    st = load().spin_w4a4_gemm_f6f6(_ptr(Xf6), _ptr(x_sum), _ptr(x_scale), _ptr(Wf6), _ptr(w_sum), _ptr(w_scale),
                                    M, N, _int(K, "K"), _ptr(Y), _ptr(acc_out), _stream())
    _raise("spin_w4a4_gemm_f6f6", st)
    return Y, acc_out


_workspaces = {}


def fused_workspace(device):
    """The zero-initialised workspace spin_fwht_quant_gemm needs, one per device
    (each call leaves it zero; calls sharing it must not overlap)."""
    dev = torch.device(device)
    key = (dev.type, dev.index if dev.index is not None else torch.cuda.current_device())
    ws = _workspaces.get(key)
    if ws is None:
        ws = torch.zeros(SPIN_FWHT_QUANT_GEMM_WORKSPACE_WORDS, dtype=torch.int32, device=dev)
        _workspaces[key] = ws
    return ws


def spin_fwht_quant_gemm(X, Wq, w_scale, Xq=None, x_scale=None, Y=None, acc_out=None, want_acc=False,
                         workspace=None, stream=None):
    """X [M, 12288] fp16 (R4 = H_12288 applied online) and the folded Wq [N, 6144], w_scale [N]
    -> (Y [M, N] fp32, Xq [M, 6144] u8, x_scale [M] fp32, acc [M, N] int32 or None), one launch."""
    if stream is not None:
        return _on_stream(stream, X, spin_fwht_quant_gemm, X, Wq, w_scale, Xq, x_scale, Y, acc_out, want_acc,
                          workspace)
    _check(X, "X", (torch.float16,))
    _check(Wq, "Wq", (torch.uint8,))
    M, K = X.shape
    N = Wq.shape[0]
    _check(Wq, "Wq", (torch.uint8,), (N, K // 2))
    _check(w_scale, "w_scale", (torch.float32,), (N,))
    dev = X.device
    Xq = torch.empty((M, K // 2), dtype=torch.uint8, device=dev) if Xq is None else Xq
    x_scale = torch.empty((M,), dtype=torch.float32, device=dev) if x_scale is None else x_scale
    Y = torch.empty((M, N), dtype=torch.float32, device=dev) if Y is None else Y
    if acc_out is None and want_acc:
        acc_out = torch.empty((M, N), dtype=torch.int32, device=dev)
    _check(Xq, "Xq", (torch.uint8,), (M, K // 2))
    _check(x_scale, "x_scale", (torch.float32,), (M,))
    _check(Y, "Y", (torch.float32,), (M, N))
    if acc_out is not None:
        _check(acc_out, "acc_out", (torch.int32,), (M, N))
    ws = fused_workspace(dev) if workspace is None else workspace
    _check(ws, "workspace", (torch.int32,), (SPIN_FWHT_QUANT_GEMM_WORKSPACE_WORDS,))
    st = load().spin_fwht_quant_gemm(_ptr(X), SPIN_F16, M, K, K, _ptr(Wq), _ptr(w_scale), N, _ptr(Xq),
                                     _ptr(x_scale), _ptr(Y), _ptr(acc_out), _ptr(ws), _stream())
    _raise("spin_fwht_quant_gemm", st)
    return Y, Xq, x_scale, acc_out


def spin_fwht_quant_gemm_noalloc(X, Wq, w_scale, Xq, x_scale, Y, acc_out=None, stream=None):
    """spin_fwht_quant_gemm into caller-given outputs, with the library's own flags:
    the call allocates nothing (every tensor is passed in)."""
    _check(X, "X", (torch.float16,))
    M, K = X.shape
    N = Wq.shape[0]
    _check(Wq, "Wq", (torch.uint8,), (N, K // 2))
    _check(w_scale, "w_scale", (torch.float32,), (N,))
    _check(Xq, "Xq", (torch.uint8,), (M, K // 2))
    _check(x_scale, "x_scale", (torch.float32,), (M,))
    _check(Y, "Y", (torch.float32,), (M, N))
    if acc_out is not None:
        _check(acc_out, "acc_out", (torch.int32,), (M, N))
    st = load().spin_fwht_quant_gemm_noalloc(_ptr(X), SPIN_F16, M, K, K, _ptr(Wq), _ptr(w_scale), N, _ptr(Xq),
                                             _ptr(x_scale), _ptr(Y), _ptr(acc_out), _stream(stream))
    _raise("spin_fwht_quant_gemm_noalloc", st)
    return Y, Xq, x_scale, acc_out


def spin_kv_quant(X, rotate, quantize=True, codes=None, scale=None, X_rot=None, want_rot=False,
                  stream=None):
    """X [T, H, 128] fp16/fp32 -> (codes [T, H, 64] u8 | None, scale [T, H] fp16 | None, X_rot | None).

    ``scale`` is returned as a float16 tensor holding the fp16 bit patterns the
    library writes.
    """
    if stream is not None:
        return _on_stream(stream, X, spin_kv_quant, X, rotate, quantize, codes, scale, X_rot, want_rot)
    _check(X, "X", (torch.float16, torch.float32))
    T, H, D = X.shape
    dev = X.device
    if quantize:
        codes = torch.empty((T, H, D // 2), dtype=torch.uint8, device=dev) if codes is None else codes
        scale = torch.empty((T, H), dtype=torch.float16, device=dev) if scale is None else scale
        _check(codes, "codes", (torch.uint8,), (T, H, D // 2))
        _check(scale, "scale", (torch.float16,), (T, H))
    if X_rot is None and (want_rot or not quantize):
        X_rot = torch.empty((T, H, D), dtype=torch.float32, device=dev)
    if X_rot is not None:
        _check(X_rot, "X_rot", (torch.float32,), (T, H, D))
    st = load().spin_kv_quant(_ptr(X), _dtype_code(X), T, H, D, _int(rotate, "rotate"), _ptr(codes),
                              _ptr(scale), _ptr(X_rot), _stream())
    _raise("spin_kv_quant", st)
    return codes, scale, X_rot


# ---------------------------------------------------------------- W4A8KV8 variant

def spin_fwht_quant8(X, had_n, Xq8=None, x_scale=None, X_rot=None, want_rot=False, stream=None):
    """X [M, K] fp16/fp32 -> (Xq8 [M, K] int8, x_scale [M] fp32, X_rot [M, K] fp32 or None)."""
    if stream is not None:
        return _on_stream(stream, X, spin_fwht_quant8, X, had_n, Xq8, x_scale, X_rot, want_rot)
    _check(X, "X", (torch.float16, torch.float32))
    M, K = X.shape
    dev = X.device
    Xq8 = torch.empty((M, K), dtype=torch.int8, device=dev) if Xq8 is None else Xq8
    x_scale = torch.empty((M,), dtype=torch.float32, device=dev) if x_scale is None else x_scale
    if X_rot is None and want_rot:
        X_rot = torch.empty((M, K), dtype=torch.float32, device=dev)
    _check(Xq8, "Xq8", (torch.int8,), (M, K))
    _check(x_scale, "x_scale", (torch.float32,), (M,))
    if X_rot is not None:
        _check(X_rot, "X_rot", (torch.float32,), (M, K))
    st = load().spin_fwht_quant8(_ptr(X), _dtype_code(X), M, K, _int(had_n, "had_n"), _ptr(Xq8), _ptr(x_scale),
                                 _ptr(X_rot), _stream())
    _raise("spin_fwht_quant8", st)
    return Xq8, x_scale, X_rot


def spin_w4a8_gemm(Xq8, x_scale, Wq, w_scale, Y=None, acc_out=None, want_acc=False, stream=None):
    """Int8 Xq8 [M, K], packed Wq [N, K/2] + scales -> (Y [M, N] fp32, acc [M, N] int32 or None)."""
    if stream is not None:
        return _on_stream(stream, Xq8, spin_w4a8_gemm, Xq8, x_scale, Wq, w_scale, Y, acc_out, want_acc)
    _check(Xq8, "Xq8", (torch.int8,))
    _check(Wq, "Wq", (torch.uint8,))
    M, K = Xq8.shape
    N, Kh = Wq.shape
    if K != 2 * Kh:
        raise ValueError("Xq8 and Wq disagree on K")
    _check(x_scale, "x_scale", (torch.float32,), (M,))
    _check(w_scale, "w_scale", (torch.float32,), (N,))
    dev = Xq8.device
    Y = torch.empty((M, N), dtype=torch.float32, device=dev) if Y is None else Y
    if acc_out is None and want_acc:
        acc_out = torch.empty((M, N), dtype=torch.int32, device=dev)
    _check(Y, "Y", (torch.float32,), (M, N))
    if acc_out is not None:
        _check(acc_out, "acc_out", (torch.int32,), (M, N))
    st = load().spin_w4a8_gemm(_ptr(Xq8), _ptr(x_scale), _ptr(Wq), _ptr(w_scale), M, N, K,
                               _ptr(Y), _ptr(acc_out), _stream())
    _raise("spin_w4a8_gemm", st)
    return Y, acc_out


def spin_kv_quant8(X, rotate, quantize=True, codes=None, scale=None, X_rot=None, want_rot=False,
                   stream=None):
    """X [T, H, 128] fp16/fp32 -> (codes [T, H, 128] int8 | None, scale [T, H] fp16 | None, X_rot | None)."""
    if stream is not None:
        return _on_stream(stream, X, spin_kv_quant8, X, rotate, quantize, codes, scale, X_rot, want_rot)
    _check(X, "X", (torch.float16, torch.float32))
    T, H, D = X.shape
    dev = X.device
    if quantize:
        codes = torch.empty((T, H, D), dtype=torch.int8, device=dev) if codes is None else codes
        scale = torch.empty((T, H), dtype=torch.float16, device=dev) if scale is None else scale
        _check(codes, "codes", (torch.int8,), (T, H, D))
        _check(scale, "scale", (torch.float16,), (T, H))
    if X_rot is None and (want_rot or not quantize):
        X_rot = torch.empty((T, H, D), dtype=torch.float32, device=dev)
    if X_rot is not None:
        _check(X_rot, "X_rot", (torch.float32,), (T, H, D))
    st = load().spin_kv_quant8(_ptr(X), _dtype_code(X), T, H, D, _int(rotate, "rotate"), _ptr(codes),
                               _ptr(scale), _ptr(X_rot), _stream())
    _raise("spin_kv_quant8", st)
    return codes, scale, X_rot


def spin_kv_qkv(K, V, Q=None, bits=4, want_k_rot=False, out=None, stream=None):
    """One launch for a layer's KV step: K [T, Hkv, 128] rotated + quantized, V [T, Hkv, 128]
    quantized, Q [T, Hq, 128] (optional) rotated.

    Returns a dict with ``K_codes``, ``K_scale``, ``V_codes``, ``V_scale`` (scales as float16
    tensors holding the fp16 bit patterns), ``Q_rot`` (or None) and ``K_rot`` (or None).
    Codes are [T, Hkv, 64] uint8 at bits=4 and [T, Hkv, 128] int8 at bits=8.  ``out`` may
    hold preallocated tensors under the same names; missing ones are allocated.
    """
    if stream is not None:
        return _on_stream(stream, K, spin_kv_qkv, K, V, Q, bits, want_k_rot, out)
    _check(K, "K", (torch.float16, torch.float32))
    T, Hkv, D = K.shape
    _check(V, "V", (K.dtype,), (T, Hkv, D))
    Hq = 0
    if Q is not None:
        _check(Q, "Q", (K.dtype,))
        if Q.dim() != 3 or Q.shape[0] != T or Q.shape[2] != D:
            raise ValueError(f"Q has shape {tuple(Q.shape)}, expected ({T}, Hq, {D})")
        Hq = Q.shape[1]
    dev = K.device
    if bits == 4:
        cshape, cdtype = (T, Hkv, D // 2), torch.uint8
    elif bits == 8:
        cshape, cdtype = (T, Hkv, D), torch.int8
    else:
        raise ValueError("bits must be 4 or 8")
    want = {
        "K_codes": (cshape, cdtype),
        "K_scale": ((T, Hkv), torch.float16),
        "V_codes": (cshape, cdtype),
        "V_scale": ((T, Hkv), torch.float16),
    }
    if Q is not None:
        want["Q_rot"] = ((T, Hq, D), torch.float32)
    if want_k_rot:
        want["K_rot"] = ((T, Hkv, D), torch.float32)
    given = dict(out or {})
    res = {"Q_rot": None, "K_rot": None}
    for name, (shape, dtype) in want.items():
        t = given.get(name)
        if t is None:
            t = torch.empty(shape, dtype=dtype, device=dev)
        _check(t, name, (dtype,), shape)
        res[name] = t
    st = load().spin_kv_qkv(_ptr(Q), _ptr(K), _ptr(V), _dtype_code(K), T, Hq, Hkv, D, int(bits),
                            _ptr(res["Q_rot"]), _ptr(res["K_codes"]), _ptr(res["K_scale"]),
                            _ptr(res["K_rot"]), _ptr(res["V_codes"]), _ptr(res["V_scale"]), _stream())
    _raise("spin_kv_qkv", st)
    return res


# ---------------------------------------------------------------- the paged KV cache

def _launch(fn, dev, args):
    """Call fn(*args, stream) on GPU number `dev`, on its current stream."""
    call = _entry(fn)
    if _raw_stream is not None and _cur_device is not None and _cur_device() == dev:
        st = call(*args, _raw_stream(dev))
    else:
        with torch.cuda.device(dev):
            st = call(*args, torch.cuda.current_stream().cuda_stream)
    if st != SPIN_OK:
        raise SpinError(fn, st)


@functools.lru_cache(None)
def _entry(fn):
    return getattr(load(), fn)


def _want(t, name, dtype, shape, dev):
    """Raise unless t is a contiguous tensor of this type and shape on GPU `dev`; returns its address."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    _check(t, name, (dtype,), shape)
    raise ValueError(f"{name} lives on {t.device}, the others on GPU {dev}")


def _gpu(t, name):
    """The number of the GPU a tensor lives on."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must live on the GPU (got {t.device})")
    return t.get_device()


def kv_cache(n_pages, Hkv, page_size, bits=4, device="cuda"):
    """An empty pool of cache pages: a dict of ``K_codes`` [n_pages, Hkv, page_size, 16 * bits] and ``V_codes``
    [n_pages, Hkv, page_size / 4, 16, 4, bits] uint8, ``K_scale`` and ``V_scale`` [n_pages, Hkv, page_size] fp16
    (layouts: include/libspin.h)."""
    if bits not in (4, 8):
        raise ValueError("bits must be 4 or 8")
    if page_size < 16 or page_size & (page_size - 1):
        raise ValueError("page_size must be a power of two of at least 16")
    return {"K_codes": torch.zeros((n_pages, Hkv, page_size, 16 * bits), dtype=torch.uint8, device=device),
            "K_scale": torch.zeros((n_pages, Hkv, page_size), dtype=torch.float16, device=device),
            "V_codes": torch.zeros((n_pages, Hkv, page_size // 4, 16, 4, bits), dtype=torch.uint8, device=device),
            "V_scale": torch.zeros((n_pages, Hkv, page_size), dtype=torch.float16, device=device)}


def _cache(cache, dev):
    """Check a cache's four tensors; returns their addresses and (n_pages, Hkv, page_size, bits)."""
    kc = cache["K_codes"]
    if kc.dim() != 4 or kc.shape[3] not in (64, 128):
        raise ValueError(f"K_codes has shape {tuple(kc.shape)}, expected [n_pages, Hkv, page_size, 64 or 128]")
    shape = kc.shape
    n_pages, Hkv, page, width = shape
    bits = width // 16
    ks, vc, vs = cache["K_scale"], cache["V_codes"], cache["V_scale"]
    scale, values, f16, u8 = (n_pages, Hkv, page), (n_pages, Hkv, page // 4, 16, 4, bits), torch.float16, torch.uint8
    # the checks of _want, in one expression: this runs in every call
    if not (kc.dtype is u8 and vc.dtype is u8 and ks.dtype is f16 and vs.dtype is f16 and ks.shape == scale and
            vs.shape == scale and vc.shape == values and kc.get_device() == dev and ks.get_device() == dev and
            vc.get_device() == dev and vs.get_device() == dev and kc.is_contiguous() and ks.is_contiguous() and
            vc.is_contiguous() and vs.is_contiguous()):
        _want(kc, "K_codes", u8, shape, dev)
        _want(ks, "K_scale", f16, scale, dev)
        _want(vc, "V_codes", u8, values, dev)
        _want(vs, "V_scale", f16, scale, dev)
    return (kc.data_ptr(), ks.data_ptr(), vc.data_ptr(), vs.data_ptr()), n_pages, Hkv, page, bits


def _batch(page_table, q_start, kv_len, dev):
    """Check a batch's three arrays; returns the addresses of q_start, kv_len and page_table and (B, max_pages)."""
    if page_table.dim() != 2:
        raise ValueError(f"page_table has shape {tuple(page_table.shape)}, expected [B, max_pages]")
    B, max_pages = page_table.shape
    i32 = torch.int32
    if not (q_start.dtype is i32 and kv_len.dtype is i32 and page_table.dtype is i32 and q_start.shape == (B + 1,) and
            kv_len.shape == (B,) and B | max_pages < 2 ** 31 and q_start.get_device() == dev and kv_len.get_device() == dev and
            page_table.get_device() == dev and q_start.is_contiguous() and kv_len.is_contiguous() and page_table.is_contiguous()):
        _want(q_start, "q_start", i32, (B + 1,), dev)
        _want(kv_len, "kv_len", i32, (B,), dev)
        _want(page_table, "page_table", i32, (B, max_pages), dev)
        _int(B, "B")
        _int(max_pages, "max_pages")
    return (q_start.data_ptr(), kv_len.data_ptr(), page_table.data_ptr()), B, max_pages


def _rows(x, name, dtype, T, dev):
    """Check [T, H, 128] rows whose heads lie beside each other; returns (address, H, values from a token to the
    next)."""
    if not isinstance(x, torch.Tensor) or x.dim() != 3:
        raise ValueError(f"{name} must be a [{T}, H, 128] tensor")
    rows, H, D = x.shape
    per_token, per_head, per_value = x.stride()
    if not (rows == T and D == 128 and x.get_device() == dev and x.dtype is dtype and per_head == 128 and per_value == 1):
        if rows != T or D != 128:
            raise ValueError(f"{name} has shape {tuple(x.shape)}, expected [{T}, H, 128]")
        if x.get_device() != dev:
            raise ValueError(f"{name} lives on {x.device}, the others on GPU {dev}")
        if x.dtype is not dtype:
            raise TypeError(f"{name} has dtype {x.dtype}, expected {dtype}, the same for all")
        if T and H and (per_value != 1 or (H > 1 and per_head != 128)):
            raise ValueError(f"{name}: the heads of a token must lie beside each other (strides {x.stride()})")
    return x.data_ptr(), H, per_token if T > 1 else max(128 * H, 128)


def spin_rope_table(inv_freq, n_pos, pos0=0, attn_scale=1.0, table=None, stream=None):
    """inv_freq [n] float64 -> table [n_pos, 2 n] fp32: n cosines, then n sines of (pos0 + p) * inv_freq."""
    if stream is not None:
        return _on_stream(stream, inv_freq, spin_rope_table, inv_freq, n_pos, pos0, attn_scale, table)
    dev = _gpu(inv_freq, "inv_freq")
    if inv_freq.dim() != 1:
        raise ValueError(f"inv_freq has shape {tuple(inv_freq.shape)}, expected [n]")
    n, n_pos = _int(inv_freq.shape[0], "n"), _int(n_pos, "n_pos")
    freq = _want(inv_freq, "inv_freq", torch.float64, (n,), dev)
    if table is None:
        table = torch.empty((n_pos, 2 * n), dtype=torch.float32, device=inv_freq.device)
    out = _want(table, "table", torch.float32, (n_pos, 2 * n), dev)
    if n_pos != 0:                  # an empty tensor has no address to pass
        _launch("spin_rope_table", dev, (freq, n, _int(pos0, "pos0"), n_pos, float(attn_scale), out))
    return table


def spin_kv_append(Q, K, V, cache, page_table, q_start, kv_len, rope=None, interleaved=False, q_norm=None, k_norm=None,
                   eps=1e-6, pos0=0, Q_out=None, stream=None):
    """Rows of qkv_proj (Q [T, Hq, 128] or None, K and V [T, Hkv, 128], fp16 / fp32, views of one product are
    fine) -> Q_out [T, Hq, 128] fp16 (or None); the codes of K and V go into the pages of ``cache``.

    ``rope`` is a spin_rope_table of the rotated part of a head; ``q_norm`` and ``k_norm`` are [128] fp32 weights."""
    if stream is not None:
        return _on_stream(stream, K, spin_kv_append, Q, K, V, cache, page_table, q_start, kv_len, rope,
                          interleaved, q_norm, k_norm, eps, pos0, Q_out)
    dev = _gpu(K, "K")
    (kc, ks, vc, vs), n_pages, Hkv, page, bits = _cache(cache, dev)
    (starts, lens, table), B, max_pages = _batch(page_table, q_start, kv_len, dev)
    T, dtype = K.shape[0], K.dtype
    if dtype is not torch.float16 and dtype is not torch.float32:
        raise TypeError(f"K has dtype {dtype}, expected float16 or float32")
    k, hk, k_stride = _rows(K, "K", dtype, T, dev)
    v, hv, v_stride = _rows(V, "V", dtype, T, dev)
    if hk != Hkv or hv != Hkv:
        raise ValueError(f"K has {hk} and V {hv} heads, the cache {Hkv}")
    q = out = None
    Hq, q_stride = 0, 0
    if Q is not None:
        q, Hq, q_stride = _rows(Q, "Q", dtype, T, dev)
        if Q_out is None:
            Q_out = Q.new_empty((T, Hq, 128), dtype=torch.float16)
            out = Q_out.data_ptr()
        else:
            out = _want(Q_out, "Q_out", torch.float16, (T, Hq, 128), dev)
    elif Q_out is not None:
        raise ValueError("Q_out without Q")
    qn = None if q_norm is None else _want(q_norm, "q_norm", torch.float32, (128,), dev)
    kn = None if k_norm is None else _want(k_norm, "k_norm", torch.float32, (128,), dev)
    rows, rope_len, rot_dim = None, 0, 0
    if rope is not None:
        if rope.dim() != 2:
            raise ValueError(f"rope has shape {tuple(rope.shape)}, expected [positions, rotated values]")
        rope_len, rot_dim = _int(rope.shape[0], "positions"), _int(rope.shape[1], "rotated values")
        rows = _want(rope, "rope", torch.float32, rope.shape, dev)
    if T != 0 and B != 0:           # an empty tensor has no address to pass
        _launch("spin_kv_append", dev,
                (q, k, v, SPIN_F16 if dtype is torch.float16 else SPIN_F32, T, Hq, Hkv, 128, q_stride, k_stride, v_stride, qn,
                 kn, eps, rows, rope_len, rot_dim, _int(interleaved, "interleaved"), _int(pos0, "pos0"), bits, kc, ks, vc, vs, n_pages, page, B, starts,
                 lens, table, max_pages, out))
    return Q_out


@functools.lru_cache(4096)
def spin_kv_attn_workspace(T, Hq, Hkv, B, max_pages, page_size, prefix_len=0):
    """Bytes of workspace that spin_kv_attn (spin_kv_attn_shared with a prefix) takes at these sizes."""
    for name, x in dict(T=T, Hq=Hq, Hkv=Hkv, B=B, max_pages=max_pages, page_size=page_size, prefix_len=prefix_len).items():
        _int(x, name)
    n = ctypes.c_size_t(0)
    _raise("spin_kv_attn_workspace", load().spin_kv_attn_workspace(T, Hq, Hkv, B, max_pages, page_size, prefix_len,
                                                                   ctypes.byref(n)))
    return n.value


def _attn(fn, Q, cache, prefix, page_table, q_start, kv_len, scale, softcap, slopes, window, causal, bidir_len, O,
          workspace):
    dev = _gpu(Q, "Q")
    (kc, ks, vc, vs), n_pages, Hkv, page, bits = _cache(cache, dev)
    (starts, lens, table), B, max_pages = _batch(page_table, q_start, kv_len, dev)
    shape = Q.shape
    if len(shape) != 3 or shape[2] != 128:
        raise ValueError(f"Q has shape {tuple(shape)}, expected [T, Hq, 128]")
    T, Hq, _ = shape
    q = _want(Q, "Q", torch.float16, shape, dev)
    slope = None if slopes is None else _want(slopes, "slopes", torch.float32, (Hq,), dev)
    both = None if bidir_len is None else _want(bidir_len, "bidir_len", torch.int32, (B,), dev)
    prefix_len, front = 0, ()
    if prefix is not None:
        prefix_len = prefix[1]
        front = (_want(prefix[0], "prefix_table", torch.int32, prefix[0].shape, dev) or None, prefix_len)
    if O is None:
        O = torch.empty_like(Q)
        out = O.data_ptr()
    else:
        out = _want(O, "O", torch.float16, shape, dev)
    if T == 0 or B == 0:            # an empty tensor has no address to pass
        return O
    need = spin_kv_attn_workspace(T, Hq, Hkv, B, max_pages, page, prefix_len)
    ws, ws_bytes = None, 0
    if workspace is not None:
        ws_bytes = workspace.numel()
        ws = _want(workspace, "workspace", torch.uint8, (ws_bytes,), dev)
    elif need:
        workspace = Q.new_empty((need + 1) // 2)
        ws, ws_bytes = workspace.data_ptr(), need
    _launch(fn, dev,
            (q, T, Hq, Hkv, 128, bits, kc, ks, vc, vs, n_pages, page, *front, B, starts, lens, table, max_pages,
             0.08838834764831845 if scale is None else scale, softcap, slope, _int(window, "window"), _int(causal, "causal"), both, out, ws, ws_bytes))
    return O


def spin_kv_attn(Q, cache, page_table, q_start, kv_len, scale=None, softcap=0.0, slopes=None, window=0, causal=True,
                 bidir_len=None, O=None, workspace=None, stream=None):
    """Q [T, Hq, 128] fp16 (from spin_kv_append) over the pages of each sequence -> O [T, Hq, 128] fp16.

    ``scale`` is 1 / sqrt(128) by default.  ``workspace`` (uint8, spin_kv_attn_workspace bytes) is allocated if
    it is not given."""
    if stream is not None:
        return _on_stream(stream, Q, spin_kv_attn, Q, cache, page_table, q_start, kv_len, scale, softcap,
                          slopes, window, causal, bidir_len, O, workspace)
    return _attn("spin_kv_attn", Q, cache, None, page_table, q_start, kv_len, scale, softcap, slopes, window, causal,
                 bidir_len, O, workspace)


def spin_kv_attn_shared(Q, cache, prefix_table, prefix_len, page_table, q_start, kv_len, scale=None, softcap=0.0,
                        slopes=None, window=0, causal=True, bidir_len=None, O=None, workspace=None, stream=None):
    """spin_kv_attn where the first ``prefix_len`` tokens of every sequence lie in the pages ``prefix_table``
    names ([ceil(prefix_len / page_size)] int32) and ``page_table`` and ``kv_len`` count what follows."""
    if stream is not None:
        return _on_stream(stream, Q, spin_kv_attn_shared, Q, cache, prefix_table, prefix_len, page_table,
                          q_start, kv_len, scale, softcap, slopes, window, causal, bidir_len, O, workspace)
    prefix_len = _int(prefix_len, "prefix_len")
    if prefix_table.dim() != 1 or prefix_table.shape[0] < -(-prefix_len // cache["K_codes"].shape[2]):
        raise ValueError(f"prefix_table has shape {tuple(prefix_table.shape)}, too few pages for {prefix_len} tokens")
    return _attn("spin_kv_attn_shared", Q, cache, (prefix_table, prefix_len), page_table, q_start, kv_len, scale,
                 softcap, slopes, window, causal, bidir_len, O, workspace)
