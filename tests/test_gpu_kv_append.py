"""GPU parity of spin_rope_table and spin_kv_append with the float64 oracle: tables within one rounding, the bytes
of the cache equal, queries within the roundings of their float32 path; then a layer's steps together."""

import numpy as np
import pytest
import torch

import oracle
from rotation_bit_quantization_amd import spin

from .paged_case import DEV, close, dev, host, pool, starts, tables

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spin.load()


def frequencies(rot, base=1e4):
    return base ** (-np.arange(rot // 2) / (rot // 2))


@pytest.mark.parametrize("n,pos0,P,scale", [(1, 0, 1, 1.0), (64, 0, 777, 1.0), (16, 1 << 20, 513, 1.1), (33, 12345, 64, -0.5),
                                            (64, (1 << 29) - 40, 40, 1.0), (8, 5, 0, 1.0)])
def test_rope_table(n, pos0, P, scale):
    inv = 1e4 ** (-np.arange(n) / n)
    got = host(spin.spin_rope_table(dev(inv), P, pos0=pos0, attn_scale=scale))
    ref = oracle.rope_table(inv, P, pos0, scale)
    assert got.shape == (P, 2 * n)
    # float64 functions on both sides, each within a few 2^-53; then one rounding to float32
    assert (np.abs(got - ref) <= 2.0 ** -24 * np.abs(ref) + abs(scale) * 2.0 ** -48).all()


def check(rng, q_len, kv_len, Hq, Hkv, bits, page, dtype=np.float32, rot=128, interleaved=False, norm=True, pos0=0, before=0,
          behind=0, one_product=True, table=None, cache=None, loud=30.0, rope_len=None, eps=1e-6):
    q_start = starts(q_len, before)
    T = before + int(sum(q_len)) + behind
    x = rng.standard_normal((T, Hq + 2 * Hkv, 128))
    x[:, :, rng.integers(0, 128, 2)] *= loud
    x = x.astype(dtype)
    n_pages = sum(-(-max(n, 0) // page) for n in kv_len) + 2
    cache = pool(rng, n_pages, Hkv, page, bits) if cache is None else cache
    table = tables(rng, kv_len, page, n_pages) if table is None else table
    room = table.shape[1] * page
    rope = None
    if rot:
        rope = oracle.rope_table(frequencies(rot), (room if rope_len is None else rope_len) + pos0).astype(np.float32)
    w = (1 + 0.3 * rng.standard_normal((2, 128))).astype(np.float32) if norm else (None, None)
    more = dict(interleaved=interleaved, eps=eps, pos0=pos0)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    ref, q_ref = oracle.kv_append(q, k, v, cache, table, q_start, kv_len, rope=rope, q_norm=w[0], k_norm=w[1], **more)
    d = dev(x)
    qd, kd, vd = (d[:, :Hq], d[:, Hq:Hq + Hkv], d[:, Hq + Hkv:]) if one_product else (dev(q), dev(k), dev(v))
    cd = dev(cache)
    Q_out = torch.full((T, Hq, 128), 77.0, dtype=torch.float16, device=DEV)
    spin.spin_kv_append(qd, kd, vd, cd, dev(table), dev(q_start), dev(np.asarray(kv_len, np.int32)), rope=dev(rope),
                        q_norm=dev(w[0]), k_norm=dev(w[1]), Q_out=Q_out, **more)
    for name in ref:
        got = host(cd[name])
        assert np.array_equal(got.view(np.uint8), ref[name].view(np.uint8)), name
    got = host(Q_out).astype(np.float64)
    silent = np.isnan(q_ref)
    assert (got[silent] == 77.0).all()
    # float32: norm factor and weight (3), rotation (3), seven levels and the factor (8): at most 16 roundings of
    # 2^-24, each of a value no larger than sum |x'| / sqrt(128) <= norm of x'; rounding to fp16 half a step
    y = np.where(silent, 0, q_ref)
    size = np.linalg.norm(y, axis=-1, keepdims=True)
    tol = 2.0 ** -11 * np.abs(y) + 2.0 ** -25 + 16 * 2.0 ** -24 * size
    assert (np.abs(got - y)[~silent] <= tol[~silent]).all()


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", [np.float32, np.float16])
@pytest.mark.parametrize("q_len,kv_len,Hq,Hkv,page", [
    ([1], [1], 1, 1, 16), ([1, 1, 1], [17, 1, 64], 4, 2, 16), ([3, 0, 1, 6], [40, 9, 9, 6], 6, 3, 32),
    ([37, 1, 18], [37, 80, 130], 5, 1, 64), ([1] * 40, list(range(1, 41)), 8, 2, 16), ([300], [300], 4, 4, 128)])
def test_shapes(bits, dtype, q_len, kv_len, Hq, Hkv, page):
    rng = np.random.default_rng(bits + Hq + page)
    check(rng, q_len, kv_len, Hq, Hkv, bits, page, dtype=dtype, before=2, behind=3)


@pytest.mark.parametrize("rot", [0, 16, 32, 80, 96, 128])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_rotations_and_norms(rot, interleaved, norm):
    rng = np.random.default_rng(rot + norm)
    check(rng, [9, 1, 4], [30, 44, 4], 4, 2, 4, 16, rot=rot, interleaved=interleaved, norm=norm, pos0=100, one_product=False)
    check(rng, [9, 1, 4], [30, 44, 4], 4, 2, 8, 16, dtype=np.float16, rot=rot, interleaved=interleaved, norm=norm)


def test_many_sequences():
    """More sequences than one level of the search holds, some without rows."""
    rng = np.random.default_rng(21)
    for B in (15, 16, 17, 255, 256, 257, 300):
        q_len = rng.integers(0, 3, B)
        kv_len = [int(n + rng.integers(0, 20)) for n in q_len]
        check(rng, q_len, kv_len, 2, 1, 4, 16, before=1, behind=1)


def test_values_of_every_size():
    rng = np.random.default_rng(22)
    for loud in (0.0, 1e-30, 1e30):
        check(rng, [5], [5], 1, 2, 4, 16, loud=loud, norm=True)
    # a token of zeros: scale 0, codes 0, and a norm that only eps keeps finite
    q_start, kv = dev(starts([2])), dev(np.array([2], np.int32))
    cache = dev(pool(rng, 2, 1, 16, 4))
    z = torch.zeros((2, 1, 128), device=DEV)
    out = spin.spin_kv_append(z, z, z, cache, dev(np.array([[1]], np.int32)), q_start, kv, q_norm=torch.ones(128, device=DEV),
                              k_norm=torch.ones(128, device=DEV))
    assert (host(out) == 0).all() and (host(cache["K_scale"])[1, 0, :2] == 0).all() and (host(cache["K_codes"])[1, 0, :2] == 0).all()
    assert (host(cache["V_codes"])[1, 0, 0, :, :2] == 0).all() and (host(cache["V_codes"])[1, 0, 0, :, 2:] != 0).any()


def test_tokens_without_a_place():
    rng = np.random.default_rng(23)
    # more new tokens than tokens; a kv_len beyond the table; pages that are none of the pool; a table of positions
    # that ends early
    check(rng, [5, 2], [3, 40], 2, 1, 4, 16, table=np.array([[1, 0], [2, 3]], np.int32))
    check(rng, [3, 2], [30, 20], 2, 1, 4, 16, table=np.array([[1, -1], [9, 2 ** 31 - 1]], np.int32))
    check(rng, [4, 6], [20, 21], 2, 1, 8, 16, rope_len=18)


def test_no_queries_and_empty_batches():
    rng = np.random.default_rng(24)
    cache = pool(rng, 3, 2, 16, 4)
    k, v = (rng.standard_normal((4, 2, 128)).astype(np.float16) for _ in "kv")
    table, q_start, kv = np.array([[1, 2]], np.int32), starts([4]), np.array([20], np.int32)
    ref, _ = oracle.kv_append(np.zeros((4, 0, 128)), k, v, cache, table, q_start, kv)
    d = dev(cache)
    assert spin.spin_kv_append(None, dev(k), dev(v), d, dev(table), dev(q_start), dev(kv)) is None
    for name in ref:
        assert np.array_equal(host(d[name]).view(np.uint8), ref[name].view(np.uint8)), name
    none = torch.empty((0, 2, 128), dtype=torch.float16, device=DEV)
    spin.spin_kv_append(None, none, none, d, dev(table), dev(np.zeros(2, np.int32)), dev(kv))
    spin.spin_kv_append(None, dev(k), dev(v), d, torch.zeros((0, 2), dtype=torch.int32, device=DEV),
                        dev(np.zeros(1, np.int32)), torch.zeros(0, dtype=torch.int32, device=DEV))
    for name in ref:
        assert np.array_equal(host(d[name]).view(np.uint8), ref[name].view(np.uint8)), name


def test_without_rotation_values_match_spin_kv_quant():
    """The same codes as the contiguous cache's writer, for values; for keys up to its float32 near-ties."""
    rng = np.random.default_rng(25)
    T, H = 64, 3
    x = dev(rng.standard_normal((T, H, 128)).astype(np.float16))
    cache = spin.kv_cache(4, H, 16, 4)
    spin.spin_kv_append(None, x, x, cache, dev(np.arange(4, dtype=np.int32)[None]), dev(starts([T])), dev(np.array([T], np.int32)))
    for rotate, name in ((1, "K"), (0, "V")):
        codes, scale, _ = spin.spin_kv_quant(x, rotate)
        got = host(cache[name + "_codes"])
        if name == "V":
            got = got.transpose(0, 1, 2, 4, 3, 5).reshape(4, H, 16, 64)
        got = got.transpose(0, 2, 1, 3).reshape(T, H, 64)
        same = np.array_equal(got, host(codes)) and np.array_equal(host(cache[name + "_scale"]).transpose(0, 2, 1).reshape(T, H), host(scale))
        assert same or name == "K"
        assert (got != host(codes)).mean() < 1e-3


def test_the_binding_refuses():
    rng = np.random.default_rng(26)
    cache = dev(pool(rng, 4, 2, 16, 4))
    x = dev(rng.standard_normal((2, 8, 128)).astype(np.float32))
    ok = dict(Q=x[:, :4], K=x[:, 4:6], V=x[:, 6:], cache=cache, page_table=dev(np.zeros((1, 2), np.int32)),
              q_start=dev(starts([2])), kv_len=dev(np.array([20], np.int32)))
    spin.spin_kv_append(**ok)
    wide = torch.zeros((2, 8, 130), device=DEV)[:, :, :128]
    for bad in (dict(K=x[:, 4:7]), dict(V=x[:, 6:].half()), dict(K=x[:1, 4:6]), dict(K=x.double()[:, 4:6]), dict(Q=wide[:, :4]),
                dict(q_norm=torch.ones(64, device=DEV)), dict(k_norm=torch.ones(128, device=DEV).double()),
                dict(rope=torch.ones((40, 24), device=DEV)), dict(rope=torch.ones((40, 144), device=DEV)), dict(pos0=-1),
                dict(k_norm=torch.ones(128, device=DEV), eps=-1.0), dict(K=x[:, 4:6].cpu()), dict(Q=None, Q_out=x.half()),
                dict(K=torch.zeros((2, 2, 128), device=DEV).transpose(0, 1)), dict(V=x[:1, 6:].expand(2, 2, 128))):
        with pytest.raises((ValueError, TypeError, spin.SpinError)):
            spin.spin_kv_append(**dict(ok, **bad))


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("graph", [False, True])
def test_a_layer_serves_a_prompt_and_then_tokens(bits, graph):
    """qkv_proj's product -> append -> attention -> o_proj's quantizer, a prompt of two sequences behind a shared
    prefix and then single tokens, against the oracle on the cache the GPU wrote (itself equal to the oracle's)."""
    rng = np.random.default_rng(27)
    Hq, Hkv, page, prefix = 4, 2, 16, 37
    x_all = rng.standard_normal((prefix + 90, Hq + 2 * Hkv, 128)).astype(np.float32)
    w = (1 + 0.2 * rng.standard_normal((2, 128))).astype(np.float32)
    rope = spin.spin_rope_table(dev(frequencies(128)), 512)
    cache = spin.kv_cache(16, Hkv, page, bits)
    front = np.array([4, 9, 1], np.int32)
    table = np.array([[0, 2, 3, 5], [6, 7, 8, 10]], np.int32)
    mirror = {k: host(v).copy() for k, v in cache.items()}

    def rows(n):
        return rng.standard_normal((n, Hq + 2 * Hkv, 128)).astype(np.float32)

    def step(x, tab, q_start, kv, pos0):
        q, k, v = x.split([Hq, Hkv, Hkv], dim=1)
        return spin.spin_kv_append(q, k, v, cache, tab, q_start, kv, rope=rope, q_norm=dev(w[0]), k_norm=dev(w[1]), pos0=pos0)

    def both(x, tab, q_start, kv, pos0, run):
        nonlocal mirror
        mirror, _ = oracle.kv_append(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], mirror, tab, q_start, kv, rope=host(rope),
                                     q_norm=w[0], k_norm=w[1], pos0=pos0)
        out = run()
        for name in mirror:
            assert np.array_equal(host(cache[name]).view(np.uint8), mirror[name].view(np.uint8)), name
        return out

    # the shared prefix, once, into its own pages
    x = x_all[:prefix]
    xd, one = dev(x), (dev(front[None]), dev(starts([prefix])), dev(np.array([prefix], np.int32)))
    both(x, front[None], starts([prefix]), [prefix], 0, lambda: step(xd, *one, 0))

    # prompts of 20 and 33 tokens, then three single tokens each
    kv = np.zeros(2, np.int32)
    kv_d = dev(kv)
    captured = None
    for n in ([20, 33], [1, 1], [1, 1], [1, 1]):
        kv = kv + np.array(n, np.int32)
        kv_d.copy_(dev(kv))
        x, q_start = rows(sum(n)), starts(n)
        if sum(n) > 2 or not graph:
            xd, qs, td, fd = dev(x), dev(q_start), dev(table), dev(front)
            qd = both(x, table, q_start, kv, prefix, lambda: step(xd, td, qs, kv_d, prefix))
            O = spin.spin_kv_attn_shared(qd, cache, fd, prefix, td, qs, kv_d)
            codes, _, _ = spin.spin_fwht_quant(O.reshape(sum(n), Hq * 128), 1)
        else:
            if captured is None:
                xg, qs, td, fd = dev(x), dev(q_start), dev(table), dev(front)
                wg = dev(w[0]), dev(w[1])
                torch.cuda.synchronize()
                captured = torch.cuda.CUDAGraph()
                with torch.cuda.graph(captured):
                    q, k, v = xg.split([Hq, Hkv, Hkv], dim=1)
                    qd = spin.spin_kv_append(q, k, v, cache, td, qs, kv_d, rope=rope, q_norm=wg[0], k_norm=wg[1], pos0=prefix)
                    O = spin.spin_kv_attn_shared(qd, cache, fd, prefix, td, qs, kv_d)
                    codes, _, _ = spin.spin_fwht_quant(O.reshape(sum(n), Hq * 128), 1)
            xg.copy_(dev(x))
            both(x, table, q_start, kv, prefix, captured.replay)
        ref, bound = oracle.kv_attend(host(qd), mirror, table, q_start, kv, 128 ** -0.5, prefix_table=front, prefix_len=prefix)
        close(host(O).astype(np.float64), ref, bound)
        want, _ = oracle.quantize_rows(host(O).reshape(sum(n), Hq * 128).astype(np.float32))
        assert np.array_equal(host(codes), oracle.pack_int4(want))


@pytest.mark.parametrize("T,Hq,Hkv", [(336, 31, 17), (1030, 30, 18), (1400, 1, 23)])     # two, four and four heads a lane group
@pytest.mark.parametrize("bits,dtype,rot,interleaved,norm", [(4, np.float32, 128, False, True), (8, np.float16, 64, True, False),
                                                             (8, np.float32, 48, False, True), (4, np.float16, 0, False, False)])
def test_several_heads_of_a_token_at_once(T, Hq, Hkv, bits, dtype, rot, interleaved, norm):
    rng = np.random.default_rng(T + bits)
    q_len = [T - 120, 0, 1, 90, 20]
    kv_len = [T - 120 + 7, 30, 9, 60, 25]          # the fourth has more new tokens than tokens
    check(rng, q_len, kv_len, Hq, Hkv, bits, 64, dtype=dtype, rot=rot, interleaved=interleaved, norm=norm, before=3, behind=6,
          rope_len=T - 130 if rot else None)


def test_rope_table_of_any_frequency():
    """Turned a step at a time below 2^25 radians, by the functions above; the formula's value on both sides of it."""
    inv = np.array([300.0, -0.7, 0.0, 1e5, 2.0 ** 25 / 4100, -2.0 ** 25 / 4100, 1e-300, 1e20, 2.0 ** 60, np.inf, np.nan])
    for pos0 in (0, 4000, (1 << 25) - 20, (1 << 29) - 333):
        with np.errstate(invalid="ignore"):
            ref = oracle.rope_table(inv, 333, pos0)
        got = host(spin.spin_rope_table(dev(inv), 333, pos0=pos0))
        bad = np.isnan(ref)
        assert np.isnan(got[bad]).all()
        assert (np.abs(got - ref)[~bad] <= 2.0 ** -24 * np.abs(ref[~bad]) + 2.0 ** -48).all()
