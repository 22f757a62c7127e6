"""Drafted trees and eviction as a server runs them, on the paged cache: a step of speculative decoding, a cache that is
thinned and goes on, all of it captured, on a second stream and on two at once."""

import numpy as np
import pytest
import torch

import oracle
from rotation_bit_quantization_amd import spin

from .paged_case import DEV, close, dev, host, pool, starts, tables
from .test_gpu_kv_append import frequencies

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spin.load()


def paths(parent):
    """Of each drafted token, its continuation from the context on."""
    out = []
    for i, p in enumerate(parent):
        out.append(([] if p < 0 else out[p]) + [i])
    return out


@pytest.mark.parametrize("bits,page,prefix", [(4, 16, 0), (8, 64, 0), (4, 32, 70)])
def test_speculative_steps(bits, page, prefix):
    """Draft, verify, accept, three times over: the cache's bytes are those of appending the accepted tokens alone, and each
    accepted row's attention is that of the plain sequence."""
    rng = np.random.default_rng(bits)
    B, Hq, Hkv, ctx = 3, 8, 2, np.array([37, 5, 130])
    first = -(-prefix // page)
    n_pages = first + B * (-(-260 // page)) + 1
    start = pool(rng, n_pages, Hkv, page, bits)
    cache, plain = dev(start), dev(start)
    table = dev(tables(rng, [200] * B, page, n_pages, extra=1, first=first))
    front = dev(np.arange(first, dtype=np.int32))
    rope = spin.spin_rope_table(dev(frequencies(64)), 400)
    norm = dev((1 + 0.1 * rng.standard_normal(128)).astype(np.float32))
    for step in range(3):
        q_len = [12, 33, 1] if step != 1 else [1, 70, 20]
        T, q_start, words = sum(q_len), dev(starts(q_len)), 3
        parent = [rng.integers(-1, np.arange(n)) if n > 1 else np.array([-1]) for n in q_len]
        parent = [np.where(np.arange(len(p)) == 0, -1, p) for p in parent]
        x = dev(rng.standard_normal((T, Hq + 2 * Hkv, 128)).astype(np.float16))
        q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        kv = dev((ctx + q_len).astype(np.int32))
        tree, at = spin.spin_kv_tree(dev(np.concatenate(parent).astype(np.int32)), q_start, kv, words, pos0=prefix)
        how = dict(rope=rope, k_norm=norm, q_norm=norm)
        Q = spin.spin_kv_append(q, k, v, cache, table, q_start, kv, positions=at, **how)
        lse = torch.empty((T, Hq), device=DEV)
        O = host(spin.spin_kv_attn_tree(Q, cache, table, q_start, kv, tree, positions=at, prefix_table=front if prefix else None,
                                        prefix_len=prefix, lse=lse))
        # the model's own choice here is the deepest token of each tree
        chosen = [max(paths(p), key=len) for p in parent]
        kept = np.full((B, 1, max(map(len, chosen))), -1, np.int32)
        for b, p in enumerate(chosen):
            kept[b, 0, :len(p)] = p
        spin.spin_kv_move(cache, table, dev(kept), at=dev(ctx.astype(np.int32)))
        # the same tokens, one sequence each
        rows = np.concatenate([starts(q_len)[b] + np.array(p) for b, p in enumerate(chosen)])
        alone = x[torch.from_numpy(rows).to(DEV)]
        m_start, m_kv = dev(starts([len(p) for p in chosen])), dev(np.array([c + len(p) for c, p in zip(ctx, chosen)], np.int32))
        Q1 = spin.spin_kv_append(alone[:, :Hq], alone[:, Hq:Hq + Hkv], alone[:, Hq + Hkv:], plain, table, m_start, m_kv, pos0=prefix, **how)
        assert np.array_equal(host(Q1), host(Q)[rows])
        lse1 = torch.empty((len(rows), Hq), device=DEV)
        if prefix:
            O1 = host(spin.spin_kv_attn_shared(Q1, plain, front, prefix, table, m_start, m_kv, lse=lse1))
        else:
            O1 = host(spin.spin_kv_attn(Q1, plain, table, m_start, m_kv, lse=lse1))
        # two results of the same sums, each within 2^-8 of values below 4 (bounds of the scores and weights: see the oracle's)
        assert np.abs(O1.astype(np.float64) - O[rows]).max() <= 4 * 2.0 ** -7
        assert np.abs(host(lse1) - host(lse)[rows]).max() <= 2.0 ** -10
        ctx = ctx + [len(p) for p in chosen]
        pages = table.cpu().numpy()
        for b in range(B):
            for name in cache:
                got, ref = (host(c[name])[pages[b, :-(-int(ctx[b]) // page)]] for c in (cache, plain))
                if name == "V_codes":
                    got, ref = (t.transpose(0, 2, 4, 1, 3, 5).reshape(-1, Hkv, 16, bits) for t in (got, ref))
                else:
                    got, ref = (np.moveaxis(t, 1, 2).reshape(-1, Hkv, *t.shape[3:]) for t in (got, ref))
                assert np.array_equal(got[:ctx[b]], ref[:ctx[b]]), (step, b, name)


def test_a_thinned_cache_goes_on():
    """A prompt, its weights, the choice, the move in place and into other pages, then tokens at their own positions."""
    rng = np.random.default_rng(3)
    B, Hq, Hkv, page, bits, keep = 2, 8, 2, 16, 4, 60
    q_len = np.array([200, 50])
    cache = dev(pool(rng, 60, Hkv, page, bits))
    table = tables(rng, [256, 256], page, 40)
    rope = spin.spin_rope_table(dev(frequencies(128)), 400)
    q_start, kv = dev(starts(q_len)), dev(q_len.astype(np.int32))
    x = dev(rng.standard_normal((250, Hq + 2 * Hkv, 128)).astype(np.float32))
    split = lambda t: (t[:, :Hq], t[:, Hq:Hq + Hkv], t[:, Hq + Hkv:])  # noqa: E731
    Q = spin.spin_kv_append(*split(x), cache, dev(table), q_start, kv, rope=rope)
    lse = torch.empty((250, Hq), device=DEV)
    spin.spin_kv_attn(Q, cache, dev(table), q_start, kv, lse=lse)
    # the last 20 rows of each sequence decide
    last = torch.cat([torch.arange(180, 200), torch.arange(230, 250)]).to(DEV)
    W = spin.spin_kv_weights(Q[last].contiguous(), lse[last].contiguous(), cache, dev(table), dev(starts([20, 20])), kv)
    ref_W, bound = oracle.kv_weights(host(Q)[last.cpu().numpy()], host(lse)[last.cpu().numpy()], {k: host(t) for k, t in cache.items()}, table,
                                     starts([20, 20]), q_len, 128 ** -0.5)
    there = ~np.isnan(ref_W)
    assert (np.abs(host(W) - ref_W)[there] <= bound[there]).all()
    kept, lens = spin.spin_kv_choose(W, dev(table), kv, keep, first=2, recent=16)
    assert host(lens).tolist() == [60, 50]
    want, _ = oracle.kv_choose(host(W), table, q_len, keep, 2, 16)
    assert np.array_equal(host(kept), want)
    before, weights = {k: host(t).copy() for k, t in cache.items()}, host(W).copy()
    other = {k: t.clone() for k, t in cache.items()}
    to = np.arange(40, 40 + 2 * 6).reshape(2, 6).astype(np.int32)
    spin.spin_kv_move(cache, dev(table), kept, W=W)
    ref, ref_W = oracle.kv_move(before, table, want, None, None, weights)
    assert all(np.array_equal(host(cache[k]).view(np.uint8), ref[k].view(np.uint8)) for k in ref) and np.array_equal(host(W), ref_W)
    spin.spin_kv_move(other, dev(table), kept, to_table=dev(to))
    # three more tokens a sequence, at positions 200 .. and 50 ..
    new, n_start = dev(rng.standard_normal((6, Hq + 2 * Hkv, 128)).astype(np.float32)), dev(starts([3, 3]))
    at = dev(np.array([200, 201, 202, 50, 51, 52], np.int32))
    outs = []
    for c, t in ((cache, table), (other, to)):
        more = lens + 3
        Q = spin.spin_kv_append(*split(new), c, dev(t), n_start, more, rope=rope, positions=at)
        outs.append(host(spin.spin_kv_attn(Q, c, dev(t), n_start, more)))
    assert np.array_equal(outs[0][3:], outs[1][3:]) or np.abs(outs[0].astype(np.float64) - outs[1]).max() <= 2.0 ** -8
    ref, bound = oracle.kv_attend(host(Q), {k: host(t) for k, t in cache.items()}, table, starts([3, 3]), [63, 53], 128 ** -0.5)
    close(outs[0].astype(np.float64), ref, bound)
    close(outs[1].astype(np.float64), ref, bound)


def served(rng, B, n, kv, keep, Hq=8, Hkv=2, page=16, room=0):
    """Arguments of a call of each kind on one batch of B sequences with n rows each."""
    need = -(-kv // page)
    width = max(need, -(-room // page))
    pages = B * need
    cache = pool(rng, pages + B * -(-keep // page), Hkv, page, 4)
    table = np.pad(tables(rng, [kv] * B, page, pages, extra=0), ((0, 0), (0, width - need)), constant_values=-1)
    T = B * n
    parent = np.concatenate([rng.integers(-1, np.arange(n)) if n > 1 else [-1] for _ in range(B)]).astype(np.int32)
    parent.reshape(B, n)[:, 0] = -1
    to = (pages + np.arange(B * -(-keep // page))).reshape(B, -1).astype(np.int32)
    s = dict(Q=rng.standard_normal((T, Hq, 128)).astype(np.float16), cache=cache, table=table, q_start=starts([n] * B),
             kv=np.full(B, kv, np.int32), parent=parent, to=to, W=np.zeros(cache["K_scale"].shape, np.float32),
             prior=rng.random(cache["K_scale"].shape).astype(np.float32))
    s = {k: dev(v) for k, v in s.items()}
    s.update(words=-(-n // 32), keep=keep)
    return s


def serve(s, stream=None):
    """All calls, one after the other; returns what they made."""
    on = dict(stream=stream)
    tree, at = spin.spin_kv_tree(s["parent"], s["q_start"], s["kv"], s["words"], **on)
    lse = s.setdefault("lse", torch.empty(s["Q"].shape[:2], device=DEV))
    O = spin.spin_kv_attn_tree(s["Q"], s["cache"], s["table"], s["q_start"], s["kv"], tree, positions=at, softcap=30.0, lse=lse, **on)
    logs = s.setdefault("logs", torch.empty(s["Q"].shape[:2], device=DEV))
    P = spin.spin_kv_attn(s["Q"], s["cache"], s["table"], s["q_start"], s["kv"], lse=logs, **on)
    W = spin.spin_kv_weights(s["Q"], logs, s["cache"], s["table"], s["q_start"], s["kv"], prior=s["prior"], decay=0.9, W=s["W"], **on)
    kept, lens = spin.spin_kv_choose(W, s["table"], s["kv"], s["keep"], first=1, recent=2, **on)
    spin.spin_kv_move(s["cache"], s["table"], kept, to_table=s["to"], W=W, **on)
    return dict(s["cache"], tree=tree, at=at, O=O, P=P, lse=lse, logs=logs, W=W, kept=kept, lens=lens)


CASES = {
    "few rows": dict(B=5, n=1, kv=300, keep=70),
    "rows in shares, tables in parts": dict(B=2, n=150, kv=700, keep=333, Hkv=1, room=40000),
    "tiles": dict(B=3, n=100, kv=400, keep=100, Hkv=2, room=2 ** 20),
}


@pytest.mark.parametrize("case", sorted(CASES))
def test_captured(case):
    """Replayed in turn with eager calls, with other lengths and queries each time; two graphs at once have workspaces of
    their own."""
    s = served(np.random.default_rng(4), **CASES[case])
    kv0 = int(s["kv"][0])
    serve(s)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = serve(s)
        graphs.append((g, out))
    seen = []
    for rep, less in enumerate([0, 7, 1000, 31, 0]):
        s["kv"].fill_(max(kv0 - less, 0))
        s["Q"].copy_(torch.roll(s["Q"], 1, 0))
        s["W"].zero_()
        want = {k: host(v).copy() for k, v in serve(s).items()}
        seen.append(want["O"])
        for g, out in graphs + graphs[::-1]:
            for t in (s["W"], out["O"], out["P"], out["kept"]):
                t.zero_()
            g.replay()
            for k, v in out.items():
                assert np.array_equal(host(v), want[k]), (rep, k)
    assert not np.array_equal(seen[0], seen[1])


@pytest.mark.parametrize("case", sorted(CASES))
def test_on_streams_at_once(case):
    """The current stream is behind with long products and calls whose workspaces it has let go."""
    rng = np.random.default_rng(5)
    here, there = served(rng, **CASES[case]), served(rng, **CASES[case])
    want = [{k: host(v).copy() for k, v in serve(s).items()} for s in (here, there)]
    a, side = torch.randn((4096, 4096), device=DEV, dtype=torch.float16), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    got = [[], []]
    for handle in (side, side.cuda_stream):
        for _ in range(6):
            a @ a
            for i, (s, on) in enumerate(((here, None), (there, handle))):
                out = serve(s, on)
                got[i].append({k: out[k] for k in ("tree", "at", "O", "P", "kept", "lens")})
    torch.cuda.synchronize()
    for i in range(2):
        for out in got[i]:
            for k, v in out.items():
                assert np.array_equal(host(v), want[i][k]), (i, k)
    for s, w in zip((here, there), want):
        for k in s["cache"]:
            assert np.array_equal(host(s["cache"][k]).view(np.uint8), w[k].view(np.uint8))


def test_refusals_of_the_binding():
    s = served(np.random.default_rng(6), 2, 3, 50, 20)
    tree, at = spin.spin_kv_tree(s["parent"], s["q_start"], s["kv"], 1)
    lse = torch.empty(s["Q"].shape[:2], device=DEV)
    attn = lambda **kw: spin.spin_kv_attn_tree(**{**dict(Q=s["Q"], cache=s["cache"], page_table=s["table"], q_start=s["q_start"],  # noqa: E731
                                                         kv_len=s["kv"], tree=tree, positions=at, lse=lse), **kw})
    weights = lambda **kw: spin.spin_kv_weights(**{**dict(Q=s["Q"], lse=lse, cache=s["cache"], page_table=s["table"],  # noqa: E731
                                                          q_start=s["q_start"], kv_len=s["kv"]), **kw})
    choose = lambda **kw: spin.spin_kv_choose(**{**dict(W=s["W"], page_table=s["table"], kv_len=s["kv"], keep=9), **kw})  # noqa: E731
    move = lambda **kw: spin.spin_kv_move(**{**dict(cache=s["cache"], page_table=s["table"], kept=choose()[0]), **kw})  # noqa: E731
    for call in (attn, weights, choose, move):
        call()
    i32 = lambda *shape: torch.zeros(shape, dtype=torch.int32, device=DEV)  # noqa: E731
    bad = [lambda: spin.spin_kv_tree(s["parent"], s["q_start"], s["kv"], 0), lambda: spin.spin_kv_tree(s["parent"], s["kv"], s["kv"], 1),
           lambda: spin.spin_kv_tree(s["parent"], s["q_start"], s["kv"], 1, tree=i32(6, 2)), lambda: spin.spin_kv_tree(s["parent"], s["q_start"], s["kv"], 1 << 40),
           lambda: attn(tree=i32(5, 1)), lambda: attn(tree=tree[0]), lambda: attn(positions=i32(5)), lambda: attn(lse=lse[:, :3]),
           lambda: attn(prefix_len=4), lambda: attn(prefix_len=4, prefix_table=i32(0)),
           lambda: weights(lse=lse[:, :3]), lambda: weights(prior=s["W"][:1]), lambda: weights(W=s["W"][:, :1]), lambda: weights(pos0=1 << 31),
           lambda: choose(keep=0), lambda: choose(W=s["W"][0]), lambda: choose(kv_len=i32(3)), lambda: choose(kept=i32(2, 2, 8)),
           lambda: move(kept=i32(2, 3, 4)), lambda: move(kept=i32(1, 2, 4)), lambda: move(at=i32(3)), lambda: move(to_table=i32(3, 2)),
           lambda: move(W=s["W"][:1])]
    x = torch.zeros((6, 2, 128), device=DEV)
    append = lambda **kw: spin.spin_kv_append(None, x, x, s["cache"], s["table"], s["q_start"], s["kv"], **kw)  # noqa: E731
    append(positions=at)
    bad += [lambda: append(positions=at, pos0=3), lambda: append(positions=i32(5)), lambda: append(positions=at[None])]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    for call in (lambda: attn(tree=tree.long()), lambda: attn(positions=at.long()), lambda: attn(lse=lse.half()), lambda: weights(W=s["W"].half()),
                 lambda: choose(W=s["W"].double()), lambda: move(kept=i32(2, 2, 4).long()), lambda: spin.spin_kv_tree(s["parent"].long(), s["q_start"], s["kv"], 1)):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: attn(positions=None, window=5), lambda: attn(tree=i32(6, 129)), lambda: choose(first=5, recent=5), lambda: choose(first=-1),
                 lambda: spin.spin_kv_tree(s["parent"], s["q_start"], s["kv"], 129), lambda: weights(decay=float("nan"))):
        with pytest.raises(spin.SpinError):
            call()
    # what has nothing to do does nothing
    empty = i32(0)
    spin.spin_kv_tree(empty, i32(1), empty, 1)
    spin.spin_kv_attn_tree(s["Q"][:0], s["cache"], s["table"], i32(3), s["kv"], tree[:0], positions=at[:0])
    assert spin.spin_kv_choose(s["W"], s["table"][:0], s["kv"][:0], 5)[0].shape == (0, 2, 5)
    spin.spin_kv_move(s["cache"], s["table"], i32(2, 1, 0))
    spin.spin_kv_move(s["cache"], s["table"][:0], i32(0, 2, 4))
