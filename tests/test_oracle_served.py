"""Pins of oracle/paged.py's trees, weights, choices and moves that do not use its own code."""

import numpy as np
import torch

import oracle
from oracle.paged import cache_tokens

rng = np.random.default_rng(41)


def small(n_pages=6, H=2, page=16):
    q = lambda *s: rng.integers(0, 256, s).astype(np.uint8)  # noqa: E731
    return {"K_codes": q(n_pages, H, page, 128), "K_scale": rng.uniform(0.001, 0.02, (n_pages, H, page)).astype(np.float16),
            "V_codes": q(n_pages, H, page // 4, 16, 4, 8), "V_scale": rng.uniform(0.001, 0.02, (n_pages, H, page)).astype(np.float16)}


def test_a_tree_by_hand():
    #  0        0 and 4 follow the context; 1, 2 follow 0; 3 follows 1; 5 follows 4
    tree, at = oracle.kv_tree([9, -1, 0, 0, 1, -1, 4], [1, 7], [26], 1, 100)
    assert tree[1:, 0].tolist() == [0b1, 0b11, 0b101, 0b1011, 0b10000, 0b110000] and tree[0, 0] == 0
    assert at[1:].tolist() == [120, 121, 121, 122, 120, 121]


def test_a_path_of_a_tree_is_a_sequence():
    """A row's attention, log sum and distances are those of the context and its path as a plain causal sequence."""
    cache, parent = small(), [-1, 0, 0, 2, -1, 3]
    table, kv, n = np.array([[3, 1, 5]]), 40, 6
    q = rng.standard_normal((n, 4, 128))
    tree, at = oracle.kv_tree(parent, [0, n], [kv], 1)
    slopes = np.array([0.5, 0.1, 0.0, 0.3])
    for more in (dict(), dict(window=9, slopes=slopes, softcap=3.0)):
        O, _, logs, _ = oracle.kv_attend(q, cache, table, [0, n], [kv], 0.05, tree=tree, positions=at, sums=True, **more)
        for t, path in ((5, [0, 2, 3, 5]), (4, [4]), (1, [0, 1])):
            order = np.array([*range(kv - n), *(kv - n + i for i in path)])
            for h in range(2):
                kd, ks, vd, vs, _ = cache_tokens(cache, table[0], h, kv)
                k, v = torch.tensor((kd * ks[:, None])[order]), torch.tensor((vd * vs[:, None])[order])
                for g in (2 * h, 2 * h + 1):
                    z = k @ torch.tensor(q[t, g]) * 0.05
                    far = torch.arange(len(order) - 1, -1, -1)
                    if more:
                        z = 3.0 * torch.tanh(z / 3.0) - slopes[g] * far
                        z = z.masked_fill(far >= 9, -torch.inf)
                    assert np.allclose(O[t, g], torch.softmax(z, 0) @ v, atol=1e-9)
                    assert np.allclose(logs[t, g], torch.logsumexp(z, 0))


def test_a_prefix_is_context_where_rows_outnumber_tokens():
    """Three of five new tokens have no place: their bits say nothing, and the prefix is seen all the same."""
    cache, n, kv, prefix = small(), 5, 2, 20
    q = rng.standard_normal((n, 4, 128))
    tree, at = oracle.kv_tree([-1, 0, 1, 2, 3], [0, n], [kv], 1, prefix)
    tree[3] = 0
    O, _ = oracle.kv_attend(q, cache, np.array([[3]]), [0, n], [kv], 0.05, tree=tree, positions=at, prefix_table=[0, 1], prefix_len=prefix)
    last, _ = oracle.kv_attend(q[[4]], cache, np.array([[3]]), [0, 1], [kv], 0.05, prefix_table=[0, 1], prefix_len=prefix)
    assert np.allclose(O[4], last[0])
    alone, _ = oracle.kv_attend(q[[3]], cache, np.array([[3]]), [0, 1], [0], 0.05, causal=False, prefix_table=[0, 1], prefix_len=prefix)
    assert np.allclose(O[3], alone[0])


def test_weights_are_the_columns_of_softmax():
    cache, table, kv, n = small(), np.array([[2, 0, 4]]), 40, 7
    q = rng.standard_normal((n, 4, 128)).astype(np.float16)
    _, _, logs, _ = oracle.kv_attend(q, cache, table, [0, n], [kv], 0.05, sums=True)
    W, _ = oracle.kv_weights(q, logs, cache, table, [0, n], [kv], 0.05)
    for h in range(2):
        kd, ks, _, _, _ = cache_tokens(cache, table[0], h, kv)
        z = torch.tensor(q[:, 2 * h:2 * h + 2].astype(np.float64)) @ torch.tensor((kd * ks[:, None]).T) * 0.05
        seen = torch.arange(kv)[None] <= torch.arange(kv - n, kv)[:, None]
        p = torch.softmax(z.masked_fill(~seen[:, None], -torch.inf), -1).sum((0, 1)).numpy()
        got = np.concatenate([W[2, h], W[0, h], W[4, h, :8]])
        assert np.allclose(got, p) and np.isnan(W[4, h, 8:]).all()
    assert np.isnan(W[[1, 3, 5]]).all()
    prior = rng.random(W.shape)
    both, _ = oracle.kv_weights(q, logs, cache, table, [0, n], [kv], 0.05, prior=prior, decay=0.5)
    assert np.allclose(both[2], W[2] + 0.5 * prior[2])


def test_a_choice_by_hand():
    W = np.zeros((2, 1, 16), np.float32)
    W[1, 0, :8] = [5, 1, 3, 3, np.nan, 0, 3, 0]
    pick = lambda **kw: [x.tolist() for x in oracle.kv_choose(W, np.array([[1]]), [8], **kw)]  # noqa: E731
    assert pick(keep=3) == [[[[0, 2, 3]]], [3]]
    assert pick(keep=4, first=2, recent=1) == [[[[0, 1, 2, 7]]], [4]]
    assert pick(keep=9) == [[[[0, 1, 2, 3, 4, 5, 6, 7, -1]]], [8]]
    assert pick(keep=7) == [[[[0, 1, 2, 3, 5, 6, 7]]], [7]]


def test_a_move_keeps_tokens():
    cache, table = small(), np.array([[3, 1, 5]])
    W = rng.random((6, 2, 16)).astype(np.float32)
    kept = np.array([[[0, 4, 30, 31, -1]]])
    new, w = oracle.kv_move(cache, table, kept, at=[3], W=W)
    for h in range(2):
        before, after = cache_tokens(cache, table[0], h, 48), cache_tokens(new, table[0], h, 48)
        for a, b in zip(before[:4], after[:4]):
            assert np.array_equal(b[3:7], a[[3, 7, 33, 34]]) and np.array_equal(b[7:], a[7:]) and np.array_equal(b[:3], a[:3])
    assert np.array_equal(w[3, 0, 3:7], [W[3, 0, 3], W[3, 0, 7], W[5, 0, 1], W[5, 0, 2]])
    out, _ = oracle.kv_move(cache, table, kept, to_table=np.array([[0]]))
    assert np.array_equal(out["K_codes"][0, :, 2], cache["K_codes"][1, :, 14]) and np.array_equal(out["K_codes"][3], cache["K_codes"][3])
