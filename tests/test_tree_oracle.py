"""Pins of the tree and log probability oracle (CPU), against values that can be followed by eye."""
import numpy as np
import pytest

import oracle
import synth

# 0 -> 1, 2; 1 -> 3; 3 -> 5; 2 -> 4; row 6 stands behind the context itself
PARENT = [-1, 0, 0, 1, 2, 3, -1]


def test_norm():
    y = oracle.norm_f64(np.array([[3.0, 4.0, 0.0, 0.0]]), [1, 2, 1, 1], 0.0)
    assert np.allclose(y, [[3 / 2.5, 8 / 2.5, 0, 0]])            # mean square 6.25
    assert np.allclose(oracle.norm_f64(np.zeros((1, 4)), np.ones(4), 1e-6), 0)
    assert np.isnan(oracle.norm_f64(np.zeros((1, 4)), np.ones(4), 0.0)).all()


def test_rows_above_and_masks():
    assert oracle.tree_above(PARENT) == [[0], [1, 0], [2, 0], [3, 1, 0], [4, 2, 0], [5, 3, 1, 0], [6]]
    assert oracle.tree_words(oracle.tree_seen(PARENT), 1)[:, 0].tolist() == [1, 3, 5, 11, 21, 43, 64]
    assert oracle.tree_words(oracle.tree_seen(PARENT, 2), 1)[:, 0].tolist() == [1, 3, 5, 10, 20, 40, 64]
    wide = np.zeros((1, 130), bool)
    wide[0, [0, 63, 64, 129]] = True
    assert oracle.tree_words(wide, 2)[0].tolist() == [1 + 2 ** 63, 1]


def test_a_chain_is_causal():
    chain = np.arange(-1, 5)
    for window, sinks in ((0, 0), (3, 0), (4, 2), (9, 1)):
        a = oracle.tree_context(6, 7, oracle.tree_seen(chain, window), window, sinks)
        assert np.array_equal(a, oracle.causal_context(6, 7, window, sinks))


def test_contexts_by_hand():
    c = oracle.causal_context(2, 4, 2, 1)
    assert c.astype(int).tolist() == [[1, 0, 0, 1, 1, 0], [1, 0, 0, 0, 1, 1]]
    assert oracle.causal_context(3, -1).astype(int).tolist() == [[0, 0], [1, 0], [1, 1]]
    seen = np.array([[True, False], [False, False]])
    assert oracle.tree_context(2, 3, seen, 2, 1).astype(int).tolist() == [[1, 0, 1, 1, 0], [1, 1, 1, 0, 0]]


def test_attention_of_what_is_seen():
    rng = np.random.default_rng(0)
    c = synth.make_kv_pool(rng, 1, 2, 1, 64, "int8")
    q = rng.standard_normal((3, 2, 64)).astype(np.float16)
    for window in (0, 5):
        a = oracle.kv_attn_f64(c, 0, [1, 0], 90, q, 0.1, True, window)
        b = oracle.kv_attn_seen_f64(c, 0, [1, 0], 90, q, 0.1, oracle.causal_context(3, 87, window))
        assert np.allclose(a[0], b[0]) and np.allclose(a[1], b[1])
    assert not oracle.kv_attn_seen_f64(c, 0, [1, 0], 90, q, 0.1, np.zeros((3, 90), bool))[0].any()


def test_accept():
    token = [9, 1, 2, 3, 4, 5, 1]
    assert oracle.tree_accept([1, 3, 0, 5, 0, 8, 0], token, PARENT, 9) == ([0, 1, 3, 5], 8)
    assert oracle.tree_accept([1, 3, 0, 5, 0, 8, 0], token, PARENT, 2) == ([0, 1], 3)
    assert oracle.tree_accept([2, 3, 7, 5, 0, 8, 0], token, PARENT, 9) == ([0, 2], 7)
    assert oracle.tree_accept([6, 0, 0, 0, 0, 0, 0], token, PARENT, 9) == ([0], 6)
    # of two children with the same token the first
    assert oracle.tree_accept([2, 7, 8], [0, 2, 2], [-1, 0, 0], 9) == ([0, 1], 7)
    assert oracle.tree_accept([], [], [], 3) == ([], -1)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_keep(fmt):
    rng = np.random.default_rng(1)
    c = synth.make_kv_pool(rng, 2, 3, 2, 64, fmt)
    c["ks"][:], c["vs"][:] = 0.5, 0.25                           # one scale for all: nothing is rounded
    row, base, path = [2, 0], 60, [0, 2, 3, 9]
    before = {w: [oracle.kv_sequence(c, i, row, 75, w) for i in range(2)] for w in "kv"}
    oracle.kv_keep_f64(c, row, base, path)
    for w in "kv":
        for i in range(2):
            want = before[w][i].copy()
            want[[61, 62, 63]] = before[w][i][[62, 63, 69]]
            assert np.array_equal(oracle.kv_sequence(c, i, row, 75, w), want)


def test_keep_scales():
    c = {"format": "int8", "k": np.full((1, 1, 1, 4096), 128, np.uint8), "v": np.full((1, 1, 1, 4096), 128 + 50, np.uint8),
         "ks": np.ones((1, 1, 1, 4), np.float32), "vs": np.array([[[[1.0, 2.0, 4.0, 1.0]]]], np.float32)}
    oracle.kv_keep_f64(c, [0], 14, [0, 20])                      # token 34 (scale 4) to 15
    assert c["vs"][0, 0, 0].tolist() == [4, 2, 4, 1]
    v = oracle.kv_sequence(c, 0, [0], 64, "v")[:, 0, 0]
    assert v[15] == 200 and v[0] == 48                           # 50 / 4 = 12.5, to even 12, times 4
    assert (v[16:32] == 100).all() and (v[32:48] == 200).all()


def test_logprobs():
    lp, h, tt, tl = oracle.logprobs_f64(np.log([0.5, 0.25, 0.25]), [1, 5, -1], 4)
    assert np.allclose(lp[0], np.log(0.25)) and lp[1] == lp[2] == -np.inf
    assert np.isclose(h, 1.5 * np.log(2)) and tt.tolist() == [0, 1, 2, -1] and tl[3] == -np.inf
    lp, h, tt, tl = oracle.logprobs_f64([-np.inf, 3.0, -np.inf], [0, 1], 2)
    assert lp.tolist() == [-np.inf, 0.0] and h == 0 and tt.tolist() == [1, 0]
    for bad in ([1.0, np.nan], [1.0, np.inf], [-np.inf, -np.inf]):
        lp, h, tt, tl = oracle.logprobs_f64(bad, [0], 2)
        assert np.isnan(lp).all() and np.isnan(h) and np.isnan(tl).all()
    assert oracle.logprobs_f64([1.0, np.nan, np.nan], [], 3)[2].tolist() == [1, 2, 0]


def test_trees():
    rng = np.random.default_rng(2)
    for n, levels in ((0, 3), (1, 3), (2, 1), (61, 8), (200, 200)):
        p = synth.make_tree(rng, n, levels)
        assert len(p) == n and all(-1 <= x < i for i, x in enumerate(p)) and (p[1:] >= 0).all()
        if n > 1:
            assert max(len(a) for a in oracle.tree_above(p)) == min(levels, n - 1) + 1
