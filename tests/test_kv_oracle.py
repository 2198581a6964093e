"""Pins of the cache oracle (CPU): the page order written out as a loop over
its dimensions, the two formats' numbers, worked rotations and attentions, and
page operations that can be followed by eye."""
import numpy as np
import pytest

import oracle
from oracle import kv_oracle as K


@pytest.mark.parametrize("D", [64, 128, 192, 256])
def test_places_are_the_documented_order(D):
    at = 0
    k = {}
    for i in range(4):
        for c in range(D // 64):
            for g in range(4):
                for t in range(16):
                    for j in range(16):
                        k[(16 * i + t, 64 * c + 16 * g + j)] = at
                        at += 1
    at = 0
    v = {}
    for n in range(D // 16):
        for g in range(4):
            for d in range(16):
                for i in range(4):
                    for j in range(4):
                        v[(16 * i + 4 * g + j, 16 * n + d)] = at
                        at += 1
    for which, want in (("k", k), ("v", v)):
        got = oracle.kv_places(which, D)
        assert all(got[t, d] == p for (t, d), p in want.items())
        assert sorted(got.ravel()) == list(range(64 * D))


def test_tables():
    t = oracle.kv_table("int8")
    assert t[128] == 0 and t[255] == 127 and t[1] == -127
    e = oracle.kv_table("e4m3")
    # 1.0 = exponent 7, largest 1.75 * 2^8, smallest 2^-9
    assert e[0x38] == 1.0 and e[0x7E] == 448.0 and e[1] == 2.0 ** -9 and e[0xB8] == -1.0 and np.isnan(e[0x7F])


def test_encode():
    assert oracle.kv_encode(np.array([0.5, 1.5, -2.5, 300, -np.inf, np.nan, 127.4]), "int8").tolist() == \
        [128, 130, 126, 255, 1, 128, 255]
    t = oracle.kv_table("e4m3")
    every = np.delete(np.arange(256), [127, 255, 128])
    assert oracle.kv_encode(t[every], "e4m3").tolist() == every.tolist()
    # halfway between 1 (mantissa 0) and 1.125 (1): even; past 448: 448
    assert oracle.kv_encode(np.array([1.0625, 1.1875, 500, np.inf, -0.0009765625]), "e4m3").tolist() == \
        [0x38, 0x3A, 0x7E, 0x7E, 0x80]


def test_encode_matches_torch_e4m3():
    torch = pytest.importorskip("torch")
    x = np.random.default_rng(0).standard_normal(4000) * 2.0 ** np.random.default_rng(1).uniform(-12, 8, 4000)
    x = np.clip(x.astype(np.float32), -448, 448)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(oracle.kv_encode(x, "e4m3"), want)


def test_rope_quarter_turn():
    # a pair at angle pi/2: (1, 0) -> (0, 1); the axis of the second pair stands still
    x = np.zeros((1, 1, 6))
    x[0, 0, :4] = [1, 2, 0, 0]
    x[0, 0, 4:] = [7, 8]
    y = oracle.rope_f64(x, np.array([[1], [0]]), np.array([np.pi / 2, np.pi / 2]), axis=[0, 1])
    assert np.allclose(y[0, 0], [0, 2, 1, 0, 7, 8])
    z = oracle.rope_f64(x, np.array([[1], [0]]), np.array([np.pi / 2, np.pi / 2]), axis=[0, 1], adjacent=True)
    assert np.allclose(z[0, 0], [-2, 1, 0, 0, 7, 8])


def _cache(pages, heads=1, D=64, fmt="int8"):
    c = {w: np.full((1, pages, heads, 64 * D), 128 if fmt == "int8" else 0, np.uint8) for w in ("k", "v")}
    return c | {w + "s": np.zeros((1, pages, heads, 4), np.float32) for w in ("k", "v")} | {"format": fmt}


def test_append_then_read_by_hand():
    c = _cache(2)
    row = [1, 0]
    k = np.zeros((2, 1, 64))
    k[0, 0, 3], k[1, 0, 3] = 127.0, 12.7
    K.kv_append_f64(c, 0, row, 0, k, k)
    assert c["ks"][0, 1, 0].tolist() == [1.0, 0, 0, 0]
    assert c["k"][0, 1, 0, K.kv_place_k(0, 3, 64)] == 255 and c["k"][0, 1, 0, K.kv_place_k(1, 3, 64)] == 128 + 13
    # a token twice as large: the scale doubles, held codes halve (127 / 2 = 63.5 -> 64, 13 / 2 = 6.5 -> 6)
    K.kv_append_f64(c, 0, row, 2, 2 * k[:1], k[:1])
    got = K.kv_sequence(c, 0, row, 3, "k")[:, 0, 3]
    assert got.tolist() == [128.0, 12.0, 254.0]
    assert K.kv_sequence(c, 0, row, 3, "v")[:, 0, 3].tolist() == [127.0, 13.0, 127.0]


def test_attention_by_hand():
    c = _cache(1)
    k = np.zeros((3, 1, 64))
    v = np.zeros((3, 1, 64))
    v[:, 0, 0] = [127, 0, -127]
    K.kv_append_f64(c, 0, [0], 0, k, v)
    q = np.ones((3, 1, 64))
    out, mass = K.kv_attn_f64(c, 0, [0], 3, q, 1.0)
    assert np.allclose(out[:, 0, 0], [127, 63.5, 0]) and np.allclose(mass[:, 0, 0], [127, 63.5, 254 / 3])
    out, _ = K.kv_attn_f64(c, 0, [0], 3, q, 1.0, causal=False)
    assert np.allclose(out[:, 0, 0], 0)
    out, _ = K.kv_attn_f64(c, 0, [0], 3, q, 1.0, window=1)
    assert np.allclose(out[:, 0, 0], [127, 0, -127])
    out, _ = K.kv_attn_f64(c, 0, [-1], 3, q, 1.0)
    assert not out.any()


def test_pages_by_hand():
    P = oracle.PagesOracle([[3, 1, -1], [-1] * 3, [-1] * 3], [100, 0, 0], [0, 1, 0, 1, 0], "abcde")
    assert P.fork([0, 0], [1, 2]) == (0, 2)
    assert P.table == [[3, 1, -1], [3, 0, -1], [3, 2, -1]] and P.refs == [1, 1, 1, 3, 0]
    assert "".join(P.contents) == "bbbde" and P.lens == [100, 100, 100]
    # row 1 cut inside the shared page 3: its own copy, page 0 let go first and taken again
    assert P.resize([-1, 10, -1]) == (0, 1)
    assert P.table[1] == [0, -1, -1] and P.refs == [1, 1, 1, 2, 0] and P.contents[0] == "d"
    assert P.resize([0, 130, -1]) == (0, 0)
    assert P.table == [[-1] * 3, [0, 1, 4], [3, 2, -1]] and P.refs == [1, 1, 1, 1, 1]
    assert P.resize([192, -1, -1]) == (3, 0)
    assert P.resize([-1, 0, -1]) == (0, 0)
    assert P.compact() == (0, 2) and P.table[2] == [1, 0, -1] and P.refs == [1, 1, 0, 0, 0]
    assert P.fork([2], [2]) == (-1, 0) and P.fork([1], [2]) == (-1, 0)
