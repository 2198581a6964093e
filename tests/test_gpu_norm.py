"""GPU parity of bq_norm_rope and bq_kv_append_norm against the fp64 oracle.

Tolerance.  The sum of D <= 1024 squares is formed by at most 16 additions in
a lane and 10 across lanes (append: across up to 16 partial sums), each off by
2^-24 of it, as is each square: 2^-19 of the sum, half of it of its root; the
hardware's reciprocal root, the weight and the product add 2^-22: a normed
value z is within 2^-19 |z|.  The rotation adds 2^-17 of the pair's |z1| + |z2|
(angle and hardware sine, as in the tests of bq_rope), and the result is
rounded to fp16 once, 2^-11 |y| (2^-25 below the normal range).

In the cache a value x to be coded is within d = 2^-16 + 2^-18 of the largest
|z| of the exact one, and its block's scale s, a maximum of such values over
127 or 448, within d over that and 2^-22 s.  The code is the one nearest to x
over the scale as it is held, formed in fp32 (2^-22 of it): so what is held is
within half a code's step of the exact value, plus d, plus 2^-21 of the value.
(Held against the exact value and not against the oracle's code, of which the
neighbour is as near where the exact value lies in the middle: a value that is
an odd multiple of half a step of the block's largest one is exactly there.)"""
import numpy as np
import pytest

import oracle
import synth
from gpu_helpers import torch_mod
from kv_helpers import cu_of, download_cache, up, upload_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    torch = torch_mod()
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    import bit_quantized_decode_qmv_amd as bq
    bq.load_library()


def check(y, x, w, eps, pos, inv, axis, adjacent):
    z = oracle.norm_f64(x, w, eps)
    ref = oracle.rope_f64(z, pos, inv, axis, adjacent)
    rot = 2 * len(inv)
    mass = np.zeros_like(ref)
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if adjacent else (slice(0, rot // 2), slice(rot // 2, rot))
    mass[..., a] = mass[..., b] = np.abs(z[..., a]) + np.abs(z[..., b])
    tol = 2.0 ** -11 * np.abs(ref) + 2.0 ** -25 + 2.0 ** -17 * mass + 2.0 ** -19 * np.maximum(mass, np.abs(z))
    worst = np.max(np.abs(y.astype(np.float64) - ref) / tol)
    assert worst <= 1.0, worst


CASES = [  # tokens, heads, D, rot, axes, adjacent
    (1, 1, 64, 64, 1, False), (5, 48, 128, 128, 1, False), (17, 3, 128, 64, 3, False), (33, 8, 256, 128, 3, True),
    (2, 5, 192, 192, 2, False), (7, 2, 80, 32, 1, True), (4099, 2, 64, 48, 3, False), (3, 1, 16, 16, 8, False),
    (6, 4, 128, 0, 1, False), (3, 2, 1024, 512, 1, False), (9, 3, 48, 48, 1, False), (2, 7, 1008, 1008, 1, True),
    (700, 5, 192, 64, 1, False),
]


@pytest.mark.parametrize("tokens,heads,D,rot,axes,adjacent", CASES)
def test_norm_rope(tokens, heads, D, rot, axes, adjacent):
    import bit_quantized_decode_qmv_amd as bq
    rng = np.random.default_rng(tokens * 1000 + D + rot)
    x = (rng.standard_normal((tokens, heads, D)) * np.exp(rng.uniform(-4, 4, (tokens, heads, 1)))).astype(np.float16)
    w = np.exp(rng.uniform(-1, 1, D)).astype(np.float32) * rng.choice([-1, 1], D).astype(np.float32)
    pos = rng.integers(0, 40000, (axes, tokens)).astype(np.int32)
    inv, axis = synth.rope_freqs(rot), rng.integers(0, axes, rot // 2).astype(np.int32)
    args = dict(pos=up(pos), inv_freq=up(inv), axis=up(axis), adjacent=adjacent) if rot else {}
    y = bq.norm_rope(up(x), up(w), 1e-5, **args).cpu().numpy()
    check(y, x, w, 1e-5, pos, inv, axis, adjacent)
    # the same bits on a strided view, in place, and on other streams
    torch = torch_mod()
    wide = torch.zeros((tokens, heads * D + 64), dtype=torch.float16, device="cuda:0")
    view = wide[:, 8:8 + heads * D].unflatten(1, (heads, D))
    view.copy_(up(x))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = bq.norm_rope(view, up(w), 1e-5, out=view, **args)
    s.synchronize()
    assert got is view and np.array_equal(view.cpu().numpy(), y)
    assert float(wide[:, :8].abs().max()) == 0 and float(wide[:, 8 + heads * D:].abs().max()) == 0


def test_zeros_infinities_and_nan_stay_in_their_row():
    import bit_quantized_decode_qmv_amd as bq
    rng = np.random.default_rng(1)
    x = rng.standard_normal((6, 2, 64)).astype(np.float16)
    w, pos, inv = np.ones(64, np.float32), np.arange(6)[None].astype(np.int32), synth.rope_freqs(64)
    y0 = bq.norm_rope(up(x), up(w), 1e-6, up(pos), up(inv)).cpu().numpy()
    x[0, 1], x[1, 0, 5], x[2, 1, 40], x[3, 0, 7] = 0, np.inf, np.nan, -np.inf
    y1 = bq.norm_rope(up(x), up(w), 1e-6, up(pos), up(inv)).cpu().numpy()
    hit = np.zeros((6, 2), bool)
    hit[0, 1] = hit[1, 0] = hit[2, 1] = hit[3, 0] = True
    assert np.array_equal(y0[~hit], y1[~hit]) and not y1[0, 1].any()
    # x / sqrt(inf) = 0 beside an infinity, which has no value itself
    assert np.isnan(y1[1, 0, 5]) and np.isnan(y1[3, 0, 7]) and np.isnan(y1[2, 1]).all()
    y2 = bq.norm_rope(up(x), up(w), 0.0).cpu().numpy()
    assert np.isnan(y2[0, 1]).all()                         # 0 / 0
    # the smallest and the largest of fp16: no square is lost, none overflows
    x = np.full((2, 1, 64), 2.0 ** -24, np.float16)
    x[1] = 65504
    check(bq.norm_rope(up(x), up(w), 0.0).cpu().numpy(), x, w, 0.0, pos, synth.rope_freqs(0), None, False)


def test_empty():
    import bit_quantized_decode_qmv_amd as bq
    torch = torch_mod()
    x = torch.empty((0, 4, 64), dtype=torch.float16, device="cuda:0")
    assert bq.norm_rope(x, up(np.ones(64, np.float32)), 1e-6).shape == (0, 4, 64)


def steps(value, scale, fmt):
    if fmt == "int8":
        return np.broadcast_to(scale, np.shape(value))
    a = np.abs(value) / np.where(scale > 0, scale, 1)
    return scale * 2.0 ** (np.floor(np.log2(np.maximum(a, 2.0 ** -6))) - 3)


def check_cache(got, before, fmt, layer, table, starts, news, cu, k, v, moved):
    """Every block of the cache: those that take new tokens hold them and their older ones, the others are as before."""
    qmax, zero = (127, 128) if fmt == "int8" else (448, 0)
    numbers = oracle.kv_table(fmt)
    rest = {x: np.ones(before[x].shape, bool) for x in ("k", "v", "ks", "vs")}
    for which, new, off in (("k", k, moved), ("v", v, 0.0)):
        D = new.shape[2]
        place = oracle.kv_places(which, D)
        for b, (start, n) in enumerate(zip(starts, news)):
            for block in range(start // 16, (start + n - 1) // 16 + 1) if n else ():
                page, i = int(table[b, block // 4]), block % 4
                tokens = np.arange(block * 16, block * 16 + 16)
                at = place[tokens % 64]                                            # [16][D]
                was, now = (c[which + "s"][layer, page, :, i].astype(np.float64) for c in (before, got))
                fresh = new[cu[b] + max(tokens[0] - start, 0):cu[b] + min(tokens[-1] + 1 - start, n)]  # [tokens][heads][D]
                size = np.where(np.isfinite(fresh), np.abs(fresh), 0).max((0, 2))
                scale = np.maximum(size / qmax, was if tokens[0] < start else 0)
                assert np.all(np.abs(now - scale) <= scale * 2.0 ** -22 + off / qmax), (which, "scale")
                held = numbers[got[which][layer, page][:, at]] * now[:, None, None]    # [heads][16][D]
                old = numbers[before[which][layer, page][:, at]] * was[:, None, None]
                for j, t in enumerate(tokens):
                    if t >= start + n:
                        assert np.all(got[which][layer, page][:, at[j]] == zero)
                        continue
                    exact = old[:, j] if t < start else new[cu[b] + t - start]
                    exact = np.where(np.isnan(exact), 0, np.clip(exact, -qmax * now[:, None], qmax * now[:, None]) if t >= start else exact)
                    step = np.maximum(steps(held[:, j], now[:, None], fmt), steps(exact, now[:, None], fmt))
                    assert np.all(np.abs(held[:, j] - exact) <= step / 2 + off + 2.0 ** -21 * np.abs(exact)), (which, t)
                for h in range(new.shape[1]):
                    rest[which][layer, page, h, at] = False
                    rest[which + "s"][layer, page, h, i] = False
    for x, m in rest.items():
        assert np.array_equal(got[x][m], before[x][m]), f"{x} of other blocks"


def run(rng, fmt, D, heads, q_heads, starts, news, axes=1, rot=None, adjacent=False, k_norm=True, q_norm=True, spoil=None):
    import bit_quantized_decode_qmv_amd as bq
    torch = torch_mod()
    lens = [s + n for s, n in zip(starts, news)]
    table, pages = synth.make_kv_table(rng, lens)
    before = synth.make_kv_pool(rng, 2, pages, heads, D, fmt)
    total = sum(news)
    qkv = (rng.standard_normal((total, (q_heads + 2 * heads), D)) * 3).astype(np.float16)
    q, k, v = qkv[:, :q_heads], qkv[:, q_heads:q_heads + heads], qkv[:, q_heads + heads:]
    if spoil:
        spoil(k)
    rot = D if rot is None else rot
    inv, axis = synth.rope_freqs(rot), (np.arange(rot // 2) % axes).astype(np.int32)
    pos = rng.integers(0, 30000, (axes, total)).astype(np.int32)
    kw, qw = (np.exp(rng.uniform(-1, 1, D)).astype(np.float32) for _ in range(2))
    cu, cache = cu_of(news), upload_cache(before)
    whole = up(qkv).flatten(1)
    a, b = q_heads * D, (q_heads + heads) * D
    dq, dk, dv = (whole[:, i:j].unflatten(1, (-1, D)) if j > i else None for i, j in ((0, a), (a, b), (b, b + heads * D)))
    args = dict(pos=up(pos), inv_freq=up(inv), axis=up(axis), adjacent=adjacent) if rot else {}
    out = bq.kv_append_norm(cache, 1, dk, dv, up(cu), up(lens, np.int32), up(table), q=dq, k_weight=up(kw) if k_norm else None,
                            q_weight=up(qw) if q_norm else None, eps=1e-6, **args)
    got = download_cache(cache)
    z = oracle.norm_f64(k, kw, 1e-6) if k_norm else k.astype(np.float64)
    moved = (2.0 ** -16 * bool(rot) + 2.0 ** -18 * k_norm) * float(np.max(np.abs(z[np.isfinite(z)])))
    check_cache(got, before, fmt, 1, table, starts, news, cu, oracle.rope_f64(z, pos, inv, axis, adjacent), v.astype(np.float64), moved)
    if q_heads:
        alone = bq.norm_rope(dq, up(qw), 1e-6, **args) if q_norm else bq.rope(dq, **args) if rot else dq
        assert torch.equal(out, alone)


APPENDS = [  # D, heads, q_heads, starts, news, axes, rot, adjacent
    (128, 2, 12, [0], [1], 1, 128, False),
    (128, 8, 48, [63, 0, 15, 64], [1, 1, 1, 1], 1, 128, False),
    (64, 1, 0, [5], [70], 1, 64, True),
    (128, 2, 4, [100, 0, 7, 33], [5, 0, 64, 3], 3, 64, False),
    (192, 1, 3, [17], [30], 2, 192, False),
    (192, 2, 3, [0, 3], [600, 2], 1, 128, False),      # pages whole: all four blocks a thread
    (256, 2, 4, [1, 129], [130, 2], 3, 128, False),
    (64, 3, 3, [40], [9], 1, 0, False),
]


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("D,heads,q_heads,starts,news,axes,rot,adjacent", APPENDS)
def test_append(fmt, D, heads, q_heads, starts, news, axes, rot, adjacent):
    run(np.random.default_rng(D + heads + sum(starts)), fmt, D, heads, q_heads, starts, news, axes, rot, adjacent)


@pytest.mark.parametrize("k_norm,q_norm", [(True, False), (False, True)])
def test_one_of_two_normed(k_norm, q_norm):
    run(np.random.default_rng(2), "int8", 128, 2, 4, [30, 1], [40, 1], k_norm=k_norm, q_norm=q_norm)


def test_keys_without_value():
    """Rows of zeros, and one with an infinity, whose other values are then 0 and itself no number: held as 0."""
    def spoil(k):
        k[3], k[40, 1, 9] = 0, np.inf
    run(np.random.default_rng(3), "int8", 64, 2, 0, [0], [66], rot=0, spoil=spoil)


def test_no_weights_is_the_append_itself():
    import bit_quantized_decode_qmv_amd as bq
    rng = np.random.default_rng(4)
    lens = [70, 9]
    table, pages = synth.make_kv_table(rng, lens)
    c = synth.make_kv_pool(rng, 1, pages, 2, 64, "int8")
    k, v, q = (up(rng.standard_normal((12, n, 64)).astype(np.float16)) for n in (2, 2, 6))
    pos, inv = up(np.arange(12)[None], np.int32), up(synth.rope_freqs(64))
    got = []
    for call in (bq.kv_append, bq.kv_append_norm):
        cache = upload_cache(c)
        out = call(cache, 0, k, v, up([0, 8, 12], np.int32), up(lens, np.int32), up(table), q=q, pos=pos, inv_freq=inv)
        got.append((out.cpu().numpy(), download_cache(cache)))
    assert np.array_equal(got[0][0], got[1][0])
    assert all(np.array_equal(got[0][1][x], got[1][1][x]) for x in ("k", "v", "ks", "vs"))


def test_helpers_refuse():
    import bit_quantized_decode_qmv_amd as bq
    torch = torch_mod()
    x = torch.zeros((2, 2, 64), dtype=torch.float16, device="cuda:0")
    w = torch.ones(64, device="cuda:0")
    bq.norm_rope(x, w, 1e-6)
    for bad in (w[:32], w.half(), w.cpu(), None, torch.ones(128, device="cuda:0")[::2]):
        with pytest.raises((ValueError, TypeError)):
            bq.norm_rope(x, bad, 1e-6)
    for eps in (-1.0, float("nan")):
        with pytest.raises(bq.BQError):
            bq.norm_rope(x, w, eps)
    cache = bq.KVCache.empty(1, 4, 2, 64)
    args = (cache, 0, x, x, up([0, 2], np.int32), up([2], np.int32), up([[0]], np.int32))
    for name in ("k_weight", "q_weight"):
        with pytest.raises((ValueError, TypeError)):
            bq.kv_append_norm(*args, q=x, **{name: w[:32]})
