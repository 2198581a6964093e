"""GPU parity of bq_kv_append and bq_kv_read against the fp64 oracle.

Tolerances.  The rotated k is within d = 2^-17 (|x1| + |x2|) of the exact one
(angle and hardware sine, as in the tests of bq_rope), at most 2^-16 of the
largest |x| of the call.  The block scale, a maximum of such values over 127
or 448, moves by no more than d over that and by fp32 roundings (2^-22
relative).  A held value is within half a code step of the exact one plus what
x and the scale moved: the step is the scale (int8), or 2^-3 of the value's
power of two, at least 2^-9 scales (e4m3), and a value that lies within the
movement of a step's middle may take either neighbour."""
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


def steps(value, scale, fmt):
    if fmt == "int8":
        return scale
    a = np.abs(value) / np.where(scale > 0, scale, 1)
    return scale * 2.0 ** (np.floor(np.log2(np.maximum(a, 2.0 ** -6))) - 3)


def check_cache(got, want, before, fmt, touched, moved):
    """got, want: caches; touched: (layer, page, block) of written blocks; moved: bound on the rotated values' error."""
    D = got["k"].shape[3] // 64
    table = oracle.kv_table(fmt)
    mask = np.zeros(got["ks"].shape[:2] + (4,), bool)
    for layer, page, block in touched:
        mask[layer, page, block] = True
    for w in ("k", "v"):
        off = moved if w == "k" else 0.0
        place = oracle.kv_places(w, D)
        g, x, b = (c[w][..., place.ravel()].reshape(*c[w].shape[:3], 4, 16 * D) for c in (got, want, before))
        gs, xs = got[w + "s"].astype(np.float64), want[w + "s"].astype(np.float64)
        m = np.broadcast_to(mask[:, :, None], gs.shape)
        assert np.array_equal(g[~m], b[~m]) and np.array_equal(got[w + "s"][~m], before[w + "s"][~m]), "untouched blocks"
        qmax = 127 if fmt == "int8" else 448
        tol = xs * 2.0 ** -22 + off / qmax
        assert np.all(np.abs(gs - xs)[m] <= tol[m]), f"{w} scales"
        gv, xv = table[g] * gs[..., None], table[x] * xs[..., None]
        # the two may be neighbouring codes where the exact value is near a middle
        gap = np.abs(gv - xv)
        step = np.maximum(steps(gv, gs[..., None], fmt), steps(xv, xs[..., None], fmt))
        near = np.abs(xv) * 2.0 ** -21 + off * (1 + np.abs(table[x]) / qmax)
        assert np.all((gap <= step * 1.0001 + near)[m]), f"{w} values"
        # and differ by a step only rarely: the movement covers this share of a step (plus one value)
        share = np.mean((gap > near + 1e-6 * step)[m]) if m.any() else 0
        expect = 4 * np.mean((near / np.where(step > 0, step, 1))[m]) if m.any() else 0
        assert share <= expect + 3 / max(1, m.sum() * 16 * D) + 1e-4, (w, share, expect)


def run(rng, fmt, D, heads, q_heads, starts, news, axes=1, rot=None, adjacent=False, layers=2, layer=1, spoil=None,
        strided=False):
    import bit_quantized_decode_qmv_amd as bq
    lens = [s + n for s, n in zip(starts, news)]
    table, pages = synth.make_kv_table(rng, lens)
    before = synth.make_kv_pool(rng, layers, pages, heads, D, fmt)
    total = sum(news)
    k, v = (rng.standard_normal((total, heads, D)).astype(np.float16) for _ in range(2))
    if spoil:
        spoil(k, v)
    q = rng.standard_normal((total, q_heads, D)).astype(np.float16) if q_heads else None
    rot = D if rot is None else rot
    inv = synth.rope_freqs(rot)
    axis = (np.arange(rot // 2) % axes).astype(np.int32)
    pos = rng.integers(0, 30000, (axes, total)).astype(np.int32)
    cu = cu_of(news)
    cache = upload_cache(before)
    dk, dv, dq = up(k), up(v), up(q) if q_heads else None
    if strided:
        torch = torch_mod()
        whole = torch.cat([t.flatten(1) for t in (dq, dk, dv)], 1)
        a, b = q_heads * D, (q_heads + heads) * D
        dq, dk, dv = (whole[:, i:j].unflatten(1, (-1, D)) for i, j in ((0, a), (a, b), (b, b + heads * D)))
    args = dict(pos=up(pos), inv_freq=up(inv), axis=up(axis), adjacent=adjacent) if rot else {}
    out = bq.kv_append(cache, layer, dk, dv, up(cu), up(lens, np.int32), up(table), q=dq, **args)
    got = download_cache(cache)
    want = {x: y.copy() if x != "format" else y for x, y in before.items()}
    turned = oracle.rope_f64(k, pos, inv, axis, adjacent)
    touched = []
    for b, (s, n) in enumerate(zip(starts, news)):
        if n:
            oracle.kv_append_f64(want, layer, table[b], s, turned[cu[b]:cu[b + 1]], v[cu[b]:cu[b + 1]].astype(np.float64))
            touched += [(layer, table[b, i // 4], i % 4) for i in range(s // 16, (s + n - 1) // 16 + 1)]
    finite = np.abs(k[np.isfinite(k)]).max() if total else 0
    check_cache(got, want, before, fmt, touched, 2.0 ** -16 * float(finite) if rot else 0.0)
    if q_heads:
        alone = bq.rope(dq, **args) if rot else dq
        assert np.array_equal(out.cpu().numpy(), alone.cpu().numpy())
    return cache, got, table, lens, cu


CASES = [  # D, heads, q_heads, starts, news, axes, rot, adjacent
    (128, 2, 12, [0], [1], 1, 128, False),            # the first token of all
    (128, 8, 48, [63, 0, 15, 64], [1, 1, 1, 1], 1, 128, False),
    (64, 1, 0, [5], [70], 1, 64, True),               # across blocks and a page, behind older tokens
    (128, 2, 4, [100, 0, 7, 33], [5, 0, 64, 3], 3, 64, False),
    (192, 1, 3, [17], [30], 2, 192, False),
    (256, 2, 4, [1, 129], [130, 2], 3, 128, False),
    (64, 3, 0, [40], [9], 1, 0, False),
]


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("D,heads,q_heads,starts,news,axes,rot,adjacent", CASES)
def test_append(fmt, D, heads, q_heads, starts, news, axes, rot, adjacent):
    rng = np.random.default_rng(D + heads + sum(starts))
    run(rng, fmt, D, heads, q_heads, starts, news, axes, rot, adjacent)


def test_rows_of_a_fused_product():
    run(np.random.default_rng(3), "int8", 128, 2, 6, [9, 200], [40, 3], strided=True)


def test_many_sequences():
    """More sequences than a wave has lanes, some without rows."""
    rng = np.random.default_rng(4)
    starts = rng.integers(0, 90, 150).tolist()
    news = rng.integers(0, 4, 150).tolist()
    run(rng, "int8", 64, 1, 2, starts, news)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_zeros_infinities_and_nan(fmt):
    def spoil(k, v):
        k[0:20] = 0                                   # whole blocks of zeros
        v[3, 0, 5], v[40, 1, 9], v[41, 0, 60] = np.inf, -np.inf, np.nan
        v[48:64] = np.inf                             # nothing finite in the block
    run(np.random.default_rng(5), fmt, 64, 2, 0, [0], [66], rot=0, spoil=spoil)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_one_at_a_time_and_rewritten(fmt):
    """Tokens written one by one: a block's scale is the running maximum, codes follow; then a rejected token is replaced."""
    import bit_quantized_decode_qmv_amd as bq
    rng = np.random.default_rng(6)
    D, heads, n = 64, 2, 21
    table, pages = synth.make_kv_table(rng, [n])
    before = synth.make_kv_pool(rng, 1, pages, heads, D, fmt)
    cache, want = upload_cache(before), {x: y.copy() if x != "format" else y for x, y in before.items()}
    kv = rng.standard_normal((2, n, heads, D)).astype(np.float16) * np.linspace(0.1, 3, n)[None, :, None, None].astype(np.float16)
    for t in list(range(n)) + [n - 2]:
        k, v = kv[0, t:t + 1], kv[1, t:t + 1]
        bq.kv_append(cache, 0, up(k), up(v), up([0, 1], np.int32), up([t + 1], np.int32), up(table))
        oracle.kv_append_f64(want, 0, table[0], t, k.astype(np.float64), v.astype(np.float64))
    got = download_cache(cache)
    for w in ("k", "v"):
        for b in range(2):
            assert np.allclose(got[w + "s"][0, table[0, 0], :, b], want[w + "s"][0, table[0, 0], :, b], rtol=2.0 ** -20, atol=0)
        g, x = (oracle.kv_sequence(c, 0, table[0], n, w) for c in (got, want))
        # each growth of the scale rounds the older codes once more; fp32 against fp64 may take the other neighbour
        step = np.repeat(want[w + "s"][0, table[0, 0]], 16, axis=-1)[:, :n].T[..., None] * (1 if fmt == "int8" else 32)
        assert np.all(np.abs(g - x) <= step * 1.001) and np.mean(np.abs(g - x) > 1e-3 * step) < 0.01


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_read(fmt):
    import bit_quantized_decode_qmv_amd as bq
    rng = np.random.default_rng(8)
    D, heads = 128, 3
    lens, counts = [100, 0, 64, 7, 200], [33, 2, 64, 9, 0]      # row 1 and 3 ask for more than is held
    table, pages = synth.make_kv_table(rng, lens)
    table[0, 1] = pages + 5                                     # a page that is none
    c = synth.make_kv_pool(rng, 2, pages, heads, D, fmt)
    cu = cu_of(counts)
    k, v = bq.kv_read(upload_cache(c), 1, up(cu), up(lens, np.int32), up(table), int(cu[-1]))
    for b, (n, m) in enumerate(zip(lens, counts)):
        for got, w in ((k, "k"), (v, "v")):
            want = np.zeros((m, heads, D))
            held = oracle.kv_sequence(c, 1, table[b], n, w)[max(n - m, 0):] if n else want[:0]
            if m:
                want[m - len(held):] = held
            # one rounding to fp16 of a product of two floats that is exact in fp32 up to 2^-24
            np.testing.assert_allclose(got[cu[b]:cu[b + 1]].cpu().numpy(), want, rtol=2.0 ** -11 + 2.0 ** -23, atol=2.0 ** -25)


def test_arrays_that_do_not_fit_are_not_followed():
    """Lengths past the table, page ids out of range, cu past total: nothing outside the pages of the rows is written."""
    import bit_quantized_decode_qmv_amd as bq
    rng = np.random.default_rng(9)
    D, heads, pages = 64, 1, 3
    before = synth.make_kv_pool(rng, 1, pages, heads, D, "int8")
    cache = upload_cache(before)
    k, v = (up(rng.standard_normal((6, heads, D)).astype(np.float16)) for _ in range(2))
    table = up([[-1, 3], [1 << 30, -5]], np.int32)
    bq.kv_append(cache, 0, k, v, up([0, 3, 900], np.int32), up([70, 1 << 30], np.int32), table)
    got = download_cache(cache)
    assert all(np.array_equal(got[x], before[x]) for x in ("k", "v", "ks", "vs"))
