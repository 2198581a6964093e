"""GPU parity of bq_kv_attn_sinks and bq_kv_attn_tree with many rows where a
workspace has room for few parts, so that the parts of the tiles are 12 pages
and more: how long they are is then searched for.  What lies in the workspace
ahead of the call, NaN here, and behind it is not touched.  Tolerance: that of
the tests of bq_kv_attn; a sum over several parts is one of fp32 numbers."""
import numpy as np
import pytest

import oracle
import synth
from gpu_helpers import torch_mod
from kv_helpers import cu_of, up, upload_cache
from test_gpu_kv_attn_tree import check, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    torch = torch_mod()
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    import bit_quantized_decode_qmv_amd as bq
    bq.load_library()


def uneven(seed, n, lo, hi, long=()):
    lens = [int(x) for x in np.random.default_rng(seed).integers(lo, hi, n)]
    for i in long:
        lens[i] = 3800
    return lens


SHORT, LONG = uneven(1, 70, 30, 330, (3, 20, 66)), uneven(2, 70, 600, 2600)
CASES = [  # kind, format, D, heads, group, lens, news, window, sinks, parts to aim at; a part's pages
    ("tree", "int8", 64, 1, 2, [4000], [20], 0, 0, 4),                       # 16, the first that is tried
    ("tree", "int8", 64, 1, 2, [2500, 2600], [20, 40], 0, 0, 5),             # 20, the fourth
    ("tree", "e4m3", 128, 2, 3, [2460, 900], [61, 13], 0, 0, 5),             # 20, the second; a tile more than sequences
    ("tree", "int8", 64, 1, 2, [26000, 20000], [20, 30], 0, 0, 5),           # 159, the last, in steps of 3
    ("tree", "int8", 64, 1, 2, [26000, 25000], [20, 30], 0, 0, 5),           # none fits: 170
    ("tree", "int8", 64, 1, 2, SHORT, [17] * 70, 0, 0, 20),                  # more tiles than parts: 22
    ("tree", "int8", 64, 1, 2, LONG, [17] * 70, 0, 0, 128),                  # 20, the last
    ("tree", "e4m3", 64, 1, 2, LONG, [17] * 70, 0, 0, 100),                  # none: 21
    ("tree", "int8", 64, 2, 4, [9000, 5000, 70], [13, 70, 20], 4000, 150, 7),  # none: 42
    ("sinks", "int8", 64, 1, 2, [4000], [20], 3000, 70, 3),                  # 17, the first
    ("sinks", "int8", 64, 1, 2, [2500, 2600], [20, 40], 2200, 4, 5),         # 19, the fifth
    ("sinks", "e4m3", 128, 1, 3, [5000, 3500], [60, 100], 0, 3, 12),        # 28, the second
    ("sinks", "int8", 64, 1, 2, SHORT, [17] * 70, 3000, 70, 20),             # none: 20
    ("sinks", "int8", 64, 1, 2, LONG, [17] * 70, 2000, 64, 128),             # 17, the fourth
    ("sinks", "e4m3", 64, 1, 2, LONG, [17] * 70, 2300, 64, 95),              # none: 22
]


@pytest.mark.parametrize("kind,fmt,D,heads,group,lens,news,window,sinks,target", CASES)
def test_long_parts(kind, fmt, D, heads, group, lens, news, window, sinks, target):
    import bit_quantized_decode_qmv_amd as bq
    torch = torch_mod()
    rng = np.random.default_rng(sum(lens) + target)
    c, table, q, cu = make(rng, fmt, D, heads, group, lens, news)
    tiles = len(lens) + sum(news) * group // 128
    size = bq.KV_ATTN_COUNTER_BYTES + (tiles + target) * heads * 128 * (D + 2) * 4
    guarded = torch.full((size + (1 << 20),), 255, dtype=torch.uint8, device="cuda:0")
    workspace = guarded[:size]
    workspace[:bq.KV_ATTN_COUNTER_BYTES] = 0
    args = (upload_cache(c), 1, up(q), up(cu), up(lens, np.int32), up(table))
    how = dict(window=window, sinks=sinks, workspace=workspace)
    if kind == "tree":
        parents = [synth.make_tree(rng, n, 7) for n in news]
        mask, _ = bq.tree_plan(up(np.concatenate(parents), np.int32), args[3], args[4], -(-max(news) // 64), window)
        seen = [oracle.tree_context(n, m - n, oracle.tree_seen(p, window), window, sinks) for n, m, p in zip(news, lens, parents)]
        call = lambda: bq.kv_attn_tree(*args, mask, **how)
    else:
        seen = [oracle.causal_context(n, m - n, window, sinks) for n, m in zip(news, lens)]
        call = lambda: bq.kv_attn(*args, **how)
    out = call()
    check(out.cpu().numpy(), c, 1, table, lens, cu, q, D ** -0.5, seen)
    assert torch.equal(out, call())
    assert bool((guarded[size:] == 255).all()) and not bool(guarded[:bq.KV_ATTN_COUNTER_BYTES].any())


@pytest.mark.parametrize("pages,parts", [([16, 1, 1], 16), ([17, 1, 1], 9), ([61, 1, 1, 1], 31), ([16, 16], 32)])
def test_parts_of_a_page(pages, parts):
    """A part is one page where no tile has more than 16, however few the others have: a tile of more is not cut into as
    many parts as it has pages.  Parts of a head are counted by what they leave in the workspace."""
    import bit_quantized_decode_qmv_amd as bq
    torch = torch_mod()
    rng = np.random.default_rng(sum(pages))
    lens, news, D = [64 * p - 3 for p in pages], [13] * len(pages), 64
    c, table, q, cu = make(rng, "int8", D, 2, 6, lens, news)
    args = (upload_cache(c), 1, up(q), up(cu), up(lens, np.int32), up(table))
    parents = [synth.make_tree(rng, n, 4) for n in news]
    mask, _ = bq.tree_plan(up(np.concatenate(parents), np.int32), args[3], args[4])
    slot = 128 * (D + 2) * 4
    workspace = torch.full((bq.KV_ATTN_COUNTER_BYTES + 200 * slot,), 255, dtype=torch.uint8, device="cuda:0")
    workspace[:bq.KV_ATTN_COUNTER_BYTES] = 0
    out = bq.kv_attn_tree(*args, mask, workspace=workspace).cpu().numpy()
    check(out, c, 1, table, lens, cu, q, D ** -0.5, [oracle.tree_context(13, m - 13, oracle.tree_seen(p)) for p, m in zip(parents, lens)])
    written = (workspace[bq.KV_ATTN_COUNTER_BYTES:].view(200, slot) != 255).any(1)
    assert int(written.sum()) == 2 * parts
