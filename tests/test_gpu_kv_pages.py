"""GPU parity of the page operations: tables, lengths, reference counts and
page contents are whole numbers and must equal the oracle's."""
import numpy as np
import pytest

import oracle
from gpu_helpers import torch_mod
from kv_helpers import up

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    torch = torch_mod()
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    import bit_quantized_decode_qmv_amd as bq
    bq.load_library()


class State:
    """A pool on the GPU whose pages hold random bytes, and the oracle of it: a page's content is the id it started with."""

    def __init__(self, rng, lens, rows, pages, max_pages, layers=2, heads=2, D=64):
        import bit_quantized_decode_qmv_amd as bq
        lens = list(lens) + [0] * (rows - len(lens))
        order = rng.permutation(pages).tolist()
        table = [[order.pop() if c < -(-n // 64) else -1 for c in range(max_pages)] for n in lens]
        refs = [0] * pages
        for row in table:
            for p in row:
                if p >= 0:
                    refs[p] += 1
        self.codes = [rng.integers(0, 256, (layers, pages, heads, 64 * D)).astype(np.uint8) for _ in range(2)]
        self.scales = [rng.standard_normal((layers, pages, heads, 4)).astype(np.float32) for _ in range(2)]
        self.cache = bq.KVCache(*(up(c) for c in self.codes), *(up(s) for s in self.scales))
        self.model = oracle.PagesOracle(table, lens, refs, range(pages))
        self.table, self.lens, self.refs = (up(x, np.int32) for x in (table, lens, refs))

    def check(self, told, want):
        assert tuple(told.cpu().tolist()) == want
        m = self.model
        assert self.table.cpu().tolist() == m.table
        assert self.lens.cpu().tolist() == m.lens
        assert self.refs.cpu().tolist() == m.refs
        at = np.array(m.contents)
        # a free page's bytes are nobody's
        live = np.array(m.refs) > 0
        for got, was in zip((self.cache.k, self.cache.v, self.cache.k_scales, self.cache.v_scales), self.codes + self.scales):
            assert np.array_equal(got.cpu().numpy()[:, live], was[:, at][:, live])

    def fork(self, src, dst):
        import bit_quantized_decode_qmv_amd as bq
        told = bq.kv_fork(self.cache, self.table, self.lens, self.refs, up(src, np.int32), up(dst, np.int32))
        self.check(told, self.model.fork(src, dst))

    def resize(self, want):
        import bit_quantized_decode_qmv_amd as bq
        told = bq.kv_resize(self.cache, self.table, self.lens, self.refs, up(want, np.int32))
        self.check(told, self.model.resize(want))

    def compact(self):
        import bit_quantized_decode_qmv_amd as bq
        told = bq.kv_compact(self.cache, self.table, self.refs)
        self.check(told, self.model.compact())


def test_fork_cut_grow_free_compact():
    s = State(np.random.default_rng(0), [200, 64, 0, 130], 8, 30, 6)
    s.fork([0, 0, 1], [4, 5, 6])
    s.resize([-1, -1, 70, 100, 129, -1, 10, 0])      # grow, cut inside shared and own pages
    s.resize([0, -1, -1, -1, 128, -1, -1, -1])       # the first goes, its forks stay
    s.compact()
    s.compact()                                      # nothing left to move
    s.resize([384, -1, -1, -1, -1, -1, -1, -1])
    s.fork([4, 2], [7, 7])                           # a row twice: refused
    s.fork([4], [4])
    s.fork([0, 99], [7, 1])
    s.fork([0], [-1])
    s.fork([4], [7])
    s.resize([0] * 8)
    s.compact()


def test_every_row_cut_inside_one_shared_page():
    """All copies are made while the page is still shared; then nobody holds it."""
    s = State(np.random.default_rng(1), [192], 5, 12, 4)
    s.fork([0, 0, 0, 0], [1, 2, 3, 4])
    s.resize([100, 101, 102, 103, 104])
    s.resize([90, 80, -1, -1, -1])                   # their own pages now: no copies


def test_too_few_pages_changes_nothing():
    s = State(np.random.default_rng(2), [100, 100], 4, 5, 4)
    s.fork([0, 1], [2, 3])                           # one page short
    s.resize([256, 0, -1, -1])                       # the pages let go in the same call count
    s.resize([-1, 128, -1, -1])                      # 2 asked, 1 free
    s.resize([-2, -1, -1, -1])
    s.resize([-1, 257, -1, -1])


def test_random_steps():
    rng = np.random.default_rng(3)
    s = State(rng, [int(x) for x in rng.integers(0, 500, 10)], 16, 90, 10, layers=1, heads=1)
    for _ in range(30):
        kind = rng.integers(0, 3)
        lens = s.model.lens
        if kind == 0:
            empty = [i for i, n in enumerate(lens) if n == 0]
            n = int(rng.integers(0, len(empty) + 1))
            if n:
                s.fork([int(x) for x in rng.integers(0, 16, n)], [int(x) for x in rng.permutation(empty)[:n]])
        elif kind == 1:
            s.resize([int(x) for x in np.where(rng.random(16) < 0.4, rng.integers(0, 500, 16), -1)])
        else:
            s.compact()


@pytest.mark.parametrize("rows,pages,max_pages", [(3000, 9000, 3), (2, 40000, 300)])
def test_many_rows_and_pages(rows, pages, max_pages):
    """More rows and pages than the planning workgroup has threads."""
    rng = np.random.default_rng(rows)
    lens = [int(x) for x in rng.integers(0, 64 * max_pages + 1, rows // 2)]
    s = State(rng, lens, rows, pages, max_pages, layers=1, heads=1)
    n = rows - len(lens)
    s.fork([int(x) for x in rng.integers(0, len(lens), n)], list(range(len(lens), rows)))
    s.resize([int(x) for x in np.where(rng.random(rows) < 0.5, rng.integers(0, 64 * max_pages + 1, rows), -1)])
    s.compact()


@pytest.mark.parametrize("layers,heads,D", [(1, 1, 64), (3, 2, 192), (2, 8, 256)])
def test_copy_pages(layers, heads, D):
    import bit_quantized_decode_qmv_amd as bq
    rng = np.random.default_rng(layers)
    s = State(rng, [], 1, 9, 1, layers, heads, D)
    src, dst = [0, 3, 8, 9, -1, 5], [1, 2, 4, 6, 7, -7]     # the last three name no pages
    bq.kv_copy_pages(s.cache, up(src, np.int32), up(dst, np.int32))
    for got, was in zip((s.cache.k, s.cache.v, s.cache.k_scales, s.cache.v_scales), s.codes + s.scales):
        was = was.copy()
        was[:, [1, 2, 4]] = was[:, [0, 3, 8]]
        assert np.array_equal(got.cpu().numpy(), was)
