"""mla_cache_compact_rows moves exactly the listed rows of every layer, whatever the pages, types,
strides and lists, leaves everything else, and skips and reports bad lists."""
import numpy as np
import pytest
import torch

from pack_mla_cache_gb300 import ops

pytestmark = pytest.mark.gpu
DT = {0: torch.bfloat16, 1: torch.float8_e4m3fn, 2: torch.float8_e5m2}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from pack_mla_cache_gb300 import build
    build.build()
    ops.lib()


class Case:
    def __init__(self, starts, lists, fmt=0, block=16, layers=3, pad=0, width=None, seed=0, dim=576):
        rng = np.random.default_rng(seed)
        self.fmt, self.block, self.layers, self.dim = fmt, block, layers, dim
        self.entry = 576 + pad
        S = len(starts)
        self.width = width or max(1, max(len(x) for x in lists))
        pages = [max(1, (s + (max(x) if len(x) else 0)) // block + 1) for s, x in zip(starts, lists)]
        self.blocks = sum(pages) + 2
        ids = rng.permutation(self.blocks)
        self.table = np.zeros((S, max(pages)), np.int32)
        used = 0
        for s, p in enumerate(pages):
            self.table[s, :p] = ids[used:used + p]
            used += p
        self.starts, self.counts = np.array(starts, np.int32), np.array([len(x) for x in lists], np.int32)
        self.rows = np.zeros((S, self.width), np.int32)
        for s, x in enumerate(lists):
            self.rows[s, :len(x)] = x
        kind = np.uint16 if fmt == 0 else np.uint8
        self.host = rng.integers(0, np.iinfo(kind).max + 1, (layers, self.blocks, block, self.entry)).astype(kind)

    def expected(self, skip=()):
        want = self.host.copy()
        for s in range(len(self.starts)):
            if s in skip:
                continue
            at = lambda p: (self.table[s, p // self.block], p % self.block)
            for i in range(self.counts[s]):
                (b, r), (c, q) = at(self.starts[s] + i), at(self.starts[s] + self.rows[s, i])
                want[:, b, r, :self.dim] = self.host[:, c, q, :self.dim]
        return want

    def put(self):
        dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()
        self.cache = dev(self.host.view(np.int16) if self.fmt == 0 else self.host)
        self.ptrs = torch.tensor([self.cache[l].data_ptr() for l in range(self.layers)], dtype=torch.int64, device="cuda")
        self.d = [dev(x) for x in (self.table, self.starts, self.rows, self.counts)]
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        return self

    def run(self, **kw):
        es = self.entry
        ops.mla_cache_compact_rows(self.ptrs, DT[self.fmt], self.blocks, self.block, self.block * es, es, self.dim,
                                   *self.d, **{**dict(err_word=self.err), **kw})
        return self

    def check(self, err=0, skip=()):
        torch.cuda.synchronize()
        got = self.cache.cpu().numpy()
        assert np.array_equal(got.view(self.host.dtype), self.expected(skip))
        assert int(self.err.item()) == err


def lists_of(rng, n, most, longest):
    return [sorted(rng.choice(most, int(rng.integers(0, min(most, longest) + 1)), replace=False).tolist()) for _ in range(n)]


@pytest.mark.parametrize("fmt", [0, 1, 2])
@pytest.mark.parametrize("block", [1, 7, 16, 64])
def test_moves(fmt, block):
    rng = np.random.default_rng(block)
    lists = lists_of(rng, 6, 61, 12) + [[0, 1, 2], [5], [], [3, 4, 5, 6], list(range(1, 61))]
    starts = [int(x) for x in rng.integers(0, 200, len(lists))]
    Case(starts, lists, fmt, block).put().run().check()


@pytest.mark.parametrize("kw", [dict(pad=16), dict(dim=512), dict(layers=1), dict(layers=61), dict(width=40), dict(dim=16, pad=48)])
def test_layouts(kw):
    rng = np.random.default_rng(1)
    lists = lists_of(rng, 5, 40, 20)
    Case([int(x) for x in rng.integers(0, 90, 5)], lists, int(rng.integers(0, 3)), **kw).put().run().check()


def test_long_lists():
    """Lists of up to 1024 rows: every step reads before it is overwritten."""
    rng = np.random.default_rng(4)
    full = list(range(1024))
    late = list(range(9, 1033))
    odd = sorted(rng.choice(4000, 1024, replace=False).tolist())
    Case([3, 70, 0], [full, late, odd], 1, 64, layers=2).put().run().check()


def test_many_sequences():
    rng = np.random.default_rng(6)
    Case([int(x) for x in rng.integers(0, 60, 3000)], lists_of(rng, 3000, 20, 6), 2, 16, layers=2).put().run().check()


@pytest.mark.parametrize("bad,bit", [("twice", "POS"), ("falling", "POS"), ("below", "POS"), ("start", "POS"), ("count", "POS"),
                                     ("over", "POS"), ("block", "BLOCK"), ("behind", "BLOCK"), ("wide", "BLOCK")])
def test_bad_sequences_are_left_and_reported(bad, bit):
    c = Case([10, 20, 30], [[1, 4, 6], [2, 5, 9, 30], [0, 7]], 1, 16)
    if bad == "twice":
        c.rows[1, 2] = 5
    elif bad == "falling":
        c.rows[1, 3] = 3
    elif bad == "below":
        c.rows[1, 0] = -1
    elif bad == "start":
        c.starts[1] = -1
    elif bad == "count":
        c.counts[1] = -2
    elif bad == "over":
        c.counts[1] = c.width + 1
    elif bad == "block":
        c.table[1, (20 + 9) // 16] = c.blocks
    elif bad == "behind":
        c.rows[1, 3] = c.table.shape[1] * 16
    else:
        c.starts[1] = 2 ** 31 - 5
    c.put().run().check(err=getattr(ops, f"MLA_ERRBIT_{bit}_OOB"), skip=(1,))


def test_bad_layer_is_skipped():
    c = Case([10], [[1, 4, 6]], 0, 16).put()
    c.ptrs[1] = 0
    c.run()
    torch.cuda.synchronize()
    want = c.expected()
    want[1] = c.host[1]
    assert np.array_equal(c.cache.cpu().numpy().view(np.uint16), want)
    assert int(c.err.item()) == ops.MLA_ERRBIT_MISALIGNED


def test_wide_tables_and_lists_streams_and_graphs():
    c = Case([10, 50], [[1, 4, 6], [0, 2, 30]], 0, 16).put()
    wide = torch.full((2, c.table.shape[1] + 3), -1, dtype=torch.int32, device="cuda")
    wide[:, :c.table.shape[1]] = c.d[0]
    lists = torch.full((2, c.width + 5), -1, dtype=torch.int32, device="cuda")
    lists[:, :c.width] = c.d[2]
    c.d[0], c.d[2] = wide[:, :c.table.shape[1]], lists[:, :c.width]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        c.run(stream=s)
    g.replay()
    c.check()


def test_offsets_past_32_bits():
    """A cache of 6 GB whose used blocks are its last ones."""
    c = Case([3, 100], [[1, 4, 6], [0, 2, 30]], block=64, layers=1).put()
    blocks, far = c.blocks, 80000
    big = torch.empty((far, 64, 576), dtype=torch.int16, device="cuda")
    big[far - blocks:].copy_(c.cache[0])
    c.ptrs = torch.tensor([big.data_ptr()], dtype=torch.int64, device="cuda")
    c.d[0] += far - blocks
    c.blocks = far
    c.run()
    c.cache[0].copy_(big[far - blocks:])
    c.check()


def test_device_refusals():
    c = Case([3], [[1, 4]]).put()
    c.d[2] = c.d[2].cpu()
    with pytest.raises(ops.MlaError, match="rows must be device memory"):
        c.run()
