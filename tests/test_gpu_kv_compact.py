"""rc_kv_compact against the move done row by row on the host, every byte of every
cache compared."""
import pytest
import torch

import rope_chain_gb300 as rc

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, I32 = torch.bfloat16, torch.int32


@pytest.fixture(scope="module", autouse=True)
def built():
    from rope_chain_gb300 import _build
    _build.build()


class Case:
    def __init__(self, counts, ctx, paths, H, bs, widths=((128, BF),), width=None, seed=0):
        gen = torch.Generator().manual_seed(seed + sum(counts))
        need = [-(-(c + n) // bs) for c, n in zip(ctx, counts)]
        nb = sum(need) + 3
        order = torch.randperm(nb, generator=gen).tolist()
        self.nb, self.bs = nb, bs
        table = torch.zeros(len(counts), max(need + [1]), dtype=I32)
        for b, n in enumerate(need):
            table[b, :n] = torch.tensor([order.pop() for _ in range(n)], dtype=I32)
        self.table = table.to(DEV)
        self.counts, self.ctx, self.paths = counts, ctx, paths
        most = max([len(p) for p in paths] + [1]) if width is None else width
        path = torch.full((len(counts), most), -9, dtype=I32)
        for b, p in enumerate(paths):
            path[b, :len(p)] = torch.tensor(p, dtype=I32)
        self.path = path.to(DEV)
        self.path_len = torch.tensor([len(p) for p in paths], dtype=I32, device=DEV)
        self.context = torch.tensor(ctx, dtype=I32, device=DEV)
        self.row_start = torch.tensor([0] + counts, device=DEV).cumsum(0).to(I32)
        self.caches = []
        for w, dtype in widths:
            bits = torch.randint(0, 256, (nb, H, bs, w * torch.empty(0, dtype=dtype).element_size()), dtype=torch.uint8, generator=gen)
            self.caches.append(bits.to(DEV).view(dtype))

    def want(self, valid=None):
        """The caches after the move, and the new lengths; `valid`: entries of each path that count."""
        out = [c.view(torch.uint8).cpu().clone() for c in self.caches]
        old = [c.clone() for c in out]
        table = self.table.cpu()
        lens = []
        for b, p in enumerate(self.paths):
            m = len(p) if valid is None else valid[b]
            for k in range(m):
                s, d = self.ctx[b] + p[k], self.ctx[b] + k
                for c, o in zip(out, old):
                    c[table[b, d // self.bs], :, d % self.bs] = o[table[b, s // self.bs], :, s % self.bs]
            lens.append(self.ctx[b] + m)
        return out, torch.tensor(lens, dtype=I32)

    def run(self, **kw):
        return rc.kv_compact(self.caches, self.table, self.context, self.row_start, self.path, self.path_len, **kw)

    def check(self, valid=None, errors=0, **kw):
        caches, lens = self.want(valid)
        err = torch.zeros(1, dtype=I32, device=DEV)
        new = self.run(err=err, **kw)
        assert torch.equal(new.cpu(), lens) and int(err) == errors
        for got, want in zip(self.caches, caches):
            assert torch.equal(got.view(torch.uint8).cpu(), want)


KV4 = ((64, torch.uint8), (4, BF))


@pytest.mark.parametrize("counts,ctx,paths,H,bs", [
    ([1], [0], [[0]], 1, 1),
    ([13], [1500], [[0, 2, 3, 7]], 8, 16),
    ([13, 12, 5], [30, 0, 511], [[0, 1, 2, 3], [3, 4, 5, 6, 7, 11], [4]], 2, 16),
    ([4, 0, 9], [10, 20, 30], [[], [], [1, 2, 8]], 3, 7),
    ([64] * 3, [100, 17, 64], [list(range(1, 64)), list(range(0, 64, 3)), [63]], 4, 32),
    ([400], [77], [list(range(1, 390))], 2, 16),
    ([700], [5], [[i + (i > 128) * 37 + (i > 300) * 200 for i in range(450)]], 1, 48),
    ([40], [1000], [list(range(40))], 16, 128),
    ([20], [9], [[0, 1, 2, 5, 6, 7, 8, 9, 10, 11, 12, 13, 14, 15, 16, 18, 19]], 1, 1),
])
@pytest.mark.parametrize("widths", [((128, BF),), KV4, ((128, BF), (64, torch.uint8), (4, BF), (3, torch.float64))])
def test_against_rows_one_by_one(counts, ctx, paths, H, bs, widths):
    Case(counts, ctx, paths, H, bs, widths).check()


def test_many_caches_and_sequences():
    counts = [1 + b % 17 for b in range(200)]
    paths = [sorted({(b * 7 + i * 3) % n for i in range(1 + b % 6)}) for b, n in enumerate(counts)]
    Case(counts, [b * 3 for b in range(200)], paths, 2, 16, ((128, BF),) * 5 + KV4 * 3).check()


def test_paths_that_end_early():
    """Not increasing, outside the tree, negative, or longer than there are entries."""
    paths = [[0, 2, 2, 5], [1, 6], [-1, 3], [2, 1, 3], [0, 1, 2, 3]]
    c = Case([6, 6, 6, 6, 6], [10] * 5, paths, 2, 16)
    c.check(valid=[2, 1, 0, 1, 4], errors=4)
    c = Case([6], [10], [[1, 2]], 2, 16)
    c.path_len[0] = 5                                       # clamped to the two entries
    c.check()
    c = Case([6], [10], [[1, 2]], 2, 16)
    c.path_len[0] = -3
    c.check(valid=[0])


def test_a_long_path_that_ends_in_a_later_part():
    p = list(range(1, 300))
    p[200] = 5
    Case([400], [33], [p], 2, 16).check(valid=[200], errors=1)


def test_blocks_that_are_missing():
    c = Case([20, 20], [30, 30], [[0, 4, 12, 19], [3, 5]], 2, 16)
    c.table[0, 3] = -1                                      # keys 48 to 63: node 19 (key 49) is gone
    c.table[1, 2] = c.nb                                    # keys 32 to 47: nodes 2 to 17
    c.check(valid=[3, 0], errors=2)
    c = Case([20], [30], [[0, 4, 12, 19]], 2, 16)
    c.table = c.table[:, :3].contiguous()                   # nothing past key 47
    c.check(valid=[3], errors=1)
    c = Case([20], [30], [[0, 4, 12, 19]], 2, 16)
    c.table = c.table[:, :0]
    c.check(valid=[0], errors=1)


def test_no_paths_at_all():
    Case([3, 2], [5, 6], [[], []], 2, 16, width=0).check()


def test_strided_tables_and_paths():
    c = Case([13, 12], [30, 40], [[0, 2, 3, 7], [1, 2, 4]], 2, 16)
    c.table = torch.cat([c.table, c.table + 1], 1)[:, :c.table.shape[1]]
    c.path = torch.cat([c.path, c.path], 1)[:, :c.path.shape[1]]
    new = torch.empty(2, dtype=I32, device=DEV)
    c.check(new_len=new)
    assert new.tolist() == [34, 43]


def test_captured_and_replayed_with_another_path():
    c = Case([13], [30], [[0, 2, 3, 7]], 4, 16, ((128, BF),) + KV4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    saved = [x.clone() for x in c.caches]
    with torch.cuda.stream(side):
        c.run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        new = c.run()
    for x, y in zip(c.caches, saved):
        x.copy_(y)
    c.paths = [[1, 5]]
    c.path[0, :2] = torch.tensor([1, 5], dtype=I32)
    c.path_len[0] = 2
    caches, lens = c.want()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(new.cpu(), lens) and all(torch.equal(g.view(torch.uint8).cpu(), w) for g, w in zip(c.caches, caches))


def test_rows_past_32_bits():
    """A cache of more than 2^32 bytes."""
    c = Case([8], [20], [[1, 3, 6]], 1, 16)
    big = torch.zeros(33000, 8, 64, 128, dtype=BF, device=DEV)
    big[-1] = torch.randn(8, 64, 128, device=DEV).to(BF)
    table = torch.full((1, 1), 32999, dtype=I32, device=DEV)
    want = big[-1].clone()
    for k, j in enumerate([1, 3, 6]):
        want[:, 20 + k] = big[-1][:, 20 + j]
    rc.kv_compact([big], table, c.context, c.row_start, c.path, c.path_len)
    assert torch.equal(big[-1], want) and not bool(big[:-1].any())
