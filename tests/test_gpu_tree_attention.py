"""rc_tree_attention against the formula in 64 bits: trees, chains, single
tokens, empty rows, odd sizes, strides, pages that end inside a tile, blocks
out of range, infinities and NaN in what a row does not see.

Tolerance, per output with A = sum_p w_p |v_p| / sum_p w_p: the output's
rounding 2^-8 |ref|, the weights' rounding 2^-8 A, and 2^-12 A for FP32
scores, exponentials and sums (scores of 64 products of unit-variance values:
64 * 2^-24 * sum|q k| * scale < 2^-14, the exponential's 2^-22).  Log sums:
64 * 2^-24 times the largest scale * sum|q k|, plus 2^-20 (1 + |lse|)."""
import numpy as np
import pytest
import torch

import rope_chain_gb300 as rc

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def built():
    from rope_chain_gb300 import _build
    _build.build()
    rc.read_device_faults(clear=True)
    yield
    assert rc.read_device_faults(clear=True) == 0


def random_mask(rng, counts, words, empty=0.0):
    """Ancestor bits of random trees (bool per sequence and packed words)."""
    rows, bits = [], []
    for n in counts:
        m = np.zeros((n, n), dtype=bool)
        for i in range(n):
            if i and rng.random() < 0.9:
                m[i] = m[rng.integers(max(0, i - 4), i)]
            m[i, i] = True
        if empty:
            m[rng.random(n) < empty] = False
        rows.append(m)
        w = np.zeros((n, words), dtype=np.uint64)
        for j in range(min(n, 64 * words)):
            w[:, j // 64] |= m[:, j].astype(np.uint64) << np.uint64(j % 64)
        bits.append(w)
        m[:, 64 * words:] = False
    packed = np.concatenate(bits) if bits else np.zeros((0, words), dtype=np.uint64)
    return rows, torch.from_numpy(packed.view(np.int64)).to(DEV)


class Case:
    """Operands over a cache whose unused rows hold NaN."""

    def __init__(self, seed, counts, ctx, H, G, bs, *, mask="tree", words=None, spare=3, sigma=1.0, empty=0.0,
                 pad_rows=0, q_extra=64):
        rng = np.random.default_rng(seed)
        gen = torch.Generator(device=DEV).manual_seed(seed)
        self.counts, self.ctx, self.H, self.G, self.bs = counts, ctx, H, G, bs
        need = [-(-(c + n) // bs) for c, n in zip(ctx, counts)]
        nb = sum(need) + spare
        order = rng.permutation(nb)
        width = max(need + [1])
        table = np.zeros((len(counts), width), dtype=np.int32)
        self.cache = torch.full((nb, H, bs, 128), float("nan"), dtype=torch.bfloat16, device=DEV)
        self.kv = []
        at = 0
        for b, (c, n) in enumerate(zip(ctx, counts)):
            pages = order[at:at + need[b]]
            at += need[b]
            table[b, :need[b]] = pages
            kv = torch.randn(c + n, H, 128, generator=gen, device=DEV).mul_(sigma).to(torch.bfloat16)
            p = torch.arange(c + n, device=DEV)
            blk = torch.from_numpy(pages.astype(np.int64)).to(DEV)[p // bs]
            self.cache[blk, :, p % bs] = kv
            self.kv.append(kv)
        self.table = torch.from_numpy(table).to(DEV)
        self.rows = sum(counts) + pad_rows
        self.q = torch.randn(self.rows, H * G * 64 + q_extra, generator=gen, device=DEV).mul_(sigma).to(
            torch.bfloat16)[:, :H * G * 64].view(self.rows, H * G, 64)
        self.row_start = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device=DEV)
        self.context = torch.tensor(ctx, dtype=torch.int32, device=DEV)
        if mask == "tree":
            words = words or max(1, -(-max(counts + [1]) // 64))
            self.sees, self.mask = random_mask(rng, counts, words, empty)
            if pad_rows:
                self.mask = torch.cat([self.mask, torch.zeros(pad_rows, words, dtype=torch.int64, device=DEV)])
        else:
            self.sees, self.mask = [np.tril(np.ones((n, n), dtype=bool)) for n in counts], None

    def ref(self, scale=0.125):
        """(out, lse, tolerance of out, of lse) in 64 bits."""
        outs, lses, tol, ltol = [], [], [], []
        r = 0
        for b, n in enumerate(self.counts):
            c, kv = self.ctx[b], self.kv[b].double()
            k, v = kv[..., :64], kv[..., 64:]
            q = self.q[r:r + n].double().view(n, self.H, self.G, 64)
            r += n
            see = torch.ones(n, c + n, dtype=torch.bool, device=DEV)
            see[:, c:] = torch.from_numpy(self.sees[b]).to(DEV)
            t = torch.einsum("nhgd,phd->nhgp", q, k) * scale
            size = torch.einsum("nhgd,phd->nhgp", q.abs(), k.abs()) * scale
            hide = ~see[:, None, None]
            t = t.masked_fill(hide, -float("inf"))
            lse = torch.logsumexp(t, -1) if c + n else torch.full(t.shape[:-1], -float("inf"), device=DEV).double()
            w = torch.nan_to_num(torch.exp(t - torch.nan_to_num(lse, neginf=0.0)[..., None]), nan=0.0)
            # only what a row sees is added up
            vf, va = torch.nan_to_num(v), torch.nan_to_num(v.abs())
            out = torch.einsum("nhgp,phd->nhgd", w, vf)
            mag = torch.einsum("nhgp,phd->nhgd", w, va)
            outs.append(out.reshape(n, self.H * self.G, 64))
            tol.append((2.0 ** -8 * out.abs() + (2.0 ** -8 + 2.0 ** -12) * mag).reshape(n, self.H * self.G, 64))
            lses.append(lse.reshape(n, self.H * self.G))
            big = size.masked_fill(hide, 0).amax(-1) if c + n else torch.zeros_like(lse)
            ltol.append((64 * 2.0 ** -24 * big + 2.0 ** -20 * (1 + torch.nan_to_num(lse, neginf=0.0).abs())).reshape(n, self.H * self.G))
        return torch.cat(outs), torch.cat(lses), torch.cat(tol) + 2.0 ** -30, torch.cat(ltol)

    def run(self, ws=True, **kw):
        lse = torch.full((self.rows, self.H * self.G), 7.0, device=DEV)
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        work = rc.tree_attention_workspace(self.rows, len(self.counts), self.H * self.G, self.H, DEV) if ws else None
        out = rc.tree_attention(self.q, self.row_start, self.context, self.table, self.cache, tree_mask=self.mask,
                                lse=lse, err=err, workspace=work, **kw)
        torch.cuda.synchronize()
        return out, lse, int(err.item())


def check(case, out, lse, scale=0.125):
    ref, rlse, tol, ltol = case.ref(scale)
    n = ref.shape[0]
    bad = ~((out[:n].double() - ref).abs() <= tol)
    assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()} outside tolerance, first {bad.nonzero()[0].tolist()}"
    got = lse[:n].double()
    same = (got == rlse) | ((got - rlse).abs() <= ltol)
    assert bool(same.all()), f"{int((~same).sum())} log sums outside tolerance"


SHAPES = [
    # counts, contexts, H, G, block
    ([1], [0], 1, 1, 16), ([1], [1], 1, 1, 16), ([1], [500], 8, 8, 16), ([1], [127], 8, 8, 16), ([1], [128], 2, 4, 16),
    ([1, 1, 1], [5, 0, 4096], 8, 8, 16), ([3, 1, 2], [17, 1000, 333], 2, 3, 24), ([13, 12], [1500, 11], 8, 8, 16),
    ([16] * 3, [256, 255, 257], 8, 8, 16), ([64, 63], [700, 2049], 4, 8, 32), ([5], [300], 1, 64, 16),
    ([7], [301], 16, 1, 1), ([9, 9], [100, 90], 2, 5, 7), ([65], [64], 2, 2, 128), ([130, 1], [40, 9], 1, 4, 64),
    ([0, 4, 0], [50, 60, 70], 2, 2, 16), ([200], [0], 2, 1, 16), ([2] * 40, list(range(40)), 1, 8, 16),
    ([64], [30000], 2, 8, 16), ([1], [40000], 1, 16, 48), ([33], [5000], 1, 1, 256), ([16] * 8, [1000] * 8, 16, 4, 16),
]


@pytest.mark.parametrize("counts,ctx,H,G,bs", SHAPES)
@pytest.mark.parametrize("mask", ["tree", "chain"])
def test_against_formula(counts, ctx, H, G, bs, mask):
    case = Case(len(counts) * 1000 + sum(ctx) + H, counts, ctx, H, G, bs, mask=mask)
    out, lse, err = case.run()
    assert err == 0
    check(case, out, lse)


@pytest.mark.parametrize("counts,ctx,H,G,bs", SHAPES[4::4])
def test_without_workspace(counts, ctx, H, G, bs):
    case = Case(5, counts, ctx, H, G, bs)
    out, lse, err = case.run(ws=False)
    assert err == 0
    check(case, out, lse)


@pytest.mark.parametrize("counts,ctx,G", [([6, 9], [0, 0], 2), ([40], [0], 8), ([12, 3], [0, 200], 4), ([64] * 2, [0, 0], 8)])
def test_rows_that_see_nothing(counts, ctx, G):
    case = Case(77, counts, ctx, 2, G, 16, empty=0.4)
    out, lse, err = case.run()
    check(case, out, lse)
    blind = torch.cat([torch.from_numpy(~m.any(1)) & (c == 0) for m, c in zip(case.sees, ctx)]).to(DEV)
    assert bool(blind.any())
    assert bool((out[blind] == 0).all()) and bool((lse[blind] == -float("inf")).all())


@pytest.mark.parametrize("G", [1, 4, 8])
@pytest.mark.parametrize("ctx", [0, 100, 3000])
def test_unseen_infinities_and_nan_do_not_spread(G, ctx):
    counts = [20, 21]
    case = Case(5 + G, counts, [ctx, ctx + 3], 2, G, 16)
    # nodes seen by few rows get K and V that are not finite
    for b, (bad, value) in enumerate(((9, float("nan")), (11, float("inf")))):
        for half in (slice(0, 64), slice(64, 128)):
            p = case.ctx[b] + bad
            blk = int(case.table[b, p // 16])
            case.cache[blk, :, p % 16, half] = value
        case.kv[b][case.ctx[b] + bad] = value
    out, lse, _ = case.run()
    for b, (bad, _) in enumerate(((9, 0), (11, 0))):
        see = torch.from_numpy(case.sees[b][:, bad]).to(DEV)
        assert bool(see.any()) and bool((~see).any())
        rows = slice(sum(counts[:b]), sum(counts[:b + 1]))
        assert bool(torch.isfinite(out[rows][~see].float()).all()) and bool(torch.isfinite(lse[rows][~see]).all())
        assert not bool(torch.isfinite(out[rows][see].float()).any())
        # and the rows that do not see them have the values without them
        case.sees[b][:, bad] = False
        case.kv[b][case.ctx[b] + bad] = 0
    ref, rlse, tol, ltol = case.ref()
    for b, (bad, _) in enumerate(((9, 0), (11, 0))):
        pass
    keep = torch.isfinite(out.float()).all(-1).all(-1)
    assert bool(((out.double() - ref).abs() <= tol)[keep].all())


@pytest.mark.parametrize("G", [1, 8])
def test_infinite_values_that_are_seen(G):
    """V infinite (K finite) in one drafted token: infinite in the rows that see it, finite elsewhere."""
    case = Case(31, [24], [50], 1, G, 16)
    p = 50 + 3
    blk = int(case.table[0, p // 16])
    case.cache[blk, 0, p % 16, 64 + 5] = float("-inf")
    case.kv[0][p, 0, 64 + 5] = 0
    out, lse, _ = case.run()
    see = torch.from_numpy(case.sees[0][:, 3]).to(DEV)
    assert bool((out[see][:, :, 5] == -float("inf")).all())
    ref, _, tol, _ = case.ref()
    tol[see, :, 5] = float("inf")
    got = out.double()
    got[see, :, 5] = 0
    assert bool(((got - ref).abs() <= tol).all())


def test_large_scores_and_scale():
    case = Case(9, [3, 17], [900, 64], 2, 8, 16, sigma=6.0)
    out, lse, _ = case.run(scale=1.0)
    # scores in the thousands: FP32 scores are off by up to 64 * 2^-24 * sum|q k|, which moves the weights
    ref, rlse, tol, ltol = case.ref(1.0)
    assert bool(((lse.double() - rlse).abs() <= ltol).all())
    assert bool(((out.double() - ref).abs() <= tol + 4 * ltol.amax() * 36).all())


@pytest.mark.parametrize("counts,G", [([4, 3], 2), ([30, 20], 8)])
def test_blocks_out_of_range_and_short_tables(counts, G):
    case = Case(3, counts, [200, 150], 2, G, 16)
    case.table[0, 2] = -1
    case.table[1, 4] = case.cache.shape[0]
    keep = [torch.ones(200 + counts[0], dtype=torch.bool, device=DEV), torch.ones(150 + counts[1], dtype=torch.bool, device=DEV)]
    keep[0][32:48] = False
    keep[1][64:80] = False
    full = [kv.clone() for kv in case.kv]
    out, lse, err = case.run()
    assert err == 2
    for b in range(2):
        case.kv[b] = full[b][keep[b]]
        case.ctx[b] -= 16
    check(case, out, lse)
    # a table one block short: the keys past it are not seen
    case = Case(4, counts, [200, 150], 2, G, 16)
    width = case.table.shape[1] - 1
    case.table = case.table[:, :width]
    out, lse, err = case.run()
    cut = [b for b in range(2) if case.ctx[b] + counts[b] > 16 * width]
    assert err == len(cut) >= 1
    for b in cut:
        live = max(0, 16 * width - case.ctx[b])
        case.sees[b][:, live:] = False
        lost = case.ctx[b] - 16 * width
        if lost > 0:
            case.kv[b][16 * width:] = 0
            pytest.skip("context itself cut")
    check(case, out, lse)


def test_strided_output_rows_without_a_sequence_and_slack():
    case = Case(21, [5, 6], [90, 33], 2, 4, 16, pad_rows=3)
    whole = torch.full((case.rows, 8 * 64 + 128), 3.0, dtype=torch.bfloat16, device=DEV)
    out = whole[:, 64:64 + 512].view(case.rows, 8, 64)
    got, lse, _ = case.run(out=out)
    check(case, got, lse)
    assert bool((whole[:, :64] == 3).all()) and bool((whole[:, 576:] == 3).all()) and bool((whole[11:] == 3).all())
    assert bool((lse[11:] == 7).all())


def test_row_starts_outside_are_clamped():
    case = Case(8, [4, 4], [40, 40], 2, 2, 16)
    case.row_start = torch.tensor([-5, 4, 400], dtype=torch.int32, device=DEV)
    out, lse, _ = case.run()
    check(case, out, lse)


@pytest.mark.parametrize("counts,ctx,G", [([1], [30000], 8), ([16, 16], [3000, 9], 8), ([64], [9000], 8)])
def test_same_bits_every_time_on_streams_and_in_graphs(counts, ctx, G):
    case = Case(13, counts, ctx, 4, G, 16)
    ws = rc.tree_attention_workspace(case.rows, len(counts), 4 * G, 4, DEV)
    call = lambda out, **kw: rc.tree_attention(case.q, case.row_start, case.context, case.table, case.cache,
                                               tree_mask=case.mask, out=out, workspace=ws, **kw)
    first = call(None).clone()
    ws.fill_(0xA5)                       # the workspace needs no set-up
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(first)
    call(out, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(out.view(torch.int16), first.view(torch.int16))
    out.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out.view(torch.int16), first.view(torch.int16))
    # other lengths in the same graph
    case.context.copy_(torch.tensor([c // 2 for c in ctx], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    again = call(None)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))
    assert not torch.equal(out.view(torch.int16), first.view(torch.int16))


@pytest.mark.parametrize("n", [1, 20])
def test_offsets_past_32_bits(n):
    """A cache of more than 2^32 bytes and 2^31 elements, its last blocks in use."""
    H, bs, nb = 8, 16, 140000
    case = Case(2, [n], [1000], H, 8, bs)
    small = case.cache.shape[0]
    big = torch.empty((nb, H, bs, 128), dtype=torch.bfloat16, device=DEV)
    big[nb - small:] = case.cache
    case.cache, case.table = big, case.table + (nb - small)
    out, lse, _ = case.run()
    check(case, out, lse)


@pytest.mark.parametrize("counts,ctx,G", [
    ([1] * 40, [700 + 37 * i for i in range(40)], 8),           # two CTAs an SM, few rows
    ([3, 4] * 20, [2100 - 41 * i for i in range(40)], 7),       # one
    ([16, 15] * 6, [3000 - 201 * i for i in range(12)], 8),     # one row tile
    ([64, 0, 63] * 3, [2500, 3, 777, 2048, 10, 1300, 0, 1, 2176], 8),
])
@pytest.mark.parametrize("ws", [True, False])
def test_units_that_end_inside_a_cta(counts, ctx, G, ws):
    """Many units of uneven lengths, so that most CTAs go through ends and beginnings of several."""
    case = Case(31 + G + len(counts), counts, ctx, 8, G, 16)
    out, lse, err = case.run(ws)
    assert err == 0
    check(case, out, lse)


@pytest.mark.parametrize("counts,ctx,H,G", [
    ([12, 11] * 18, [136 + 3 * i for i in range(36)], 8, 4),    # whole units, about one a CTA
    ([25, 24, 0, 25], [90, 1, 50, 0], 1, 64),                   # several row tiles each
    ([8, 7] * 3, [1405, 703, 0, 90, 1000, 1311], 8, 8),         # parts of two tiles
    ([33, 32], [4339, 2100], 2, 16), ([1] * 33 + [50], [600] * 34, 2, 16),
])
def test_parts_of_units(counts, ctx, H, G):
    case = Case(77 + H + G + len(counts), counts, ctx, H, G, 16)
    out, lse, err = case.run()
    assert err == 0
    check(case, out, lse)


def test_empty_tensors_and_masks_without_words():
    case = Case(5, [2], [40], 2, 2, 16)
    none = torch.zeros(2, dtype=torch.int32, device=DEV)
    out = rc.tree_attention(case.q[:0], none, case.context, case.table, case.cache, tree_mask=case.mask[:0])
    assert out.shape == (0, 4, 64)
    with pytest.raises(ValueError, match="word"):
        rc.tree_attention(case.q, case.row_start, case.context, case.table, case.cache, tree_mask=case.mask[:, :0].contiguous())


def test_reads_what_the_store_wrote():
    """Through the store's own slot mapping: keys inserted by rc_kv_store, attended by block table."""
    H, T, bs = 8, 70, 16
    gen = torch.Generator(device=DEV).manual_seed(4)
    kv = torch.randn(1, T, 2 * H * 64, generator=gen, device=DEV).to(torch.bfloat16)
    nb = 8
    table = torch.randperm(nb, generator=gen, device=DEV)[:5].to(torch.int32)[None]
    p = torch.arange(T, device=DEV)
    slots = table[0].long()[p // bs] * bs + p % bs
    cache = torch.full((nb, H, bs, 128), float("nan"), dtype=torch.bfloat16, device=DEV)
    rc.kv_store_from_projection(kv, H, None, [slots], None, [cache], 1e-6)
    q = torch.randn(2, 16, 64, generator=gen, device=DEV).to(torch.bfloat16)
    out = rc.tree_attention(q, torch.tensor([0, 2], dtype=torch.int32, device=DEV),
                            torch.tensor([T - 2], dtype=torch.int32, device=DEV), table, cache)
    rows = cache[slots // bs, :, slots % bs].double()
    k, v = rows[..., :64], rows[..., 64:]
    t = torch.einsum("nhgd,phd->nhgp", q.double().view(2, H, 2, 64), k) / 8
    t[0, :, :, T - 1] = -float("inf")
    w = torch.softmax(t, -1)
    ref = torch.einsum("nhgp,phd->nhgd", w, v).reshape(2, 16, 64)
    mag = torch.einsum("nhgp,phd->nhgd", w, v.abs()).reshape(2, 16, 64)
    assert bool(((out.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -12) * mag + 2.0 ** -30).all())


@pytest.mark.parametrize("group", [1, 3, 8, 16, 64])
def test_workspace_of_the_largest_call_serves_smaller_ones(group):
    size = lambda rows, seqs: rc.lib().rc_tree_attention_workspace_size(rows, seqs, 2 * group, 2)
    rows = [1, 2, 3, 4, 5, 8, 9, 16, 17, 32, 33, 64, 65, 128, 129, 256, 257, 1000]
    for seqs in (1, 2, 7):
        sizes = [size(r, seqs) for r in rows]
        assert sizes == sorted(sizes) and sizes[0] > 0
    for r in rows:
        sizes = [size(r, seqs) for seqs in (400, 64, 9, 3, 2, 1)]
        assert sizes == sorted(sizes)
        assert size(r, 1) <= rc.lib().rc_tree_attention_workspace_size(r, 1, 4 * group, 2)


@pytest.mark.parametrize("small,large", [([2], 4), ([16], 64), ([4, 1], 64)])
def test_small_call_with_a_large_calls_workspace(small, large):
    case = Case(19, small, [3000] * len(small), 2, 8, 16)
    ws = rc.tree_attention_workspace(large, 1, 16, 2, DEV)
    lse = torch.empty(case.rows, 16, device=DEV)
    out = rc.tree_attention(case.q, case.row_start, case.context, case.table, case.cache, tree_mask=case.mask, lse=lse,
                            workspace=ws)
    check(case, out, lse)


def test_workspace_over_another_operand_is_refused():
    case = Case(23, [2, 3], [300, 40], 2, 4, 16)
    ws = rc.tree_attention_workspace(case.rows, 2, 8, 2, DEV)
    ws[64:64 + 12].view(torch.int32).copy_(case.row_start)
    lists = dict(tree_mask=case.mask, workspace=ws)
    with pytest.raises(rc.RopeChainError, match="workspace"):
        rc.tree_attention(case.q, ws[64:64 + 12].view(torch.int32), case.context, case.table, case.cache, **lists)
    with pytest.raises(rc.RopeChainError, match="workspace"):
        rc.tree_attention(case.q, case.row_start, ws[64:64 + 8].view(torch.int32), case.table, case.cache, **lists)
    with pytest.raises(rc.RopeChainError, match="workspace"):
        rc.tree_attention(case.q, case.row_start, case.context, case.table, case.cache, err=ws[:4].view(torch.int32), **lists)


def test_one_row_of_any_stride():
    case = Case(29, [1], [700], 2, 4, 16)
    out, lse, _ = case.run()
    q = torch.empty(3, 517, dtype=torch.bfloat16, device=DEV)[:1, :512].as_strided((1, 8, 64), (517, 64, 1)).copy_(case.q)
    into = torch.empty(3, 517, dtype=torch.bfloat16, device=DEV).as_strided((1, 8, 64), (517, 64, 1))
    case.q = q
    again, _, _ = case.run(out=into)
    assert torch.equal(again, out)


# one batch for each kernel: up to 16 rows a unit, 32, 128, more
KERNELS = [([1, 2], 8), ([4, 3], 8), ([13, 12], 8), ([40, 33], 8)]


@pytest.mark.parametrize("bs", [8, 24, 40, 48, 136])
@pytest.mark.parametrize("counts,G", KERNELS[2:])
@pytest.mark.parametrize("ws", [True, False])
def test_blocks_that_end_inside_a_tile(bs, counts, G, ws):
    """Boxes of 8 and 16 keys, blocks that are no power of two, some of them out of range."""
    case = Case(bs, counts, [1000, 391], 2, G, bs)
    out, lse, err = case.run(ws)
    assert err == 0
    check(case, out, lse)
    gone = [2, 200 // bs]                                       # of the first sequence: that block, of the second: another
    case.table[0, gone[0]] = -7
    case.table[1, gone[1]] = case.cache.shape[0]
    out, lse, err = case.run(ws)
    assert err == 2
    for b, page in enumerate(gone):
        keep = torch.ones(case.kv[b].shape[0], dtype=torch.bool, device=DEV)
        keep[page * bs:(page + 1) * bs] = False
        case.kv[b] = case.kv[b][keep]
        case.ctx[b] -= bs
    check(case, out, lse)


@pytest.mark.parametrize("bs", [16, 24, 1])
@pytest.mark.parametrize("counts,G", KERNELS)
@pytest.mark.parametrize("ws", [True, False])
@pytest.mark.parametrize("width", [0, 7, 300])
def test_table_that_ends_inside_the_context(bs, counts, G, ws, width):
    """Keys past the table's end are not seen, context or drafted, and each such sequence counts once."""
    case = Case(width + bs, counts, [2500, 90], 2, G, bs)
    width = min(width, case.table.shape[1] - 1)
    case.table = case.table[:, :width]
    out, lse, err = case.run(ws)
    lost = 0
    for b in range(2):
        room, ctx, n = width * bs, case.ctx[b], counts[b]
        lost += ctx + n > room
        kept = min(room, ctx + n)
        case.ctx[b] = min(ctx, room)
        case.sees[b][:, max(0, kept - ctx):] = False
        case.kv[b] = torch.cat([case.kv[b][:kept], torch.zeros(case.ctx[b] + n - kept, 2, 128, dtype=torch.bfloat16, device=DEV)])
    assert err == lost >= 1
    check(case, out, lse)


@pytest.mark.parametrize("counts,G", KERNELS)
def test_scores_in_the_thousands(counts, G):
    """As test_large_scores_and_scale, for each kernel, and with keys that raise the maximum by hundreds again and again."""
    case = Case(9, counts, [900, 64], 2, G, 16, sigma=6.0)
    for b in range(2):
        grow = torch.linspace(0.1, 3.0, case.kv[b].shape[0], device=DEV)[:, None, None]
        case.kv[b][..., :64] = (case.kv[b][..., :64].float() * grow).to(torch.bfloat16)
        p = torch.arange(case.kv[b].shape[0], device=DEV)
        case.cache[case.table[b].long()[p // 16], :, p % 16] = case.kv[b]
    out, lse, _ = case.run(scale=1.0)
    ref, rlse, tol, ltol = case.ref(1.0)
    assert bool(((lse.double() - rlse).abs() <= ltol).all())
    assert bool(((out.double() - ref).abs() <= tol + 4 * ltol.amax() * 36).all())


@pytest.mark.parametrize("ws", [True, False])
def test_single_tokens_beside_a_wide_tree(ws):
    """63 single tokens and a tree of 64: the mean says 16 rows a unit, the tree has 512."""
    case = Case(41, [1] * 40 + [64] + [1] * 23, [10 + 53 * i for i in range(64)], 2, 8, 16)
    out, lse, err = case.run(ws)
    assert err == 0
    check(case, out, lse)
