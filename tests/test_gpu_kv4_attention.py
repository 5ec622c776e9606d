"""rc_kv4_attention without a window against the formula in 64 bits on what the cache
stands for (tolerances: paged_cases.py; windows: test_gpu_window_attention.py)."""
import numpy as np
import pytest
import torch

import rope_chain_gb300 as rc
from tests.paged_cases import BF, DEV, I32, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from rope_chain_gb300 import _build
    _build.build()


def case4(*args, **kw):
    return Case(*args, four=True, **kw)


SHAPES = [
    # counts, contexts, H, G, block
    ([1], [0], 1, 1, 16), ([1], [1], 1, 1, 16), ([1], [500], 8, 8, 16), ([1], [127], 8, 8, 16), ([1], [128], 2, 4, 16),
    ([1, 1, 1], [5, 0, 4096], 8, 8, 16), ([3, 1, 2], [17, 1000, 333], 2, 3, 24), ([13, 12], [1500, 11], 8, 8, 16),
    ([16] * 3, [256, 255, 257], 8, 8, 16), ([64, 63], [700, 2049], 4, 8, 32), ([5], [300], 1, 64, 16),
    ([7], [301], 16, 1, 1), ([9, 9], [100, 90], 2, 5, 7), ([65], [64], 2, 2, 128), ([130, 1], [40, 9], 1, 4, 64),
    ([0, 4, 0], [50, 60, 70], 2, 2, 16), ([200], [0], 2, 1, 16), ([2] * 40, list(range(40)), 1, 8, 16),
    ([64], [30000], 2, 8, 16), ([1], [40000], 1, 16, 48), ([33], [5000], 1, 1, 256), ([16] * 8, [1000] * 8, 16, 4, 16),
    ([1] * 40, [700 + 37 * i for i in range(40)], 8, 8, 16), ([3, 4] * 20, [2100 - 41 * i for i in range(40)], 8, 7, 16),
    ([12, 11] * 18, [136 + 3 * i for i in range(36)], 8, 4, 16), ([25, 24, 0, 25], [90, 1, 50, 0], 1, 64, 16),
    ([1] * 40 + [64] + [1] * 23, [10 + 53 * i for i in range(64)], 2, 8, 16),
]


@pytest.mark.parametrize("counts,ctx,H,G,bs", SHAPES)
@pytest.mark.parametrize("mask", ["tree", "chain"])
@pytest.mark.parametrize("ws", [True, False])
def test_against_formula(counts, ctx, H, G, bs, mask, ws):
    case = case4(len(counts) * 1000 + sum(ctx) + H, counts, ctx, H, G, bs, mask=mask)
    out, lse, err = case.run(ws)
    assert err == 0
    case.check(out, lse)


# one batch for each kernel: up to 8 rows a unit, 16, 32, 128, more
KERNELS = [([1, 1], 8), ([1, 2], 8), ([4, 3], 8), ([13, 12], 8), ([40, 33], 8)]


@pytest.mark.parametrize("counts,G", KERNELS)
@pytest.mark.parametrize("ctx", [0, 200])
def test_rows_that_see_nothing(counts, G, ctx):
    case = case4(77, counts, [0, ctx], 2, G, 16, empty=0.4)
    out, lse, err = case.run()
    case.check(out, lse)
    blind = torch.cat([torch.from_numpy(~m.any(1)) & (c == 0) for m, c in zip(case.sees, case.ctx)]).to(DEV)
    assert bool((out[blind] == 0).all()) and bool((lse[blind] == -float("inf")).all())


@pytest.mark.parametrize("counts,G", KERNELS)
@pytest.mark.parametrize("bs", [16, 24, 1])
def test_scales_that_are_not_finite_do_not_spread(counts, G, bs):
    """Nodes that some rows do not see: those rows have their values, and every row those of the other KV head."""
    case = case4(5, counts, [300, 131], 2, G, bs)
    odd = []
    for b in range(2):
        n, p = counts[b], case.ctx[b] + counts[b] - 1
        blk, off = case.key_at(b, p)
        case.scales[blk, 1, off] = torch.tensor([float("nan"), float("inf"), -float("inf"), float("nan")], dtype=BF, device=DEV)
        odd.append(case.visible(b)[:, p])
    odd = torch.cat(odd)
    out, lse, _ = case.run()
    assert bool(odd.any())
    ref, rlse, tol, ltol = case.ref()
    fine = ((out.double() - ref).abs() <= tol).view(len(odd), 2, G, 64)
    assert bool(fine[:, 0].all()) and bool(fine[~odd].all()) and bool(torch.isfinite(lse[~odd]).all())
    assert bool(((lse.double() - rlse).abs() <= ltol)[~odd].all())


@pytest.mark.parametrize("bs", [8, 16, 24, 40, 48, 136])
@pytest.mark.parametrize("counts,G", KERNELS)
@pytest.mark.parametrize("ws", [True, False])
def test_blocks_out_of_range(bs, counts, G, ws):
    case = case4(bs, counts, [1000, 391], 2, G, bs)
    out, lse, err = case.run(ws)
    assert err == 0
    case.check(out, lse)
    case.block_out(0, 2, -7)
    case.block_out(1, 200 // bs, case.nb)
    out, lse, err = case.run(ws)
    assert err == 2
    case.check(out, lse)


@pytest.mark.parametrize("bs", [16, 24, 1])
@pytest.mark.parametrize("counts,G", KERNELS)
@pytest.mark.parametrize("ws", [True, False])
@pytest.mark.parametrize("width", [0, 7, 300])
def test_table_that_ends_inside_the_context(bs, counts, G, ws, width):
    case = case4(width + bs, counts, [2500, 90], 2, G, bs)
    width = min(width, case.table.shape[1] - 1)
    case.table = case.table[:, :width]
    out, lse, err = case.run(ws)
    lost = 0
    for b in range(2):
        lost += case.ctx[b] + counts[b] > width * bs
        case.gone[b][width * bs:] = True
    assert err == lost >= 1
    case.check(out, lse)


@pytest.mark.parametrize("counts,G", KERNELS)
def test_scores_in_the_thousands(counts, G):
    """Keys that raise the maximum by hundreds again and again.  Scores are off by up to 64 * 2^-24 * sum|q k|, which
    moves the weights by as much of themselves: of values up to 36."""
    case = case4(9, counts, [900, 64], 2, G, 16, sigma=6.0)
    for b in range(2):
        n = case.kv[b].shape[0]
        grow = torch.linspace(0.1, 3.0, n, device=DEV)[:, None, None]
        kv = case.kv[b].clone()
        kv[..., :64] = (kv[..., :64].float() * grow).to(BF)
        p = torch.arange(n, device=DEV)
        slots = case.table[b].long()[p // 16] * 16 + p % 16
        rc.kv4_store(kv[..., :64], kv[..., 64:], slots, case.cache, case.scales)
        case.kv[b] = rc.kv4_load(slots, case.cache, case.scales)
    out, lse, _ = case.run(scale=1.0)
    ref, rlse, tol, ltol = case.ref(1.0)
    assert bool(((lse.double() - rlse).abs() <= ltol).all())
    assert bool(((out.double() - ref).abs() <= tol + 4 * ltol.amax() * 36).all())


@pytest.mark.parametrize("value", [2.0 ** 60, 2.0 ** -60])
def test_scales_far_from_one(value):
    """K tiny and Q as large the other way round, V of the same size: powers of two change nothing."""
    case = case4(11, [3, 4], [200, 33], 2, 8, 16)
    plain, lse, _ = case.run()
    case.scales[..., :2] *= value
    case.scales[..., 2:] /= value
    case.q = (case.q.float() / value).to(BF)
    out, lse2, _ = case.run()
    assert torch.equal((out.double() * value).to(BF), plain) and torch.equal(lse, lse2)


def test_same_bits_every_time_on_streams_and_in_graphs():
    for counts, ctx, G in (([1], [30000], 8), ([16, 16], [3000, 9], 8), ([64], [9000], 8)):
        case = case4(13, counts, ctx, 4, G, 16)
        ws = case.workspace()
        first = case.call(workspace=ws).clone()
        ws.fill_(0xA5)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        out = torch.empty_like(first)
        case.call(out=out, workspace=ws, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), first.view(torch.int16))
        out.zero_()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            case.call(out=out, workspace=ws)
        case.context.copy_(torch.tensor([c // 2 for c in ctx], dtype=I32))
        graph.replay()
        torch.cuda.synchronize()
        again = case.call(workspace=ws)
        assert torch.equal(out.view(torch.int16), again.view(torch.int16))
        assert not torch.equal(out.view(torch.int16), first.view(torch.int16))


def test_offsets_past_32_bits():
    """A cache of more than 2^32 bytes, its last blocks in use."""
    for n in (1, 20):
        H, bs, nb = 8, 16, 600000
        case = case4(2, [n], [1000], H, 8, bs)
        small = case.cache.shape[0]
        big, scales = rc.new_kv4_cache(nb, H, bs, DEV)
        big[nb - small:], scales[nb - small:] = case.cache, case.scales
        case.cache, case.scales, case.table = big, scales, case.table + (nb - small)
        out, lse, _ = case.run()
        case.check(out, lse)


def test_strides_slack_and_no_rows():
    case = case4(21, [5, 6], [90, 33], 2, 4, 16, pad_rows=3)
    whole = torch.full((case.rows, 8 * 64 + 128), 3.0, dtype=BF, device=DEV)
    got, lse, _ = case.run(out=whole[:, 64:64 + 512].view(case.rows, 8, 64))
    case.check(got, lse)
    assert bool((whole[:, :64] == 3).all()) and bool((whole[:, 576:] == 3).all()) and bool((whole[11:] == 3).all())
    assert bool((lse[11:] == 7).all())
    case.row_start = torch.tensor([-5, 5, 400], dtype=I32, device=DEV)     # clamped to the rows
    case.counts, case.sees = [5, 9], [case.sees[0], np.zeros((9, 9), dtype=bool)]
    assert case.run()[2] == 0
    none = torch.zeros(3, dtype=I32, device=DEV)
    out = rc.kv4_attention(case.q[:0], none, case.context, case.table, case.cache, case.scales)
    assert out.shape == (0, 8, 64)


@pytest.mark.parametrize("group", [1, 3, 8, 16, 64])
def test_workspace_of_the_largest_call_serves_smaller_ones(group):
    size = lambda rows, seqs: rc.lib().rc_kv4_attention_workspace_size(rows, seqs, 2 * group, 2)  # noqa: E731
    rows = [1, 2, 3, 4, 5, 8, 9, 16, 17, 32, 33, 64, 65, 128, 129, 256, 257, 1000]
    for seqs in (1, 2, 7):
        sizes = [size(r, seqs) for r in rows]
        assert sizes == sorted(sizes) and sizes[0] > 0
    for r in rows:
        sizes = [size(r, seqs) for seqs in (400, 64, 9, 3, 2, 1)]
        assert sizes == sorted(sizes)
        assert size(r, 1) <= rc.lib().rc_kv4_attention_workspace_size(r, 1, 4 * group, 2)


@pytest.mark.parametrize("small,large", [([1], 64), ([2], 4), ([16], 64), ([4, 1], 64)])
def test_small_call_with_a_large_calls_workspace(small, large):
    case = case4(19, small, [3000] * len(small), 2, 8, 16)
    ws = rc.kv4_attention_workspace(large, 1, 16, 2, DEV)
    lse = torch.empty(case.rows, 16, device=DEV)
    case.check(case.call(lse=lse, workspace=ws), lse)


def test_output_on_a_side_stream():
    case = case4(3, [16] * 64, [100] * 64, 2, 8, 16)
    want = case.call().clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    block = torch.empty_like(want)
    torch.cuda._sleep(40_000_000)
    block.fill_(7.0)
    del block
    got = case.call(stream=side)
    side.synchronize()
    early = got.cpu()
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(early, want.cpu())
