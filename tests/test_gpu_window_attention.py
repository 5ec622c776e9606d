"""rc_window_attention, and rc_kv4_attention with a window, against the formula in 64
bits (tolerances: paged_cases.py): windows and first keys of any size, trees, chains
and single tokens, tiles that the window leaves out, blocks that were given away."""
import numpy as np
import pytest
import torch

import rope_chain_gb300 as rc
from tests.paged_cases import BF, DEV, I32, Case

pytestmark = pytest.mark.gpu
FORMATS = [pytest.param(False, id="bf16"), pytest.param(True, id="four")]


@pytest.fixture(scope="module", autouse=True)
def built():
    from rope_chain_gb300 import _build
    _build.build()
    rc.read_device_faults(clear=True)
    yield
    assert rc.read_device_faults(clear=True) == 0


# counts, contexts, H, G, block
SHAPES = [
    ([1], [0], 1, 1, 16), ([1], [1], 1, 1, 16), ([1], [500], 8, 8, 16), ([1, 1, 1], [5, 0, 4096], 8, 8, 16),
    ([3, 1, 2], [17, 1000, 333], 2, 3, 24), ([13, 12], [1500, 11], 8, 8, 16), ([64, 63], [700, 2049], 4, 8, 32),
    ([5], [300], 1, 64, 16), ([7], [301], 16, 1, 1), ([9, 9], [100, 90], 2, 5, 7), ([130, 1], [40, 9], 1, 4, 64), ([0, 4, 0], [50, 60, 70], 2, 2, 16),
    ([200], [0], 2, 1, 16), ([2] * 40, [37 * i for i in range(40)], 1, 8, 16), ([1], [40000], 1, 16, 48), ([33], [5000], 1, 1, 256),
    ([16] * 8, [1000] * 8, 16, 4, 16), ([8] * 3, [900, 901, 130], 2, 8, 128),
]
WINDOWS = [(1, 0), (1, 4), (2, 1), (16, 0), (100, 16), (128, 128), (513, 200), (1000, 3), (2 ** 31 - 1, 0), (5, 2 ** 31 - 1)]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(str(x) for x in (sum(s[0]), max(s[1])) + s[2:]))
@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("four", FORMATS)
def test_against_formula(shape, window, sinks, four):
    counts, ctx, H, G, bs = shape
    for mask in ("tree", "chain"):
        case = Case(len(counts) * 1000 + sum(ctx) + H, counts, ctx, H, G, bs, four=four, window=window, sinks=sinks, mask=mask)
        out, lse, err = case.run()
        assert err == 0
        case.check(out, lse)


# one batch for each kernel: up to 8 rows a unit, 16, 32, 128, more
KERNELS = [([1, 1], 8), ([1, 2], 8), ([4, 3], 8), ([13, 12], 8), ([40, 33], 8)]


@pytest.mark.parametrize("counts,G", KERNELS)
@pytest.mark.parametrize("window,sinks", [(3, 2), (300, 20), (1100, 140)])
@pytest.mark.parametrize("four", FORMATS)
@pytest.mark.parametrize("ws", [True, False])
def test_rows_that_see_nothing_or_little(counts, G, window, sinks, four, ws):
    """Rows whose mask leaves no node still have the window's context keys; without a context they give zeros."""
    case = Case(77, counts, [0, 1300], 2, G, 16, four=four, window=window, sinks=sinks, empty=0.5)
    out, lse, err = case.run(ws)
    assert err == 0
    case.check(out, lse)
    blind = torch.cat([torch.from_numpy(~m.any(1)) & (c == 0) for m, c in zip(case.sees, case.ctx)]).to(DEV)
    assert bool((out[blind] == 0).all()) and bool((lse[blind] == -float("inf")).all())


@pytest.mark.parametrize("counts,G", KERNELS)
@pytest.mark.parametrize("window,sinks,bs", [(50, 5, 16), (200, 0, 8), (129, 40, 24), (64, 17, 136), (30, 130, 1)])
@pytest.mark.parametrize("four", FORMATS)
def test_blocks_without_a_key_that_counts_are_not_looked_at(counts, G, window, sinks, bs, four):
    """Their entries may be anything, and are not counted; those that are needed are, once."""
    case = Case(bs, counts, [1000, 391], 2, G, bs, four=four, window=window, sinks=sinks)
    for b in range(2):
        for page in range(case.table.shape[1]):
            first, last = page * bs, page * bs + bs - 1
            if first >= sinks and last < case.ctx[b] + 1 - window:
                case.table[b, page] = (-1, 2 ** 31 - 1, case.nb)[page % 3]
    out, lse, err = case.run()
    assert err == 0
    case.check(out, lse)
    lost = 0
    if sinks:
        case.block_out(0, 0, -7)
        lost += 1
    case.block_out(1, (391 - window // 2) // bs, case.nb)
    out, lse, err = case.run()
    assert err == lost + 1
    case.check(out, lse)


@pytest.mark.parametrize("counts,G", KERNELS)
@pytest.mark.parametrize("bs", [16, 24, 1])
@pytest.mark.parametrize("four", FORMATS)
@pytest.mark.parametrize("width", [0, 7, 120])
def test_table_that_ends_inside_the_context(counts, G, bs, four, width):
    """Keys past the table's end are not seen, nor in the order: the window ends with the last that is."""
    case = Case(width + bs, counts, [2500, 90], 2, G, bs, four=four, window=70, sinks=9)
    width = min(width, case.table.shape[1] - 1)
    case.table = case.table[:, :width]
    out, lse, err = case.run()
    lost = 0
    for b in range(2):
        room, ctx, n = width * bs, case.ctx[b], counts[b]
        lost += ctx + n > room
        kept = min(room, ctx + n)
        case.ctx[b] = min(ctx, room)
        case.sees[b][:, max(0, kept - ctx):] = False
        case.kv[b] = torch.cat([case.kv[b][:kept], torch.zeros(case.ctx[b] + n - kept, 2, 128, dtype=BF, device=DEV)])
        case.gone[b] = np.zeros(case.ctx[b] + n, dtype=bool)
    assert err == lost >= 1
    case.check(out, lse)


@pytest.mark.parametrize("counts,G", KERNELS)
@pytest.mark.parametrize("window,sinks", [(20, 3), (3, 0), (300, 130)])
def test_what_is_not_seen_does_not_spread(counts, G, window, sinks):
    """Infinities and NaN in keys before, at and inside the window's begin, among the first keys, and in nodes."""
    case = Case(5 + G, counts, [700, 431], 2, G, 16, window=window, sinks=sinks)
    seen = [case.visible(b) for b in range(2)]
    clean = case.run()
    odd = [torch.zeros(n, dtype=torch.bool, device=DEV) for n in counts]
    for b in range(2):
        ctx, n = case.ctx[b], counts[b]
        places = [sinks, sinks + 1, ctx - window - 1, ctx - window, ctx + 1 - window, ctx + n - window - 1, ctx + n - window,
                  ctx + n // 2, ctx + n - 1, ctx - 130 - window]
        for i, p in enumerate(places):
            if not sinks <= p < ctx + n or bool(seen[b][:, p].all()):
                continue
            blk, off = case.key_at(b, p)
            value = (float("nan"), float("inf"), float("-inf"))[i % 3]
            half = slice(64 * (i % 2), 64 * (i % 2) + 64)
            case.cache[blk, :, off, half] = value
            odd[b] |= seen[b][:, p]
    odd = torch.cat(odd)
    for ws in (True, False):
        out, lse, _ = case.run(ws)
        assert bool(torch.isfinite(out[~odd].float()).all()) and bool(torch.isfinite(lse[~odd]).all())
        ref, rlse, tol, ltol = case.ref()
        assert bool(((out.double() - ref).abs() <= tol)[~odd].all()) and bool(((lse.double() - rlse).abs() <= ltol)[~odd].all())
    assert torch.equal(case.run()[0][~odd], clean[0][~odd])


@pytest.mark.parametrize("counts,G", KERNELS)
def test_infinite_values_that_are_seen(counts, G):
    """V infinite (K finite) at the window's begin, seen by some rows: infinite there, finite elsewhere."""
    case = Case(31, counts, [600, 500], 1, G, 16, window=40)
    p = 600 + 1 - 40 + 1
    see = case.visible(0)[:, p]
    blk, off = case.key_at(0, p)
    case.cache[blk, 0, off, 64 + 5] = float("-inf")
    case.kv[0][p, 0, 64 + 5] = 0
    for ws in (True, False):
        out, lse, _ = case.run(ws)
        n = counts[0]
        assert bool((out[:n][see][:, :, 5] == -float("inf")).all()) and bool(torch.isfinite(out[:n][~see].float()).all())
        ref, _, tol, _ = case.ref()
        got = out.double()
        got[:n][see, :, 5], tol[:n][see, :, 5] = 0, float("inf")
        assert bool(((got - ref).abs() <= tol).all())


@pytest.mark.parametrize("counts,G", KERNELS)
@pytest.mark.parametrize("four", FORMATS)
def test_a_window_past_everything_is_none(counts, G, four):
    case = Case(3, counts, [900, 64], 2, G, 16, four=four, window=5000)
    out, lse, _ = case.run()
    case.window = None
    plain, plain_lse, _ = case.run()
    case.check(out, lse)
    case.check(plain, plain_lse)


@pytest.mark.parametrize("counts,ctx,G", [([1], [30000], 8), ([16, 16], [3000, 9], 8), ([64], [9000], 8)])
@pytest.mark.parametrize("four", FORMATS)
def test_same_bits_every_time_on_streams_and_in_graphs(counts, ctx, G, four):
    case = Case(13, counts, ctx, 4, G, 16, four=four, window=700, sinks=4)
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
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out.view(torch.int16), first.view(torch.int16))
    # other lengths in the same graph
    case.context.copy_(torch.tensor([c // 2 for c in ctx], dtype=I32))
    graph.replay()
    torch.cuda.synchronize()
    again = case.call(workspace=ws)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))
    assert not torch.equal(out.view(torch.int16), first.view(torch.int16))


@pytest.mark.parametrize("four", FORMATS)
@pytest.mark.parametrize("ws", [True, False])
@pytest.mark.parametrize("counts,ctx,G", [
    ([1] * 40, [700 + 37 * i for i in range(40)], 8), ([3, 4] * 20, [2100 - 41 * i for i in range(40)], 7),
    ([16, 15] * 6, [3000 - 201 * i for i in range(12)], 8), ([64, 0, 63] * 3, [2500, 3, 777, 2048, 10, 1300, 0, 1, 2176], 8),
    ([1] * 20 + [64] + [1] * 10, [10 + 93 * i for i in range(31)], 8)])
def test_many_units(counts, ctx, G, ws, four):
    case = Case(31 + G + len(counts), counts, ctx, 8, G, 16, four=four, window=600, sinks=30)
    out, lse, err = case.run(ws)
    assert err == 0
    case.check(out, lse)


@pytest.mark.parametrize("four", FORMATS)
@pytest.mark.parametrize("counts,ctx,H", [
    ([13] * 20, [2000] * 20, 8), ([13, 5] * 10, [2000 - 31 * i for i in range(20)], 8), ([40] * 10, [1700] * 10, 8),
    ([13] * 40, [1500 + i for i in range(40)], 4), ([40, 0, 33] * 12, [1500 - 41 * i for i in range(36)], 4),
    ([13] * 20 + [0] * 14, [2000] * 34, 8), ([13] * 24, [9000] + [700] * 23, 8)])
def test_units_that_come_out_even(counts, ctx, H, four):
    """More units of several tiles than a cut would be worth: the same with a workspace as without one."""
    for window, sinks in ((700, 3), (1000, 130)):
        case = Case(len(counts) + H, counts, ctx, H, 8, 16, four=four, window=window, sinks=sinks)
        case.block_out(1, (ctx[1] - 5) // 16, -1)
        for ws in (True, False):
            out, lse, err = case.run(ws)
            assert err == (counts[1] > 0)
            case.check(out, lse)


@pytest.mark.parametrize("four", FORMATS)
def test_strided_output_and_rows_without_a_sequence(four):
    case = Case(21, [5, 6], [290, 33], 2, 4, 16, four=four, window=20, sinks=2, pad_rows=3)
    whole = torch.full((case.rows, 8 * 64 + 128), 3.0, dtype=BF, device=DEV)
    out = whole[:, 64:64 + 512].view(case.rows, 8, 64)
    got, lse, _ = case.run(out=out)
    case.check(got, lse)
    assert bool((whole[:, :64] == 3).all()) and bool((whole[:, 576:] == 3).all()) and bool((whole[11:] == 3).all())
    assert bool((lse[11:] == 7).all())
