"""rc_kv4_attention of single tokens under windows of all lengths over long contexts, whose
rows come through shared memory or straight into registers by what the window leaves
(tolerances: paged_cases.py)."""
import pytest
import torch

from tests.paged_cases import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from rope_chain_gb300 import _build
    _build.build()


@pytest.mark.parametrize("counts,ctx", [([1], [9000]), ([1] * 6, [9000, 4096, 2500, 700, 90, 0]), ([1, 0, 1], [5000, 60, 3001])])
@pytest.mark.parametrize("window,sinks", [(100, 0), (512, 4), (1700, 4), (1900, 200), (2048, 0), (2500, 130), (6000, 64), (7, 2500)])
@pytest.mark.parametrize("bs", [16, 24, 8])
@pytest.mark.parametrize("ws", [True, False])
def test_against_formula(counts, ctx, window, sinks, bs, ws):
    case = Case(sum(ctx) + window, counts, ctx, 2, 8, bs, four=True, window=window, sinks=sinks)
    out, lse, err = case.run(ws)
    assert err == 0
    case.check(out, lse)


@pytest.mark.parametrize("window,sinks", [(300, 20), (2600, 20)])
@pytest.mark.parametrize("bs", [16, 24])
def test_blocks_given_away_and_blocks_lost(window, sinks, bs):
    """What neither the first keys nor the window need may be anything; what they need and is
    out of range is counted, once."""
    ctx = [8000, 5003]
    case = Case(bs, [1, 1], ctx, 2, 8, bs, four=True, window=window, sinks=sinks)
    for b in range(2):
        for page in range(-(-sinks // bs), (ctx[b] + 1 - window) // bs):
            case.table[b, page] = -7
    out, lse, err = case.run()
    assert err == 0
    case.check(out, lse)
    case.block_out(0, ctx[0] // bs - 3, case.nb)             # in the window
    case.block_out(1, 0, -1)                                 # the first keys'
    out, lse, err = case.run()
    assert err == 2
    case.check(out, lse)
