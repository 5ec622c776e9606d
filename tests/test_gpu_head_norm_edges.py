"""rc_head_norm_rope and its gradients where much work goes through the kernels that
copy heads ahead, and where single elements are infinite or NaN.

Tolerance of a weight's gradient, a sum of N = tokens * heads products of n and g, with
u = 2^-24: a product is off by (d / 2 + 16) u of |g n| (r, n and the turn of dy, as in
test_gpu_head_norm), and what matters of the sum is how many additions lie one behind
another.  At least 8 threads of every SM have each of its columns, so a thread adds some
N / (8 SMs) of them, and up to an item (8 heads) more; then 5 + 8 within a block, 2 SMs
/ 32 + 32 over the blocks: (N / (8 SMs) + d / 2 + 96) u of sum |g n| in all.  So a head that
is left out of the sum shows, which each test asserts of its own sizes."""
import pytest
import torch

import rope_chain_gb300 as rc
from tests.test_gpu_head_norm import BF, DEV, F32, HALVES, PAIRS, U, Case, turn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from rope_chain_gb300 import _build
    _build.build()


def check_weight_gradients(c, dq, dk):
    """Returns, for each weight, the tolerances and the terms' sizes per column."""
    x, dy = c.x.double(), c.dy.double()
    n = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + c.eps)
    g = turn(dy, c.table, c.pos, c.layout, back=True)
    size = turn(dy.abs(), c.table, c.pos, c.layout, sizes=True)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    found = []
    for got, weight, part in ((dq, c.qw, slice(0, c.q_heads)), (dk, c.kw, slice(c.q_heads, c.heads))):
        if weight is None:
            assert got is None
            continue
        ref = (g * n)[:, part].sum((0, 1))
        deep = c.T * (part.stop - part.start) / (8 * sms) + c.d / 2 + 96
        tol = deep * U * (size * n.abs())[:, part].sum((0, 1)) + 2.0 ** -133
        err = (got.double() - ref).abs()
        assert got.dtype == F32 and bool((err <= tol).all()), float((err - tol).max())
        found.append((tol, ref, (g * n)[:, part]))
    return found


BUSY = [(3000, 40, 128, BF), (9000, 16, 64, BF), (2500, 33, 96, BF), (1500, 20, 256, F32), (900, 24, 512, BF), (2000, 17, 128, F32),
        (4000, 12, 64, F32)]


@pytest.mark.parametrize("T,heads,d,dtype", BUSY)
@pytest.mark.parametrize("layout", [PAIRS, HALVES])
@pytest.mark.parametrize("rot", [64, 0])
def test_weight_gradients_of_much_work(T, heads, d, dtype, layout, rot):
    c = Case(T, heads, d, rot or d, dtype, layout, weight=dtype, q_heads=heads - 7)
    _, dq, dk = c.grad()
    for tol, ref, terms in check_weight_gradients(c, dq, dk):
        # an eighth of the tokens (a warp's), or a 304th of them (a block's), would show in
        # every other column at least
        for lost in (terms[::8], terms[::304]):
            assert float((lost.sum((0, 1)).abs() > 2 * tol).float().mean()) > 0.5


@pytest.mark.parametrize("T,heads,d,dtype", BUSY[:4])
@pytest.mark.parametrize("layout", [PAIRS, HALVES])
@pytest.mark.parametrize("where", ["last token", "last heads", "first heads", "one head of a token", "every 304th token"])
def test_every_head_enters_the_weight_gradients(T, heads, d, dtype, layout, where):
    """A gradient that is zero but for a few heads, at the ends of items, tokens, kinds and
    the whole: what is left out changes the sums altogether."""
    c = Case(T, heads, d, d, dtype, layout, weight=dtype, q_heads=heads - 7)
    keep = torch.zeros(T, heads, 1, dtype=dtype, device=DEV)
    if where == "last token":
        keep[-1] = 1
    elif where == "last heads":
        keep[:, [c.q_heads - 1, heads - 1]] = 1
    elif where == "first heads":
        keep[:, [0, c.q_heads]] = 1
    elif where == "one head of a token":
        keep[T // 2, [c.q_heads // 2, c.q_heads + 3]] = 1
    else:
        keep[::304] = 1
    c.dy.mul_(keep)
    dx, dq, dk = c.grad()
    c.check_grad(dx, dq, dk)
    for tol, ref, _ in check_weight_gradients(c, dq, dk):
        assert float((ref.abs() > 4 * tol).float().mean()) > 0.9


@pytest.mark.parametrize("T,heads,d,dtype", [(3000, 40, 128, BF), (9000, 16, 64, BF), (1500, 20, 256, F32), (2000, 18, 128, F32)])
@pytest.mark.parametrize("layout", [PAIRS, HALVES])
@pytest.mark.parametrize("kw", [dict(extra=1024), dict(extra=64, order="heads"), dict()])
def test_much_work_in_place_and_strided(T, heads, d, dtype, layout, kw):
    """Columns of a projection's wider rows, or heads before tokens; the same bits as into
    an output of its own, and nothing beside the columns is touched."""
    def made():
        return Case(T, heads, d, d if d < 256 else 64, dtype, layout, weight=dtype, q_heads=heads - 5, **kw)

    def whole(t):                                        # the memory that a view lies in
        return t.as_strided((t.untyped_storage().nbytes() // t.element_size(),), (1,), 0)

    def beside(t):                                       # what of it is not the view's
        outside = torch.ones_like(whole(t), dtype=torch.bool)
        outside.as_strided(t.shape, t.stride(), t.storage_offset()).fill_(False)
        return whole(t)[outside]
    c = made()
    want = c.run()
    dx, dq, dk = c.grad()
    c.check_forward(want)
    c.check_grad(dx, dq, dk)
    check_weight_gradients(c, dq, dk)
    dense = Case(T, heads, d, c.rot, dtype, layout, weight=dtype, q_heads=heads - 5)
    dense.x, dense.dy, dense.pos = c.x.contiguous(), c.dy.contiguous(), c.pos
    dense.how = c.how
    assert torch.equal(dense.run(), want) and all(torch.equal(a, b) for a, b in zip(dense.grad(), (dx, dq, dk)))
    for over in ("dy", "x"):
        other = made()
        out = getattr(other, over)
        rest = beside(out).clone()
        got = other.grad(out=out)
        assert torch.equal(out, dx) and torch.equal(got[1], dq) and torch.equal(got[2], dk)
        assert torch.equal(beside(out), rest)
    other = made()
    rest = beside(other.x).clone()
    assert torch.equal(other.run(out=other.x), want) and torch.equal(other.x, want)
    assert torch.equal(beside(other.x), rest)


UNFINITE = [float("inf"), float("-inf"), float("nan")]


@pytest.mark.parametrize("T,heads,d,rot,dtype", [(5, 6, 64, 32, BF), (5, 6, 64, 32, F32), (6, 5, 66, 10, BF), (4, 4, 96, 32, F32), (3, 4, 512, 64, F32),
                                                 (3000, 40, 128, 64, BF), (2000, 18, 128, 32, F32)])
@pytest.mark.parametrize("layout", [PAIRS, HALVES])
@pytest.mark.parametrize("at", ["first", "middle", "last"])
def test_what_does_not_turn_keeps_infinities_to_itself(T, heads, d, rot, dtype, layout, at):
    """An element past rot_dim meets no other but in its head's means: an infinite weight or
    gradient of one column is seen in that column alone, of y and of the sums."""
    c = Case(T, heads, d, rot, dtype, layout, weight=dtype, q_heads=heads - 3)
    e = dict(first=rot, middle=(rot + d) // 2, last=d - 1)[at]
    others = torch.arange(d, device=DEV) != e
    y, (dx, dq, dk) = c.run(), c.grad()
    for odd in UNFINITE:
        for weight, part in ((c.qw, slice(0, c.q_heads)), (c.kw, slice(c.q_heads, heads))):
            held = weight[e].clone()
            weight[e] = odd
            z = c.run()
            weight[e] = held
            assert not bool(torch.isfinite(z[:, part, e]).any())
            assert torch.equal(z[..., others], y[..., others])
        held = c.dy[T // 2, 0, e].clone()
        c.dy[T // 2, 0, e] = odd
        dx2, dq2, dk2 = c.grad()
        c.dy[T // 2, 0, e] = held
        assert torch.equal(dq2[others], dq[others]) and not bool(torch.isfinite(dq2[e])) and torch.equal(dk2, dk)
        rows = torch.ones(T, heads, dtype=torch.bool, device=DEV)
        rows[T // 2, 0] = False
        assert torch.equal(dx2[rows], dx[rows])


@pytest.mark.parametrize("T,heads,d,dtype", [(5, 6, 64, BF), (5, 6, 64, F32), (6, 5, 66, BF), (3000, 40, 128, BF), (2000, 18, 128, F32)])
@pytest.mark.parametrize("layout", [PAIRS, HALVES])
def test_tokens_outside_the_table_keep_infinities_in_their_columns(T, heads, d, dtype, layout):
    """Such a token is normed but not turned: no element of it meets another."""
    c = Case(T, heads, d, d, dtype, layout, weight=dtype, q_heads=heads - 3)
    t = T // 2
    c.pos[t] = -1
    y, (_, dq, dk) = c.run()[t].clone(), c.grad()
    for e in (0, 1, d // 2, d - 1):
        others = torch.arange(d, device=DEV) != e
        for odd in UNFINITE:
            held = c.qw[e].clone()
            c.qw[e] = odd
            z = c.run()[t]
            c.qw[e] = held
            assert not bool(torch.isfinite(z[: c.q_heads, e]).any())
            assert torch.equal(z[:, others], y[:, others])
            held = c.dy[t, 1, e].clone()
            c.dy[t, 1, e] = odd
            _, dq2, dk2 = c.grad()
            c.dy[t, 1, e] = held
            assert torch.equal(dq2[others], dq[others]) and not bool(torch.isfinite(dq2[e])) and torch.equal(dk2, dk)
    # an infinite element of x makes its head's others zeros (x r w with r = 0), not NaN
    c.x[t, 1, 3] = float("inf")
    z = c.run()[t, 1]
    others = torch.arange(d, device=DEV) != 3
    assert bool((z[others] == 0).all()) and bool(torch.isnan(z[3]))
