"""rc_head_norm_rope and its gradients against the formulas in 64 bits.

Tolerances, with u = 2^-24 and d = head_dim.  r: a sum of d squares (d u), its
mean and eps (2 u), all halved by the root, and the reciprocal root (2 ulp, 4 u):
(d / 2 + 5) u.  y: x r w and the rotation, five roundings more, of |a c| + |b s|:
(d / 2 + 10) u, then the type's own rounding.  dx = r (g w - n m), m = mean(g w n):
r twice and g's rotation in m, whose sum is off by d u of mean(|g w n|):
(2 d + 32) u of r (|g w| + |n| mean(|g w n|)).  dw: N products of n and g in some
order, at most (N + d + 32) u of sum |g n|."""
import pytest
import torch

import rope_chain_gb300 as rc

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, F32, F64, I32 = torch.bfloat16, torch.float32, torch.float64, torch.int32
U = 2.0 ** -24
ROUND = {BF: 2.0 ** -8, F32: U}
PAIRS, HALVES = rc.RC_ROPE_PAIRS, rc.RC_ROPE_HALVES


@pytest.fixture(scope="module", autouse=True)
def built():
    from rope_chain_gb300 import _build
    _build.build()


def turn(x, table, pos, layout, back=False, sizes=False):
    """x [T, heads, d] turned in 64 bits; sizes: |a c| + |b s| in place of the sums."""
    rot = table.shape[1]
    half = rot // 2
    inside = (pos >= 0) & (pos < table.shape[0])
    row = table.double()[pos.clamp(0, table.shape[0] - 1)][:, None]
    one = torch.cat([torch.ones(half), torch.zeros(half)]).double().to(x.device)
    row = torch.where(inside[:, None, None], row, one)
    c, s = row[..., :half], row[..., half:]
    y = x.clone()
    a, b = (slice(0, half), slice(half, rot)) if layout == HALVES else (slice(0, rot, 2), slice(1, rot, 2))
    u, v = x[..., a], x[..., b]
    if sizes:
        y[..., a], y[..., b] = u * c.abs() + v * s.abs(), v * c.abs() + u * s.abs()
    else:
        s = -s if back else s
        y[..., a], y[..., b] = u * c - v * s, v * c + u * s
    return y


def weights64(heads, d, q_heads, qw, kw):
    w = torch.ones(heads, d, dtype=F64, device=DEV)
    if qw is not None:
        w[:q_heads] = qw.double()
    if kw is not None:
        w[q_heads:] = kw.double()
    return w


def forward64(x, w, table, pos, layout, eps):
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + eps)
    return turn(x * r * w, table, pos, layout), r


class Case:
    def __init__(self, T, heads, d, rot, dtype, layout, *, table=None, weight=None, q_heads=None, extra=0, order="tokens",
                 offset=0, seed=0, eps=1e-6):
        gen = torch.Generator(device=DEV).manual_seed(seed + T + d)
        rand = lambda *shape: torch.randn(*shape, generator=gen, device=DEV)  # noqa: E731
        self.T, self.heads, self.d, self.rot, self.layout, self.eps = T, heads, d, rot, layout, eps
        self.q_heads = heads if q_heads is None else q_heads

        def view():
            if order == "tokens":
                flat = rand(T * (heads * d + extra) + offset).to(dtype)[offset:]
                return flat.view(T, heads * d + extra)[:, :heads * d].view(T, heads, d)
            flat = rand(heads * (T * d + extra) + offset).to(dtype)[offset:]
            return flat.view(heads, T * d + extra)[:, :T * d].view(heads, T, d).transpose(0, 1)
        self.x, self.dy = view(), view()
        self.table = rc.rope_table(512, rot, dtype=table or dtype, device=DEV)
        self.pos = torch.randint(0, 512, (T,), generator=gen, device=DEV)
        self.qw = self.kw = None
        if weight is not None:
            self.qw = (1 + 0.3 * rand(d)).to(weight) if self.q_heads else None
            self.kw = (1 + 0.3 * rand(d)).to(weight) if self.q_heads < heads else None
        self.how = dict(eps=eps, q_weight=self.qw, k_weight=self.kw, q_heads=self.q_heads, layout=layout)
        self.w = weights64(heads, d, self.q_heads, self.qw, self.kw)

    def check_forward(self, y):
        x = self.x.double()
        ref, r = forward64(x, self.w, self.table, self.pos, self.layout, self.eps)
        size = turn((x * r * self.w).abs(), self.table, self.pos, self.layout, sizes=True)
        tol = ROUND[y.dtype] * ref.abs() + (self.d / 2 + 10) * U * size + 2.0 ** -133
        err = (y.double() - ref).abs()
        assert bool((err <= tol).all()), float((err - tol).max())

    def check_grad(self, dx, dq, dk):
        x, dy = self.x.double(), self.dy.double()
        r = torch.rsqrt(x.square().mean(-1, keepdim=True) + self.eps)
        n = x * r
        g = turn(dy, self.table, self.pos, self.layout, back=True)
        size = turn(dy.abs(), self.table, self.pos, self.layout, sizes=True)
        m = (g * self.w * n).mean(-1, keepdim=True)
        ref = r * (g * self.w - n * m)
        most = (size * self.w.abs() * n.abs()).mean(-1, keepdim=True)
        tol = ROUND[dx.dtype] * ref.abs() + (2 * self.d + 32) * U * r * (size * self.w.abs() + n.abs() * most) + 2.0 ** -133
        err = (dx.double() - ref).abs()
        assert bool((err <= tol).all()), float((err - tol).max())
        for got, weight, part in ((dq, self.qw, slice(0, self.q_heads)), (dk, self.kw, slice(self.q_heads, self.heads))):
            if weight is None:
                assert got is None
                continue
            ref = (g * n)[:, part].sum((0, 1))
            count = self.T * (part.stop - part.start)
            tol = (count + self.d + 32) * U * (size * n.abs())[:, part].sum((0, 1)) + 2.0 ** -133
            assert got.dtype == F32 and bool(((got.double() - ref).abs() <= tol).all())

    def run(self, **kw):
        return rc.head_norm_rope(self.x, self.pos, self.table, **self.how, **kw)

    def grad(self, **kw):
        return rc.head_norm_rope_grad(self.dy, self.x, self.pos, self.table, **self.how, **kw)


SHAPES = [
    # T, heads, d, rot
    (1, 1, 2, 2), (1, 72, 64, 64), (16, 72, 64, 64), (7, 3, 64, 32), (33, 5, 128, 128), (40, 2, 96, 64), (9, 4, 96, 96),
    (5, 2, 512, 512), (6, 3, 256, 64), (3, 7, 72, 24), (11, 2, 66, 10), (2, 3, 130, 130), (1000, 9, 64, 64), (17, 1, 320, 320),
    (2, 1, 510, 510),
]


@pytest.mark.parametrize("T,heads,d,rot", SHAPES)
@pytest.mark.parametrize("layout", [PAIRS, HALVES])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_against_formula(T, heads, d, rot, layout, dtype):
    c = Case(T, heads, d, rot, dtype, layout, weight=dtype, q_heads=heads - heads // 3)
    c.check_forward(c.run())
    c.check_grad(*c.grad())


@pytest.mark.parametrize("dtype,table,weight", [(BF, F32, BF), (BF, BF, F32), (BF, F32, F32), (F32, BF, BF), (F32, F32, BF), (F32, BF, F32)])
@pytest.mark.parametrize("layout", [PAIRS, HALVES])
@pytest.mark.parametrize("d", [64, 66, 256])
def test_types_of_tables_and_weights(dtype, table, weight, layout, d):
    c = Case(20, 6, d, min(d, 64), dtype, layout, table=table, weight=weight, q_heads=4)
    c.check_forward(c.run())
    c.check_grad(*c.grad())


@pytest.mark.parametrize("d,rot", [(40, 16), (72, 32), (88, 16), (96, 32), (128, 32), (104, 96), (504, 16), (33, 10), (511, 2), (66, 64)])
@pytest.mark.parametrize("T,heads", [(3, 5), (4000, 12)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_rest_of_a_head_in_even_and_odd_parts(d, rot, T, heads, dtype):
    """Halves, of whose rest the two runs of a lane are of the same length or the first is longer."""
    c = Case(T if d < 256 else T // 8 + 1, heads, d, rot, dtype, HALVES, weight=dtype, q_heads=heads - 4)
    c.check_forward(c.run())
    c.check_grad(*c.grad())


@pytest.mark.parametrize("q_heads", [0, 1, 5])
@pytest.mark.parametrize("weight", [None, BF])
def test_which_heads_take_which_weight(q_heads, weight):
    c = Case(50, 5, 64, 64, BF, PAIRS, weight=weight, q_heads=q_heads)
    c.check_forward(c.run())
    c.check_grad(*c.grad())


@pytest.mark.parametrize("kw", [dict(extra=64), dict(extra=8, order="heads"), dict(extra=3), dict(offset=1), dict(order="heads", extra=1)])
@pytest.mark.parametrize("layout", [PAIRS, HALVES])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_strides_and_alignment(kw, layout, dtype):
    c = Case(21, 4, 64, 64, dtype, layout, weight=F32, q_heads=3, **kw)
    c.check_forward(c.run())
    c.check_grad(*c.grad())
    out = torch.full((4, 21, 70), 7.0, dtype=dtype, device=DEV)
    rows = out[:, :, 1:65].transpose(0, 1)
    assert c.run(out=rows).data_ptr() == rows.data_ptr()
    c.check_forward(rows)
    assert bool((out[:, :, 0] == 7).all()) and bool((out[:, :, 65:] == 7).all())


@pytest.mark.parametrize("T,heads,d,dtype", [(3000, 40, 128, BF), (9000, 16, 64, BF), (2500, 33, 96, BF), (1500, 20, 256, F32), (900, 24, 512, BF),
                                             (2000, 17, 128, F32)])
@pytest.mark.parametrize("layout", [PAIRS, HALVES])
@pytest.mark.parametrize("rot", [64, 0])
def test_much_work(T, heads, d, layout, dtype, rot):
    """Several heads an item, of odd numbers of query and key heads."""
    c = Case(T, heads, d, rot or d, dtype, layout, weight=dtype, q_heads=heads - 7)
    c.check_forward(c.run())
    dx, dq, dk = c.grad()
    c.check_grad(dx, dq, dk)
    again = c.grad()
    assert all(torch.equal(a, b) for a, b in zip((dx, dq, dk), again))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 66])
def test_in_place(dtype, d):
    c = Case(30, 6, d, 64, dtype, PAIRS, weight=F32, q_heads=4, extra=16)
    want, (dx, dq, dk) = c.run(), c.grad()
    for over in ("dy", "x"):
        x, dy = c.x.clone(), c.dy.clone()
        out = x if over == "x" else dy
        got = rc.head_norm_rope_grad(dy, x, c.pos, c.table, **c.how, out=out)
        assert torch.equal(out, dx) and torch.equal(got[1], dq) and torch.equal(got[2], dk)
    assert torch.equal(c.run(out=c.x), want) and torch.equal(c.x, want)


def test_positions_outside_the_table_are_normed_and_counted():
    for heads in (1, 6):
        c = Case(12, heads, 64, 64, BF, HALVES, weight=BF)
        c.pos[3], c.pos[5], c.pos[11] = -1, 512, 2 ** 40
        err = torch.zeros(1, dtype=I32, device=DEV)
        c.check_forward(c.run(err=err))
        assert int(err) == 3
        c.check_grad(*c.grad(err=err))
        assert int(err) == 6


def test_rows_of_zeros_and_infinities_stay_by_themselves():
    c = Case(8, 4, 64, 64, F32, PAIRS, weight=F32, q_heads=2, eps=0.0)
    y = c.run()
    c.x[2, 1], c.x[4, 3, 5], c.x[6, 0, 0] = 0.0, float("inf"), float("nan")
    odd = torch.zeros(8, 4, dtype=torch.bool, device=DEV)
    odd[2, 1] = odd[4, 3] = odd[6, 0] = True
    z = c.run()
    assert torch.equal(z[~odd], y[~odd]) and bool(torch.isnan(z[odd]).any(-1).all())
    dx, _, _ = c.grad()
    assert bool(torch.isfinite(dx[~odd]).all())
    # with an eps a head of zeros gives zeros
    c = Case(3, 2, 64, 64, BF, PAIRS)
    c.x[1, 1] = 0
    assert bool((c.run()[1, 1] == 0).all())


def test_no_tokens():
    c = Case(0, 4, 64, 64, BF, PAIRS, weight=BF, q_heads=3)
    assert c.run().shape == (0, 4, 64)
    dx, dq, dk = c.grad()
    assert dx.shape == (0, 4, 64) and not bool(dq.any()) and not bool(dk.any())


@pytest.mark.parametrize("layout", [PAIRS, HALVES])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_autograd(layout, dtype):
    c = Case(40, 6, 64, 32, dtype, layout, weight=dtype, q_heads=4)
    x, qw, kw = (t.detach().clone().requires_grad_() for t in (c.x, c.qw, c.kw))
    how = dict(c.how, q_weight=qw, k_weight=kw)
    y = rc.head_norm_rope(x, c.pos, c.table, **how)
    c.check_forward(y.detach())
    y.backward(c.dy)
    dx, dq, dk = c.grad()
    assert torch.equal(x.grad, dx) and torch.equal(qw.grad, dq.to(dtype)) and torch.equal(kw.grad, dk.to(dtype))
    # a broadcast gradient, and one without x
    kw.grad = None
    rc.head_norm_rope(c.x, c.pos, c.table, **dict(c.how, k_weight=kw)).sum().backward()
    _, _, dk = rc.head_norm_rope_grad(torch.ones_like(c.dy), c.x, c.pos, c.table, **c.how)
    assert torch.equal(kw.grad, dk.to(dtype))
    with torch.no_grad():
        assert rc.head_norm_rope(x, c.pos, c.table, **how).grad_fn is None
    with pytest.raises(RuntimeError):
        (g,) = torch.autograd.grad(rc.head_norm_rope(x, c.pos, c.table, **how).sum(), x, create_graph=True)
        g.sum().backward()


@pytest.mark.parametrize("layout", [PAIRS, HALVES])
def test_gradients_against_differences(layout):
    """Differences of the 64-bit formula along random directions; the kernel's FP32
    gradient is off by its tolerance along them, (2 d + 32) u or (N + d + 32) u of
    the sizes, and the differences by h^2 = 2^-40 of third derivatives below
    2^10."""
    c = Case(6, 3, 64, 48, F32, layout, weight=F32, q_heads=2)
    dx, dq, dk = c.grad()
    gen = torch.Generator(device=DEV).manual_seed(3)
    h = 2.0 ** -20

    def loss(x, qw, kw):
        w = weights64(3, 64, 2, qw, kw)
        return (forward64(x, w, c.table, c.pos, layout, c.eps)[0] * c.dy.double()).sum()
    at = [t.double() for t in (c.x, c.qw, c.kw)]
    for i, got in enumerate((dx, dq, dk)):
        for _ in range(4):
            v = torch.randn(at[i].shape, generator=gen, device=DEV, dtype=F64)
            plus, minus = (loss(*[t + s * h * v if j == i else t for j, t in enumerate(at)]) for s in (1, -1))
            want = (plus - minus) / (2 * h)
            size = (got.double() * v).abs().sum() + c.dy.double().abs().sum()
            assert abs(float(want - (got.double() * v).sum())) <= float(size) * (600 * U)


def test_captured_with_its_gradients():
    c = Case(64, 6, 64, 64, BF, PAIRS, weight=BF, q_heads=4)
    other = Case(64, 6, 64, 64, BF, PAIRS, weight=BF, q_heads=4, seed=9)
    ws = rc.head_norm_rope_grad_workspace(64, DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.run(), c.grad(workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, grads = c.run(), c.grad(workspace=ws)
    want = other.run(), other.grad()
    for name in ("x", "dy", "pos", "table"):
        getattr(c, name).copy_(getattr(other, name))
    c.qw.copy_(other.qw), c.kw.copy_(other.kw)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want[0]) and all(torch.equal(a, b) for a, b in zip(grads, want[1]))


def test_captured_backward_pass():
    """autograd's own, once the warm-up's graphs are gone."""
    c = Case(64, 6, 64, 64, BF, PAIRS, weight=BF, q_heads=4)
    x, qw, kw = (t.detach().clone().requires_grad_() for t in (c.x, c.qw, c.kw))
    how = dict(c.how, q_weight=qw, k_weight=kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        rc.head_norm_rope(x, c.pos, c.table, **how).backward(c.dy)
    torch.cuda.current_stream().wait_stream(side)
    x.grad = qw.grad = kw.grad = None
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rc.head_norm_rope(x, c.pos, c.table, **how).backward(c.dy)
    with torch.no_grad():
        x.mul_(2).add_(c.dy)
        c.dy.neg_()
    graph.replay()
    torch.cuda.synchronize()
    c.x = x.detach()
    dx, dq, dk = rc.head_norm_rope_grad(c.dy, c.x, c.pos, c.table, **c.how)
    c.check_grad(x.grad, dq, dk)
    assert torch.equal(x.grad, dx)
    assert torch.equal(qw.grad, dq.to(BF)) and torch.equal(kw.grad, dk.to(BF))


@pytest.mark.parametrize("which", ["forward", "grad"])
def test_on_another_stream(which):
    c = Case(4096, 16, 64, 64, BF, PAIRS, weight=BF, q_heads=9)
    call = c.run if which == "forward" else (lambda **kw: c.grad(**kw)[0])
    want = call().clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    block = torch.empty_like(want)
    torch.cuda._sleep(40_000_000)
    block.fill_(7.0)
    del block
    got = call(stream=side)
    side.synchronize()
    early = got.cpu()
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(early, want.cpu())
