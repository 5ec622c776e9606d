"""rc_rope_table and rc_rope_apply against the formulas in 64 bits.

Tolerances: a rotated element has two FP32 roundings of products and sums
(2^-23 (|a c| + |b s|)) and one rounding to its type (2^-8 relative in bf16,
2^-24 in FP32); a table entry has the half-turn's 2^-24 (times pi), the sine's
2^-22, the gain's 2^-24 and the type's rounding."""
import math

import numpy as np
import pytest
import torch

import rope_chain_gb300 as rc

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, F32 = torch.bfloat16, torch.float32
ROUND = {BF: 2.0 ** -8, F32: 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def built():
    from rope_chain_gb300 import _build
    _build.build()


def angles(n, rot, theta, scaling, factor, original, fast=32.0, slow=1.0):
    j = np.arange(rot // 2, dtype=np.float64)
    if scaling == "base":
        theta = theta * factor ** (rot / (rot - 2))
    inv = theta ** (-2 * j / rot)
    if scaling == "linear":
        inv = inv / factor
    if scaling == "parts":
        d = lambda beta: rot * math.log(original / (2 * math.pi * beta)) / (2 * math.log(theta))
        lo, hi = max(math.floor(d(fast)), 0), min(math.ceil(d(slow)), rot - 1)
        ramp = np.clip((j - lo) / max(hi - lo, 0.001), 0, 1)
        inv = inv * (1 - ramp) + inv / factor * ramp
    # the angle modulo 2 pi in extended precision where numpy has it
    turns = (np.arange(n, dtype=np.longdouble)[:, None] * inv.astype(np.longdouble)) / (2 * np.longdouble(np.pi))
    return ((turns - np.floor(turns)) * 2 * np.longdouble(np.pi)).astype(np.float64)


@pytest.mark.parametrize("n,rot", [(1, 2), (7, 6), (300, 64), (4096, 128), (131072, 64), (100, 10), (33, 512)])
@pytest.mark.parametrize("scaling", ["none", "linear", "base", "parts"])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_table(n, rot, scaling, dtype):
    if rot == 2 and scaling == "base":
        pytest.skip("base scaling needs four columns")
    factor, original, gain = 4.0, max(64.0, n / 4), 1.2 if scaling == "parts" else 1.0
    got = rc.rope_table(n, rot, theta=10000.0, scaling=scaling, factor=factor, original_max_position=original,
                        attention_factor=gain, dtype=dtype, device=DEV)
    a = angles(n, rot, 10000.0, scaling, factor, original)
    ref = gain * np.concatenate([np.cos(a), np.sin(a)], 1)
    g = np.float64(np.float32(gain))
    # double's own rounding of the angle: n * 2^-53 turns of the reference
    tol = ROUND[dtype] * np.abs(ref) + g * (math.pi * 2.0 ** -24 + 2.0 ** -22 + 2.0 ** -24) + n * 2.0 ** -50 + 2.0 ** -133
    err = np.abs(got.double().cpu().numpy() - ref)
    assert (err <= tol).all(), (err - tol).max()


def test_table_is_the_chains_table():
    """bf16, 64 columns, no scaling: the table of the context workloads, to one spacing (both are rounded)."""
    import workloads
    want = torch.from_numpy(workloads.cos_sin_table(8192).view(np.int16)).view(BF).double()
    got = rc.rope_table(8192, 64, device=DEV).double().cpu()
    assert ((got - want).abs() <= 2.0 ** -7 * want.abs() + 2.0 ** -21).all()


def rotate(x, cs, pos, layout, inverse):
    rot = cs.shape[1]
    half = rot // 2
    c, s = cs.double()[pos][:, None, :half], cs.double()[pos][:, None, half:]
    s = -s if inverse else s
    y, tol = x.double().clone(), torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    a, b = (slice(0, half), slice(half, rot)) if layout == rc.RC_ROPE_HALVES else (slice(0, rot, 2), slice(1, rot, 2))
    u, v = x.double()[..., a], x.double()[..., b]
    y[..., a], y[..., b] = u * c - v * s, v * c + u * s
    size = (u * c).abs() + (v * s).abs()
    tol[..., a] = size
    tol[..., b] = (v * c).abs() + (u * s).abs()
    return y, 2.0 ** -23 * tol + ROUND[x.dtype] * y.abs() + 2.0 ** -133


APPLY = [(1, 1, 2, 2), (1, 72, 64, 64), (16, 72, 64, 64), (5, 3, 64, 32), (1000, 8, 128, 64), (33, 7, 96, 48),
         (17, 2, 80, 10), (3, 1, 6, 4), (4097, 16, 64, 64), (2, 5, 256, 256), (3, 2, 4096, 512)]


@pytest.mark.parametrize("T,heads,dim,rot", APPLY)
@pytest.mark.parametrize("layout", [rc.RC_ROPE_PAIRS, rc.RC_ROPE_HALVES])
@pytest.mark.parametrize("xt,tt", [(BF, BF), (BF, F32), (F32, BF), (F32, F32)])
def test_apply(T, heads, dim, rot, layout, xt, tt):
    gen = torch.Generator(device=DEV).manual_seed(T + heads)
    x = torch.randn(T, heads, dim, generator=gen, device=DEV).to(xt)
    cs = rc.rope_table(500, rot, dtype=tt, device=DEV)
    pos = torch.randint(0, 500, (T,), generator=gen, device=DEV)
    for inverse in (False, True):
        got = rc.rope_apply(x, pos, cs, layout=layout, inverse=inverse)
        ref, tol = rotate(x, cs, pos, layout, inverse)
        assert bool(((got.double() - ref).abs() <= tol).all())
        assert torch.equal(got[..., rot:], x[..., rot:])


@pytest.mark.parametrize("layout", [rc.RC_ROPE_PAIRS, rc.RC_ROPE_HALVES])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_views_in_place_and_odd_strides(layout, dtype):
    gen = torch.Generator(device=DEV).manual_seed(3)
    cs = rc.rope_table(64, 32, dtype=dtype, device=DEV)
    pos = torch.randint(0, 64, (9,), generator=gen, device=DEV)
    for lead, row in ((0, 640), (64, 704), (3, 647), (1, 641)):
        whole = torch.randn(9, row, generator=gen, device=DEV).to(dtype)
        x = whole[:, lead:lead + 6 * 64].view(9, 6, 64) if lead == 0 else whole.as_strided((9, 6, 64), (row, 64, 1), lead)
        ref, tol = rotate(x, cs, pos, layout, False)
        fresh = rc.rope_apply(x, pos, cs, layout=layout)
        # heads outermost in the output
        turned = torch.empty(6, 9, 64, dtype=dtype, device=DEV).transpose(0, 1)
        rc.rope_apply(x, pos, cs, layout=layout, out=turned)
        before = whole.clone()
        rc.rope_apply(x, pos, cs, layout=layout, out=x)
        for got in (fresh, turned, x):
            assert bool(((got.double() - ref).abs() <= tol).all())
        keep = torch.ones(9, row, dtype=torch.bool, device=DEV)
        keep[:, lead:lead + 6 * 64] = False
        assert torch.equal(whole[keep], before[keep])


def test_positions_outside_pass_through_and_count():
    x = torch.randn(6, 3, 64, device=DEV).to(BF)
    cs = rc.rope_table(10, 64, device=DEV)
    pos = torch.tensor([0, -1, 10, 9, 2 ** 40, -2 ** 62], device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = rc.rope_apply(x, pos, cs, err=err)
    assert int(err.item()) == 4
    for t in (1, 2, 4, 5):
        assert torch.equal(got[t], x[t])
    ref, tol = rotate(x[3:4], cs, pos[3:4], rc.RC_ROPE_PAIRS, False)
    assert bool(((got[3:4].double() - ref).abs() <= tol).all())


@pytest.mark.parametrize("layout", [rc.RC_ROPE_PAIRS, rc.RC_ROPE_HALVES])
def test_inverse_is_the_gradient(layout):
    """Against differences: f(x) = <w, rope(x)> is linear, so a step of 2^-3
    in one element changes f by exactly grad * 2^-3 up to FP32 rounding: the
    sums over 2 * 32 outputs of size below 8 each carry 2^-24 * 8 * 64."""
    gen = torch.Generator(device=DEV).manual_seed(9)
    x = torch.randn(2, 1, 48, generator=gen, device=DEV)
    w = torch.randn(2, 1, 48, generator=gen, device=DEV)
    cs = rc.rope_table(4096, 32, scaling="parts", factor=4.0, original_max_position=1024, attention_factor=1.1386,
                       dtype=F32, device=DEV)
    pos = torch.tensor([17, 4001], device=DEV)
    grad = rc.rope_apply(w, pos, cs, layout=layout, inverse=True)
    for t in range(2):
        for e in range(48):
            step = torch.zeros_like(x)
            step[t, 0, e] = 0.125
            up = (w.double() * rc.rope_apply(x + step, pos, cs, layout=layout).double()).sum()
            down = (w.double() * rc.rope_apply(x - step, pos, cs, layout=layout).double()).sum()
            assert abs(float((up - down) / 0.25) - float(grad[t, 0, e])) <= 2.0 ** -24 * 8 * 64 / 0.25


def test_empty_tensors():
    cs = rc.rope_table(5, device=DEV)
    x = torch.zeros(0, 3, 64, dtype=BF, device=DEV)
    assert rc.rope_apply(x, torch.zeros(0, dtype=torch.int64, device=DEV), cs).shape == x.shape
    assert rc.rope_table(0, device=DEV).shape == (0, 64)


def test_the_fronts_rotation():
    """Pairs, all 64 columns, bf16: what the store does to keys after their norm (norm switched off by unit keys)."""
    H, T = 2, 40
    gen = torch.Generator(device=DEV).manual_seed(6)
    kv = torch.randn(1, T, 2 * H * 64, generator=gen, device=DEV).to(BF)
    pos = torch.randint(0, 100, (T,), generator=gen, device=DEV)
    cs = rc.rope_table(100, device=DEV)
    slots = torch.arange(T, device=DEV)
    plain, turned = (torch.zeros(3, H, 16, 128, dtype=BF, device=DEV) for _ in range(2))
    rc.kv_store_from_projection(kv, H, None, [slots], None, [plain], 1e-6)
    rc.kv_store_from_projection(kv, H, pos, [slots], cs, [turned], 1e-6)
    keys = plain[slots // 16, :, slots % 16, :64]
    assert torch.equal(rc.rope_apply(keys, pos, cs), turned[slots // 16, :, slots % 16, :64])


@pytest.mark.parametrize("layout", [rc.RC_ROPE_PAIRS, rc.RC_ROPE_HALVES])
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("side", [False, True])
def test_autograd_takes_the_transposed_rotation(layout, inverse, side):
    gen = torch.Generator(device=DEV).manual_seed(12)
    x = torch.randn(9, 3, 96, generator=gen, device=DEV).to(BF).requires_grad_()
    w = torch.randn(9, 3, 96, generator=gen, device=DEV).to(BF)
    cs, pos = rc.rope_table(64, 48, device=DEV), torch.randint(0, 64, (9,), generator=gen, device=DEV)
    stream = torch.cuda.Stream() if side else None
    torch.cuda.synchronize()
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    y = rc.rope_apply(x, pos, cs, layout=layout, inverse=inverse, stream=stream, err=err)
    torch.cuda.synchronize()
    y.backward(w)
    torch.cuda.synchronize()
    with torch.no_grad():
        assert torch.equal(y, rc.rope_apply(x, pos, cs, layout=layout, inverse=inverse))
        assert torch.equal(x.grad, rc.rope_apply(w, pos, cs, layout=layout, inverse=not inverse))
    # a gradient that is broadcast along the heads' elements
    x.grad = None
    rc.rope_apply(x, pos, cs, layout=layout, inverse=inverse).sum().backward()
    with torch.no_grad():
        assert torch.equal(x.grad, rc.rope_apply(torch.ones_like(w), pos, cs, layout=layout, inverse=not inverse))
    assert not rc.rope_apply(x.detach(), pos, cs, layout=layout).requires_grad


# much work: several heads a thread, from 2 * 1024 units an SM on in halves and 4 * 1024 in pairs (heads that are no
# multiple of either, a copied tail, rows of a wider tensor)
@pytest.mark.parametrize("T,heads,dim,rot,row", [(11201, 7, 64, 64, 7 * 64), (9001, 9, 128, 64, 9 * 128 + 64), (3001, 30, 96, 96, 30 * 96),
                                                 (9999, 5, 256, 64, 6 * 256)])
@pytest.mark.parametrize("layout", [rc.RC_ROPE_PAIRS, rc.RC_ROPE_HALVES])
@pytest.mark.parametrize("xt,tt", [(BF, BF), (BF, F32), (F32, F32)])
def test_apply_much_work(T, heads, dim, rot, row, layout, xt, tt):
    gen = torch.Generator(device=DEV).manual_seed(T)
    whole = torch.randn(T, row, generator=gen, device=DEV).to(xt)
    x = whole.as_strided((T, heads, dim), (row, dim, 1))
    cs, pos = rc.rope_table(700, rot, dtype=tt, device=DEV), torch.randint(0, 700, (T,), generator=gen, device=DEV)
    pos[5] = -1
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    for inverse in (False, True):
        ref, tol = rotate(x, cs, pos.clamp(min=0), layout, inverse)
        ref[5], tol[5] = x[5].double(), 0
        got = rc.rope_apply(x, pos, cs, layout=layout, inverse=inverse, err=err)
        turned = torch.empty(heads, T, dim, dtype=xt, device=DEV).transpose(0, 1)      # heads outermost
        rc.rope_apply(x, pos, cs, layout=layout, inverse=inverse, out=turned)
        assert torch.equal(got, turned) and bool(((got.double() - ref).abs() <= tol).all())
        assert torch.equal(got[..., rot:], x[..., rot:])
    assert int(err.item()) == 2
    before = whole.clone()
    rc.rope_apply(x, pos, cs, layout=layout, inverse=True, out=x)
    assert torch.equal(x, got) and torch.equal(whole[:, heads * dim:], before[:, heads * dim:])


@pytest.mark.parametrize("dtype,bound", [(F32, 2.0 ** -21), (BF, 2.0 ** -20)])
@pytest.mark.parametrize("n,rot,gain", [(1 << 20, 8, 1.0), (70001, 66, 1.25), (4099, 512, 0.5)])
def test_table_within_the_stated_bounds(dtype, bound, n, rot, gain):
    """Before its rounding an entry is within 2^-21 (FP32) or 2^-20 (bf16) of the formula's, times the gain."""
    got = rc.rope_table(n, rot, theta=10000.0, attention_factor=gain, dtype=dtype, device=DEV).double().cpu().numpy()
    a = angles(n, rot, 10000.0, "none", 1.0, 1.0)
    ref = gain * np.concatenate([np.cos(a), np.sin(a)], 1)
    assert (np.abs(got - ref) <= ROUND[dtype] * (np.abs(ref) + bound * gain) + bound * gain + n * 2.0 ** -50).all()
