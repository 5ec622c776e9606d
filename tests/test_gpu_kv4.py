"""rc_kv4_store and rc_kv4_load: bytes, scales and values against the format's
definition in 64 bits, all of them exact (a scale has four significant bits and a
number three, so their product is a bf16 number)."""
import pytest
import torch

import rope_chain_gb300 as rc

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, F64, I32, I64 = torch.bfloat16, torch.float64, torch.int32, torch.int64
MOST = 7 * 2.0 ** 100


@pytest.fixture(scope="module", autouse=True)
def built():
    from rope_chain_gb300 import _build
    _build.build()


def codes64(x):
    """x [..., 64]: whole numbers -7 .. 7 and the scales [..., 2], in 64 bits on the host."""
    g = torch.nan_to_num(x.double().cpu(), nan=0.0, posinf=MOST, neginf=-MOST).clamp(-MOST, MOST).unflatten(-1, (2, 32))
    m, e = torch.frexp(g.abs().amax(-1) / torch.tensor([7.0], dtype=F64))
    scale = torch.ldexp(torch.round(m * 16) / 16, e)         # m in [1/2, 1): four bits, ties to even
    scale = torch.where(scale < 2.0 ** -100, torch.zeros_like(scale), scale)
    q = g / torch.where(scale > 0, scale, torch.ones_like(scale))[..., None]
    n = torch.where(scale[..., None] > 0, q.sign() * (q.abs() - 0.5).ceil(), torch.zeros_like(q))
    return n.flatten(-2), scale


def view(gen, T, H, order, extra=0, sigma=1.0):
    if order == "tokens":
        return (sigma * torch.randn(T, H * 64 + extra, generator=gen, device=DEV)).to(BF)[:, :H * 64].view(T, H, 64)
    return (sigma * torch.randn(H, T, 64 + extra, generator=gen, device=DEV)).to(BF)[..., :64].transpose(0, 1)


def check(k, v, slots, cache, scales, before):
    """Every byte of the cache: rows at slots as defined, the others as before."""
    bs = cache.shape[2]
    want, wscale = (t.cpu().clone() for t in before)
    keep = (slots >= 0) & (slots < cache.shape[0] * bs)
    at = slots[keep].cpu()
    n, s = [], []
    for x in (k, v):
        a, b = codes64(x[keep])
        n.append(a)
        s.append(b)
    n, s = torch.cat(n, -1), torch.cat(s, -1)
    u = (n + 8).to(torch.uint8)
    want[at // bs, :, at % bs] = u[..., 0::2] | (u[..., 1::2] << 4)
    wscale[at // bs, :, at % bs] = s.to(BF)
    assert torch.equal(s.to(BF).double(), s)
    assert torch.equal(cache.cpu(), want) and torch.equal(scales.cpu(), wscale)
    values = n * s.repeat_interleave(32, -1)
    assert torch.equal(values.to(BF).double(), values)
    return keep, values


def fresh(nb, H, bs, seed=0):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    cache, scales = rc.new_kv4_cache(nb, H, bs, DEV)
    cache.random_(0, 256, generator=gen)
    scales.copy_(torch.rand(scales.shape, generator=gen, device=DEV))
    return cache, scales


@pytest.mark.parametrize("T,H,bs", [(1, 1, 1), (1, 8, 16), (3, 5, 7), (39, 8, 16), (500, 2, 24), (333, 16, 128), (9000, 3, 16), (20001, 8, 16)])
@pytest.mark.parametrize("order", ["tokens", "heads"])
def test_store_and_load(T, H, bs, order):
    gen = torch.Generator(device=DEV).manual_seed(T)
    nb = -(-T // bs) + 2
    cache, scales = fresh(nb, H, bs)
    before = cache.clone(), scales.clone()
    k, v = view(gen, T, H, order, extra=64), view(gen, T, H, order, sigma=30.0)
    k[T // 2, H // 2] *= 0.001
    v[T // 3, 0, 32:] = 0
    slots = torch.randperm(nb * bs, generator=gen, device=DEV)[:T]
    slots[T // 2::7] = -1 - slots[T // 2::7]
    err = torch.zeros(1, dtype=I32, device=DEV)
    rc.kv4_store(k, v, slots, cache, scales, err=err)
    keep, values = check(k, v, slots, cache, scales, before)
    got = rc.kv4_load(slots, cache, scales, err=err)
    assert got.shape == (T, H, 128) and int(err) == 0
    assert torch.equal(got[keep].double().cpu(), values) and not bool(got[~keep].any())


def test_every_mantissa():
    """Every size of eight bits over every largest one of a group, ties among them."""
    top = torch.arange(128, 256, device=DEV).repeat_interleave(64)
    k = torch.zeros(128 * 64, 1, 64, device=DEV)
    sub = torch.arange(64, device=DEV).repeat(128)
    for j in range(1, 32):
        size = 128 + (sub * 31 + j * 61) % 128
        k[:, 0, j] = torch.minimum(size.float() * 2.0 ** -(j % 6), top.float()) * (1 - 2 * (j % 2))
    k[:, 0, 0] = top
    k[:, 0, 32:] = k[:, 0, :32] * 2.0 ** -20
    k = k.to(BF)
    cache, scales = fresh(512, 1, 16)
    before = cache.clone(), scales.clone()
    slots = torch.arange(128 * 64, device=DEV)
    rc.kv4_store(k, -k, slots, cache, scales)
    keep, values = check(k, -k, slots, cache, scales, before)
    assert torch.equal(rc.kv4_load(slots, cache, scales).double().cpu(), values)


def test_sizes_at_the_ends_and_what_is_not_finite():
    k = torch.randn(12, 2, 64, device=DEV).to(BF)
    v = k.clone()
    k[0] *= 2.0 ** -99
    k[1] *= 2.0 ** -101
    k[2], v[2] = 2.0 ** -133, -2.0 ** -126
    k[3] *= 2.0 ** 99
    k[4] *= 2.0 ** 110
    k[5, 0, 3], k[6, 1, 40], v[7, 0, 0], v[8, 1] = float("inf"), float("nan"), float("-inf"), float("nan")
    k[9, 0, :32] = 0
    k[10, 0, 1], k[10, 1, 2] = float("inf"), float("inf")
    cache, scales = fresh(2, 2, 16)
    before = cache.clone(), scales.clone()
    slots = torch.arange(12, device=DEV)
    err = torch.zeros(1, dtype=I32, device=DEV)
    rc.kv4_store(k, v, slots, cache, scales, err=err)
    assert int(err) == 6                                   # a row's head each
    keep, values = check(k, v, slots, cache, scales, before)
    got = rc.kv4_load(slots, cache, scales)
    assert torch.equal(got.double().cpu(), values) and bool(torch.isfinite(got.float()).all())


def test_scales_that_the_store_does_not_write():
    cache, scales = fresh(1, 1, 8)
    scales[0, 0, 0] = float("nan")
    scales[0, 0, 1], scales[0, 0, 2], scales[0, 0, 3] = float("inf"), 2.0 ** 101, -2.0 ** 100
    scales[0, 0, 4, 2] = float("nan")
    got = rc.kv4_load(torch.arange(8, device=DEV), cache, scales)[:, 0].double()
    n = torch.stack((cache[0, 0] % 16, cache[0, 0] // 16), -1).flatten(-2).double() - 8
    # four significant bits, no sign, at most 2^100
    s = (scales[0, 0].view(torch.int16) & 0x7FF0).view(BF).double()
    s = torch.where(s <= 2.0 ** 100, s, 2.0 ** 100).repeat_interleave(32, -1)
    assert torch.equal(got, n * s) and bool(torch.isfinite(got).all())


def test_slots_past_the_cache_are_counted():
    k = torch.randn(6, 3, 64, device=DEV).to(BF)
    cache, scales = fresh(2, 3, 4)
    before = cache.clone(), scales.clone()
    slots = torch.tensor([0, 8, 7, 2 ** 40, -5, 3], device=DEV)
    err = torch.zeros(1, dtype=I32, device=DEV)
    rc.kv4_store(k, k, slots, cache, scales, err=err)
    assert int(err) == 2
    check(k, k, slots, cache, scales, before)
    got = rc.kv4_load(slots, cache, scales, err=err)
    assert int(err) == 4 and not bool(got[[1, 3, 4]].any()) and bool(got[[0, 2, 5]].any())


@pytest.mark.parametrize("T", [5, 40000])
def test_outputs_aligned_to_16_bytes(T):
    cache, scales = fresh(2500, 4, 16)
    slots = torch.randint(0, 40000, (T,), device=DEV)
    want = rc.kv4_load(slots, cache, scales)
    flat = torch.zeros(T * 512 + 8, dtype=BF, device=DEV)
    out = flat[8:].view(T, 4, 128)
    assert out.data_ptr() % 32 == 16
    assert rc.kv4_load(slots, cache, scales, out=out).data_ptr() == out.data_ptr()
    assert torch.equal(out, want) and not bool(flat[:8].any())


def test_nothing_to_store_or_load():
    cache, scales = fresh(2, 3, 4)
    none = torch.empty(0, dtype=I64, device=DEV)
    before = cache.clone()
    k = torch.empty(0, 3, 64, dtype=BF, device=DEV)
    rc.kv4_store(k, k, none, cache, scales)
    assert torch.equal(cache, before) and rc.kv4_load(none, cache, scales).shape == (0, 3, 128)


def test_a_zero_cache_holds_zeros():
    cache, scales = rc.new_kv4_cache(2, 2, 8, DEV)
    assert not bool(rc.kv4_load(torch.arange(16, device=DEV), cache, scales).any())


def test_rows_past_32_bits():
    """A cache of more than 2^31 bytes and more than 2^32 of the bf16 values it stands for."""
    nb, H, bs = 4500, 64, 128
    cache, scales = rc.new_kv4_cache(nb, H, bs, DEV)
    slots = torch.tensor([nb * bs - 1, 0, nb * bs // 2], device=DEV)
    k = torch.randn(3, H, 64, device=DEV).to(BF)
    rc.kv4_store(k, -k, slots, cache, scales)
    got = rc.kv4_load(slots, cache, scales).cpu().double()
    n, s = codes64(k)
    value = n * s.repeat_interleave(32, -1)
    assert torch.equal(got, torch.cat([value, -value], -1))
    rows = cache[-1, :, -1]
    assert bool((rows != 0).any()) and not bool(cache[1:nb // 2].any())


def test_captured_and_replayed():
    k, v = (torch.randn(100, 4, 64, device=DEV).to(BF) for _ in range(2))
    slots = torch.randperm(160, device=DEV)[:100]
    cache, scales = rc.new_kv4_cache(10, 4, 16, DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        rc.kv4_store(k, v, slots, cache, scales)
        rc.kv4_load(slots, cache, scales)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rc.kv4_store(k, v, slots, cache, scales)
        got = rc.kv4_load(slots, cache, scales)
    k.copy_(torch.randn(100, 4, 64, device=DEV))
    slots.copy_(torch.randperm(160, device=DEV)[:100])
    graph.replay()
    torch.cuda.synchronize()
    n, s = codes64(k)
    assert torch.equal(got[..., :64].double().cpu(), n * s.repeat_interleave(32, -1))


def test_on_another_stream():
    k = torch.randn(60000, 4, 64, device=DEV).to(BF)
    slots = torch.randperm(60000, device=DEV)
    cache, scales = rc.new_kv4_cache(60000 // 16, 4, 16, DEV)
    rc.kv4_store(k, k, slots, cache, scales)
    want = rc.kv4_load(slots, cache, scales).clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    block = torch.empty_like(want)
    torch.cuda._sleep(40_000_000)
    block.fill_(7.0)
    del block
    got = rc.kv4_load(slots, cache, scales, stream=side)
    side.synchronize()
    early = got.cpu()
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(early, want.cpu())
