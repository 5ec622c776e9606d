"""Outputs that the drafted tokens' calls make themselves on a stream other
than the current one: their memory belongs to that stream, so work still
queued on the current stream, over memory that was freed there, does not
reach them."""
import pytest
import torch

import rope_chain_gb300 as rc

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, F32, I32, I64 = torch.bfloat16, torch.float32, torch.int32, torch.int64


@pytest.fixture(scope="module", autouse=True)
def built():
    from rope_chain_gb300 import _build
    _build.build()


def table():
    return lambda **kw: rc.rope_table(1 << 16, 64, device=DEV, **kw)


def apply():
    x = torch.randn(4096, 16, 64, device=DEV).to(BF)
    cs, pos = rc.rope_table(4096, 64, device=DEV), torch.arange(4096, device=DEV)
    return lambda **kw: rc.rope_apply(x, pos, cs, **kw)


def attend():
    q = torch.randn(4096, 16, 64, device=DEV).to(BF)
    cache = torch.randn(16, 2, 16, 128, device=DEV).to(BF)
    start, ctx = torch.arange(0, 4097, 16, dtype=I32, device=DEV), torch.full((256,), 100, dtype=I32, device=DEV)
    blocks = torch.randint(0, 16, (256, 8), dtype=I32, device=DEV)
    return lambda **kw: rc.tree_attention(q, start, ctx, blocks, cache, **kw)


def adjust():
    x = torch.randn(64, 32768, device=DEV)
    start = torch.tensor([0, 64], dtype=I32, device=DEV)
    return lambda **kw: rc.logits_adjust(x, start, presence=torch.ones(1, device=DEV), **kw)


@pytest.mark.parametrize("make", [table, apply, attend, adjust])
def test_outputs_made_on_a_side_stream(make):
    call = make()
    want = call().clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    # a block of the output's size, freed on the current stream while work that
    # writes it is still queued there, behind some 20 ms
    block = torch.empty_like(want)
    torch.cuda._sleep(40_000_000)
    block.fill_(7.0)
    del block
    got = call(stream=side)
    side.synchronize()
    early = got.cpu()
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(early, want.cpu())
    # and the allocator has it under that stream
    at = got.data_ptr()
    owner = [s["stream"] for s in torch.cuda.memory_snapshot() if s["address"] <= at < s["address"] + s["total_size"]]
    assert owner == [side.cuda_stream]
