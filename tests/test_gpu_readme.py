"""The README's drafted tokens' step and its form over a cache in 4 bits, run as they
are written there: the rows that the second one stores stand for what the store of the
bf16 caches makes of the same projection."""
import math
import os
import re

import pytest
import torch

import rope_chain_gb300 as rc

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, I32 = torch.bfloat16, torch.int32
README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


@pytest.fixture(scope="module", autouse=True)
def built():
    from rope_chain_gb300 import _build
    _build.build()


def blocks():
    """The README's two blocks of Python that attend over drafted tokens."""
    with open(README) as f:
        found = [b for b in re.findall(r"```python\n(.*?)```", f.read(), re.S) if "attention(" in b]
    assert len(found) == 2 and "kv4_attention" in found[1]
    return found


@pytest.mark.parametrize("rows", [13, 29])
def test_steps(rows):
    gen = torch.Generator(device=DEV).manual_seed(rows)
    rand = lambda *shape, scale=1.0: (torch.randn(*shape, generator=gen, device=DEV) * scale).to(BF)  # noqa: E731
    heads, kv_heads, hidden_dim, vocab, block_size, num_blocks = 16, 2, 1024, 500, 16, 5
    W = rand(64 * (2 * heads + 2 * kv_heads), hidden_dim, scale=hidden_dim ** -0.5)
    to_vocab = rand(64 * heads, vocab, scale=0.05)
    ints = lambda *v: torch.tensor(v, dtype=I32, device=DEV)  # noqa: E731
    names = dict(
        rc=rc, math=math, torch=torch, dev=DEV, heads=heads, kv_heads=kv_heads, W=W, rows=rows, seqs=1, eps=1e-6, block_size=block_size,
        num_blocks=num_blocks, max_position=32768, hidden=rand(rows, hidden_dim), positions=torch.arange(rows, device=DEV) * 997,
        slots=torch.arange(rows, device=DEV) + block_size, qkv=torch.empty(rows, W.shape[0], dtype=BF, device=DEV),
        row_start=ints(0, rows), context_len=ints(0), block_table=ints(1, 2, 3, 4)[None], path=ints(0)[None], path_len=ints(0),
        cache=torch.zeros(num_blocks, kv_heads, block_size, 128, dtype=BF, device=DEV), ancestors=None,
        head=lambda out: out.view(rows, -1) @ to_vocab, history=None, history_start=None, tokens=torch.zeros(rows, dtype=I32, device=DEV),
        repetition=torch.ones(1, device=DEV), allowed=None)
    first, second = blocks()
    if rows <= 16:
        exec(first, names)                               # the front stores into the bf16 cache
        bf16, out = names["cache"], names["out"].double()
    else:                                                # "more": kv_store of the projection
        exec(first.split("rc.qkv_front")[0], names)      # (the table)
        qkv, bf16 = names["hidden"] @ W.t(), names["cache"]
        nq, nkv = 64 * heads, 64 * kv_heads
        k, v = (qkv[:, at:at + nkv].contiguous().view(rows, kv_heads, 64) for at in (nq, nq + nkv))
        rc.kv_store(k[None], v[None], names["positions"], [names["slots"]], names["table"], [bf16], 1e-6)
        q = rc.head_norm_rope(qkv[:, :nq].view(rows, heads, 64), names["positions"], names["table"], eps=1e-6)
        out = rc.tree_attention(q, names["row_start"], ints(0), names["block_table"], bf16).double()
    exec(second, names)
    want = bf16.permute(0, 2, 1, 3).reshape(-1, kv_heads, 128)[names["slots"]].double()
    held = rc.kv4_load(names["slots"], names["cache"], names["scales"]).double()
    # a number is off by half a scale, max / 7 to four bits (2^-4 off at most); K's bf16
    # roundings, at most three of 2^-8 of its size, move both, and ties between two numbers
    most = want.unflatten(-1, (4, 32)).abs().amax(-1, keepdim=True)
    assert bool(((held - want).unflatten(-1, (4, 32)).abs() <= most * ((1 + 2.0 ** -4) / 14 + 4 * 2.0 ** -8)).all())
    # the same keys and values but for that: outputs alike, which doubled angles are not
    got = names["out"].double()
    alike = (got * out).sum() / (got.norm() * out.norm())
    assert float(alike) > 0.95
    torch.cuda.synchronize()
