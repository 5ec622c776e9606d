"""The example's step over caches in bf16 and in 4 bits, with and without a window:
its attention against the formula in 64 bits on the step's own Q and cache, what it
inserted in 4 bits, and the accepted rows moved to follow the context, from where a
second step goes on.

Tolerances.  Attention, with A = sum_p w_p |v_p|: 2^-8 |ref| for the output's
rounding, 2^-8 A for the weights', 2^-12 A for FP32 scores, exponentials and
sums."""
import numpy as np
import pytest
import torch

import rope_chain_gb300 as rc
from examples.drafted_step import HD, DraftedStep

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from rope_chain_gb300 import _build
    _build.build()
    rc.read_device_faults(clear=True)
    yield
    assert rc.read_device_faults(clear=True) == 0


SMALL = dict(hidden=256, heads=16, kv_heads=2, vocab=1003)


def rows_at(s, b, p):
    """K | V of a sequence's keys p as the cache has them, 64 bits [keys, kv_heads, 128]."""
    bs = s.cache.shape[2]
    slots = s.block_table[b].long()[p // bs] * bs + p % bs
    if s.four:
        return rc.kv4_load(slots, s.cache, s.scales).double()
    return s.cache[slots // bs, :, slots % bs].double()


def check_attention(s):
    seqs, nodes = len(s.parents), len(s.parents[0])
    q = s.q.double().view(seqs, nodes, s.kv_heads, -1, HD)
    bits = s.tree_mask.cpu().numpy().view(np.uint64).reshape(seqs, nodes, -1)
    j = np.arange(nodes)
    for b in range(seqs):
        ctx = int(s.context_len[b])
        kv = rows_at(s, b, torch.arange(ctx + nodes, device=s.cache.device))
        k, v = kv[..., :HD], kv[..., HD:]
        see = np.ones((nodes, ctx + nodes), dtype=bool)
        see[:, ctx:] = (bits[b][:, j // 64] >> (j % 64).astype(np.uint64)) & np.uint64(1) == 1
        if s.window:
            for i in range(nodes):
                order = np.flatnonzero(see[i])
                see[i, order[s.window["sinks"]:max(s.window["sinks"], len(order) - s.window["window"])]] = False
        t = torch.einsum("nhgd,phd->nhgp", q[b], k) * HD ** -0.5
        t = t.masked_fill(~torch.from_numpy(see).to(t.device)[:, None, None], -float("inf"))
        w = torch.softmax(t, -1)
        ref, mag = torch.einsum("nhgp,phd->nhgd", w, v), torch.einsum("nhgp,phd->nhgd", w, v.abs())
        got = s.attended.view(seqs, nodes, s.kv_heads, -1, HD)[b].double()
        assert bool(((got - ref).abs() <= 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -12) * mag + 2.0 ** -30).all())


@pytest.mark.parametrize("seqs,nodes,context", [(1, 1, 3), (1, 16, 40), (3, 13, 700), (2, 70, 129)])
@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("window", [dict(), dict(window=50, sinks=3)])
def test_steps_one_after_another(seqs, nodes, context, four, window):
    s = DraftedStep(seqs, nodes, context, seed=nodes, four=four, **window, **SMALL)
    s.run()
    assert int(s.err) == 0
    check_attention(s)
    # a path in each tree: from its last node back to the root
    paths = []
    for parent in s.parents:
        node, path = len(parent) - 1, []
        while node >= 0:
            path.insert(0, node)
            node = parent[node]
        paths.append(path)
    dev = s.cache.device
    before = [rows_at(s, b, context + torch.tensor(p, device=dev)) for b, p in enumerate(paths)]
    past = [rows_at(s, b, torch.arange(context, device=dev)) for b in range(seqs)]
    s.keep(paths)
    assert s.context_len.tolist() == [context + len(p) for p in paths] and int(s.err) == 0
    for b, p in enumerate(paths):
        assert torch.equal(rows_at(s, b, context + torch.arange(len(p), device=dev)), before[b])
        assert torch.equal(rows_at(s, b, torch.arange(context, device=dev)), past[b])
    # the next step, of fewer nodes: as many as the blocks have room for
    room = nodes - max(len(p) for p in paths)
    if room == 0:
        return
    starts = s.context_len.tolist()
    s.positions.copy_(torch.tensor([min(c + i, s.table.shape[0] - 1) for c in starts for i in range(nodes)], device=dev))
    bs = s.cache.shape[2]
    slots = [[int(s.block_table[b, (c + i) // bs]) * bs + (c + i) % bs if i < room else -1 for i in range(nodes)] for b, c in enumerate(starts)]
    s.slots.copy_(torch.tensor(slots, device=dev).flatten())
    s.run()
    assert torch.isfinite(s.attended.float()).all()
    got = s.attended.view(seqs, nodes, s.kv_heads, -1, HD)
    # the root sees the context, the kept rows and itself
    q = s.q.double().view(seqs, nodes, s.kv_heads, -1, HD)[:, 0]
    for b, c in enumerate(starts):
        kv = rows_at(s, b, torch.arange(c + 1, device=dev))
        if s.window:
            keep = torch.zeros(c + 1, dtype=torch.bool, device=dev)
            keep[:s.window["sinks"]] = True
            keep[max(0, c + 1 - s.window["window"]):] = True
            kv = kv[keep]
        w = torch.softmax(torch.einsum("hgd,phd->hgp", q[b], kv[..., :HD]) * HD ** -0.5, -1)
        ref, mag = (torch.einsum("hgp,phd->hgd", w, f(kv[..., HD:])) for f in (lambda x: x, torch.abs))
        assert bool(((got[b, 0].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -12) * mag + 2.0 ** -30).all())


@pytest.mark.parametrize("nodes", [16, 21])
def test_the_inserted_rows_in_four_bits(nodes):
    """K of the step as head_norm_rope (or the front) left it in the projection's rows, V as projected: 4 bits of them."""
    s = DraftedStep(1, nodes, 40, seed=3, four=True, **SMALL)
    s.run()
    nq, nkv = HD * s.heads, HD * s.kv_heads
    k, v = (s.qkv[:, at:at + nkv].view(nodes, s.kv_heads, HD) for at in (nq, nq + nkv))
    cache, scales = rc.new_kv4_cache(nodes, s.kv_heads, 1, k.device)
    slots = torch.arange(nodes, device=k.device)
    rc.kv4_store(k, v, slots, cache, scales)
    want = rc.kv4_load(slots, cache, scales)
    got = rows_at(s, 0, 40 + slots)
    assert torch.equal(got, want.double())
    # a group's largest element over 7, and half of that for rounding: within 5/8 of a step
    exact = torch.cat([k, v], -1).double().unflatten(-1, (4, 32))
    step = exact.abs().amax(-1, keepdim=True) / 7
    assert bool(((got.unflatten(-1, (4, 32)) - exact).abs() <= 0.5625 * step).all())
    # normed: a key's mean square is 1, within bf16
    assert bool((k.double().square().mean(-1) - 1).abs().max() < 2.0 ** -6)


@pytest.mark.parametrize("four", [False, True])
def test_replayed_graph_takes_other_lengths(four):
    s, other = (DraftedStep(2, 20, 300, seed=1, four=four, window=64, sinks=4, **SMALL) for _ in range(2))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        logits = s.run()
    for t in (s, other):
        t.tokens.copy_((t.tokens + 17) % 1003)
        t.context_len.fill_(161)
        p = 161 + torch.arange(20, device=t.slots.device)
        t.slots.copy_((t.block_table.long()[:, p // 16] * 16 + p % 16).flatten())
    graph.replay()
    expected = other.run()
    torch.cuda.synchronize()
    assert torch.equal(logits, expected) and torch.equal(s.attended, other.attended)
