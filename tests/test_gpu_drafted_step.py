"""The example's step over trees of drafted tokens: its attention and adjusted
logits against the formulas in 64 bits on the step's own Q, cache and logits,
what it inserted, and a replayed graph.

Tolerances.  Attention, with A = sum_p w_p |v_p|: 2^-8 |ref| for the output's
rounding, 2^-8 A for the weights', 2^-12 A for FP32 scores, exponentials and
sums.  Adjusted logits: five FP32 roundings of the largest intermediate value,
2^-8 of the result for its own rounding.  Q after norm and rotation: bf16 twice
(2^-8 each) of at most the pair's length, 2^-10 for the table's bf16 and FP32."""
import numpy as np
import pytest
import torch

import rope_chain_gb300 as rc
from examples.drafted_step import EPS, HD, DraftedStep

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from rope_chain_gb300 import _build
    _build.build()
    rc.read_device_faults(clear=True)
    yield
    assert rc.read_device_faults(clear=True) == 0


def keys_of(s, b, n):
    """K and V of sequence b's first n logical keys, 64 bits."""
    p = torch.arange(n, device=s.cache.device)
    bs = s.cache.shape[2]
    kv = s.cache[s.block_table[b].long()[p // bs], :, p % bs].double()
    return kv[..., :HD], kv[..., HD:]


def check_attention(s, context):
    seqs, nodes = len(s.parents), len(s.parents[0])
    q = s.q.double().view(seqs, nodes, s.kv_heads, -1, HD)
    bits = s.tree_mask.cpu().numpy().view(np.uint64).reshape(seqs, nodes, -1)
    for b in range(seqs):
        k, v = keys_of(s, b, context + nodes)
        j = np.arange(nodes)
        sees = torch.from_numpy((bits[b][:, j // 64] >> (j % 64).astype(np.uint64)) & np.uint64(1) == 1).to(q.device)
        t = torch.einsum("nhgd,phd->nhgp", q[b], k) * HD ** -0.5
        t[..., context:] = t[..., context:].masked_fill(~sees[:, None, None], -float("inf"))
        w = torch.softmax(t, -1)
        ref, mag = torch.einsum("nhgp,phd->nhgd", w, v), torch.einsum("nhgp,phd->nhgd", w, v.abs())
        got = s.attended.view(seqs, nodes, s.kv_heads, -1, HD)[b].double()
        assert bool(((got - ref).abs() <= 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -12) * mag + 2.0 ** -30).all())


def check_logits(s, logits):
    seqs, nodes = len(s.parents), len(s.parents[0])
    x, got = s.raw.double().cpu().numpy(), logits.double().cpu().numpy()
    tokens, said = s.tokens.cpu().numpy(), s.history.cpu().numpy()
    start, prompt = s.history_start.cpu().numpy(), s.prompt_len.cpu().numpy()
    for b in range(seqs):
        h = said[start[b]:start[b + 1]]
        for i in range(nodes):
            g, r = np.zeros(s.vocab, np.int64), b * nodes + i
            np.add.at(g, h[prompt[b]:], 1)
            node = i
            while node >= 0:                            # the node and its ancestors
                g[tokens[b * nodes + node]] += 1
                node = s.parents[b][node]
            repeated = g > 0
            repeated[h[:prompt[b]]] = True
            rep, freq, pres = (float(t[b]) for t in (s.repetition, s.frequency, s.presence))
            y = np.where(repeated, np.where(x[r] > 0, x[r] / rep, x[r] * rep), x[r])
            tol = 5 * 2.0 ** -24 * (np.abs(y) + freq * g + pres)
            y = y - freq * g - pres * (g > 0)
            assert got[r, 0] == -np.inf                 # token 0 is never allowed
            assert (np.abs(got[r, 1:] - y[1:]) <= (tol + 2.0 ** -8 * np.abs(y) * (1 + 2.0 ** -7))[1:]).all()


@pytest.mark.parametrize("seqs,nodes,context", [(1, 1, 0), (1, 16, 40), (3, 5, 333), (3, 13, 1500), (2, 70, 129)])
def test_step(seqs, nodes, context):
    s = DraftedStep(seqs, nodes, context, hidden=256, heads=16, kv_heads=2, vocab=1003, seed=nodes)
    logits = s.run()
    torch.cuda.synchronize()
    assert int(s.err.item()) == 0
    check_attention(s, context)
    check_logits(s, logits)
    assert all(len(path) >= 1 for path in s.accepted(logits))


@pytest.mark.parametrize("seqs,nodes", [(1, 16), (2, 16)])
def test_queries_and_keys_are_normed_and_turned(seqs, nodes):
    """Both ways to project (the front, and the calls for more tokens)."""
    s = DraftedStep(seqs, nodes, 20, hidden=256, heads=16, kv_heads=2, vocab=1003, seed=9)
    s.run()
    cs = s.table.double()[s.positions][:, None]
    c, sn = cs[..., :HD // 2], cs[..., HD // 2:]
    proj = (s.embed[s.tokens].double() @ s.w_qkv.double().t())
    size = (s.embed[s.tokens].double().abs() @ s.w_qkv.double().abs().t())

    def turned(at, heads):
        x = proj[:, at:at + HD * heads].view(s.rows, heads, HD)
        r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
        # the projection's own rounding and FP32 sums, relative to the head's size
        slack = (size[:, at:at + HD * heads].view(s.rows, heads, HD).amax(-1, keepdim=True) * 256 * 2.0 ** -24
                 + 2.0 ** -8 * x.abs().amax(-1, keepdim=True)) * r
        a, b = (x * r)[..., ::2], (x * r)[..., 1::2]
        length = (a.square() + b.square()).sqrt()
        ref = torch.stack((a * c - b * sn, a * sn + b * c), -1).flatten(-2)
        tol = ((2.0 ** -7 + 2.0 ** -10) * length).repeat_interleave(2, -1) + 3 * slack
        return ref, tol

    ref, tol = turned(0, s.heads)
    assert bool(((s.q.double() - ref).abs() <= tol).all())
    ref, tol = turned(HD * s.heads, s.kv_heads)
    bs = s.cache.shape[2]
    rows = s.cache[s.slots // bs, :, s.slots % bs].double()
    assert bool(((rows[..., :HD] - ref).abs() <= tol).all())


def test_replayed_graph_takes_other_tokens():
    s, other = (DraftedStep(2, 7, 100, hidden=256, heads=16, kv_heads=2, vocab=1003, seed=1) for _ in range(2))
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
        t.context_len.fill_(61)
        # the drafted keys then follow 61 context keys
        p = 61 + torch.arange(7, device=t.slots.device)
        t.slots.copy_((t.block_table.long()[:, p // 16] * 16 + p % 16).flatten())
    graph.replay()
    expected = other.run()
    torch.cuda.synchronize()
    assert torch.equal(logits, expected) and torch.equal(s.attended, other.attended)
