"""One verification step over trees of drafted tokens, on one GPU, with random
weights and tokens:

    rope_table       the cos|sin table, once
    qkv_front        up to 16 tokens: projection, norms, rotation and insert in one
    rope_apply,      more tokens: Q turned in place in the projection's rows,
    kv_store         K normed, turned and inserted with V
    tree_attention   every node over its sequence's cache and its ancestors
    logits_adjust    penalties over history and ancestors, biases, allowed tokens

and then, per sequence, the longest path of the tree whose every token is the
adjusted logits' choice at its parent.

    python examples/drafted_step.py [--seqs 3] [--nodes 13] [--context 1500]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import rope_chain_gb300 as rc

HD, EPS = rc.HEAD_DIM, 1e-6


def random_trees(seqs, nodes, gen):
    """parent [seqs][nodes] (-1: the root, node 0), depths, and the ancestor
    words [seqs * nodes, words] with each node's own bit set."""
    words = (nodes + 63) // 64
    parents, depths, masks = [], [], []
    for _ in range(seqs):
        parent, depth, mask = [-1], [0], [1]
        for i in range(1, nodes):
            p = int(torch.randint(max(0, i - 4), i, (1,), generator=gen))
            parent.append(p)
            depth.append(depth[p] + 1)
            mask.append(mask[p] | 1 << i)
        parents.append(parent)
        depths.append(depth)
        for m in mask:
            row = [m >> 64 * w & (1 << 64) - 1 for w in range(words)]
            masks.append([v - (1 << 64) if v >> 63 else v for v in row])
    return parents, depths, torch.tensor(masks, dtype=torch.int64)


class DraftedStep:
    """The buffers of a step and the step itself.  Everything is allocated
    here, so that run() may be captured into a CUDA graph and replayed with
    other tokens, positions, lengths and blocks."""

    def __init__(self, seqs=3, nodes=13, context=1500, *, hidden=2048, heads=64, kv_heads=8, vocab=32000,
                 block_size=16, seed=0, device="cuda:0"):
        dev = torch.device(device)
        cpu = torch.Generator().manual_seed(seed)
        gpu = torch.Generator(device=dev).manual_seed(seed)
        rand = lambda *shape, scale=1.0: (torch.randn(*shape, generator=gpu, device=dev) * scale).to(torch.bfloat16)
        ints = lambda values, dtype=torch.int32: torch.tensor(values, dtype=dtype, device=dev)
        self.heads, self.kv_heads, self.vocab = heads, kv_heads, vocab
        rows = self.rows = seqs * nodes

        # weights, and the table that the front, the store and rope_apply share
        width = HD * (2 * heads + 2 * kv_heads)                     # [Q | K | V | gate]
        self.embed = rand(vocab, hidden)
        self.w_qkv = rand(width, hidden, scale=hidden ** -0.5)
        self.w_out = rand(hidden, HD * heads, scale=(HD * heads) ** -0.5)
        self.w_head = rand(vocab, hidden, scale=hidden ** -0.5)
        self.table = rc.rope_table(context + nodes, scaling="parts", factor=4.0,
                                   original_max_position=max(1, (context + nodes) // 4), device=dev)

        # the trees: rows, ancestors, positions and the cache rows of their keys
        self.parents, depths, mask = random_trees(seqs, nodes, cpu)
        self.tree_mask = mask.to(dev)
        self.tokens = torch.randint(vocab, (rows,), generator=cpu).to(torch.int32).to(dev)
        self.row_start = ints([b * nodes for b in range(seqs + 1)])
        self.context_len = ints([context] * seqs)
        self.positions = ints([context + d for tree in depths for d in tree], torch.int64)
        width_blocks = -(-(context + nodes) // block_size)
        blocks = torch.randperm(seqs * width_blocks, generator=cpu).view(seqs, width_blocks)
        self.block_table = blocks.to(torch.int32).to(dev)
        slots = [[int(blocks[b, p // block_size]) * block_size + p % block_size for p in range(context + nodes)]
                 for b in range(seqs)]
        self.slots = ints([s for b in range(seqs) for s in slots[b][context:]], torch.int64)

        # the context's keys and values, through the store
        self.cache = torch.zeros(seqs * width_blocks, kv_heads, block_size, 2 * HD, dtype=torch.bfloat16, device=dev)
        if context:
            kv = rand(1, seqs * context, 2 * HD * kv_heads)
            rc.kv_store_from_projection(kv, kv_heads, torch.arange(context, device=dev).repeat(seqs),
                                        [ints([s for b in range(seqs) for s in slots[b][:context]], torch.int64)],
                                        self.table, [self.cache], EPS)

        # what has been said, and what may come
        self.history = torch.randint(vocab, (seqs * (context + 1),), generator=cpu).to(torch.int32).to(dev)
        self.history_start = ints([b * (context + 1) for b in range(seqs + 1)], torch.int64)
        self.prompt_len = ints([context // 2] * seqs)
        self.repetition = torch.full((seqs,), 1.2, device=dev)
        self.frequency = torch.full((seqs,), 0.1, device=dev)
        self.presence = torch.full((seqs,), 0.3, device=dev)
        self.allowed = torch.full((rows, (vocab + 31) // 32), -1, dtype=torch.int32, device=dev)
        self.allowed[:, 0] = -2                                     # token 0 is never allowed

        self.qkv = torch.empty(rows, width, dtype=torch.bfloat16, device=dev)
        self.q = self.qkv[:, :HD * heads].view(rows, heads, HD)     # columns of the projection's rows
        self.attended = torch.empty(rows, heads, HD, dtype=torch.bfloat16, device=dev)
        self.err = torch.zeros(1, dtype=torch.int32, device=dev)
        self.workspace = rc.tree_attention_workspace(rows, seqs, heads, kv_heads, dev)

    def run(self):
        """The step: adjusted logits [rows, vocab]; the trees' keys and values
        are in the cache afterwards.  Also kept: `raw`, the logits before."""
        x = self.embed[self.tokens]
        nq, nkv = HD * self.heads, HD * self.kv_heads
        if self.rows <= 16:
            rc.qkv_front(x, self.w_qkv, self.heads, self.kv_heads, self.positions, self.table, self.slots, self.cache,
                         EPS, out=self.qkv, err=self.err)
        else:
            torch.matmul(x, self.w_qkv.t(), out=self.qkv)
            self.q.copy_(torch.nn.functional.rms_norm(self.q.float(), (HD,), eps=EPS))
            rc.rope_apply(self.q, self.positions, self.table, out=self.q, err=self.err)
            k, v = (self.qkv[:, at:at + nkv].view(1, self.rows, self.kv_heads, HD) for at in (nq, nq + nkv))
            rc.kv_store(k, v, self.positions, [self.slots], self.table, [self.cache], EPS, err=self.err)
        rc.tree_attention(self.q, self.row_start, self.context_len, self.block_table, self.cache,
                          tree_mask=self.tree_mask, out=self.attended, err=self.err, workspace=self.workspace)
        gated = self.attended.view(self.rows, nq) * torch.sigmoid(self.qkv[:, nq + 2 * nkv:])
        x = x + gated @ self.w_out.t()
        self.raw = x @ self.w_head.t()
        return rc.logits_adjust(self.raw, self.row_start, history=self.history, history_start=self.history_start,
                                prompt_len=self.prompt_len, draft_tokens=self.tokens, tree_mask=self.tree_mask,
                                repetition=self.repetition, frequency=self.frequency, presence=self.presence,
                                allowed=self.allowed, err=self.err)

    def accepted(self, logits):
        """Per sequence the tokens of the path that the logits agree with, and
        the token they choose after it."""
        choice = logits.argmax(-1).view(len(self.parents), -1).tolist()
        tokens = self.tokens.view(len(self.parents), -1).tolist()
        paths = []
        for parent, choose, token in zip(self.parents, choice, tokens):
            node, path = 0, []
            while True:
                path.append(choose[node])
                after = [i for i, p in enumerate(parent) if p == node and token[i] == choose[node]]
                if not after:
                    break
                node = after[0]
            paths.append(path)
        return paths


def main():
    parser = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    parser.add_argument("--seqs", type=int, default=3)
    parser.add_argument("--nodes", type=int, default=13)
    parser.add_argument("--context", type=int, default=1500)
    args = parser.parse_args()
    step = DraftedStep(args.seqs, args.nodes, args.context)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            step.run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        logits = step.run()
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    for _ in range(20):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    for b, path in enumerate(step.accepted(logits)):
        print(f"sequence {b}: {len(path) - 1} drafted tokens accepted, then {path[-1]}")
    print(f"{step.rows} drafted tokens, {args.seqs} contexts of {args.context}: "
          f"{start.elapsed_time(end) / 20 * 1e3:.1f} us a step, {int(step.err.item())} errors, "
          f"faults {rc.read_device_faults():#x}")


if __name__ == "__main__":
    main()
