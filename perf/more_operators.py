"""Cases, plain forms and 64-bit values of more operators around the paged
caches: norms of query and key heads with their rotation, a cache in 4 bits
(its store and its attention), attention with a sliding window, and the move of
accepted tokens' rows.

`run` computes an operator in elementary torch operations (own = False) or
through the framework's public calls (own = True); both take what `prepare`
makes.  Head, block and table shapes are those of the context K/V workloads and
of the decode QKV front (8 or 16 KV heads of 64, 64 query heads, blocks of 16,
tables up to 131072 positions, up to 8 layers)."""
import math

import torch

own = False

HD = 64     # head width of the paged caches
GROUP = 32  # elements that share a scale in a cache of 4 bits


def listed():
    att = dict(kv_heads=8, group=8, block=16, ragged=True, lse=False)
    window = dict(att, op="window")
    four = dict(att, op="four", window=0, sinks=0)
    return [
        # Q and K of one drafted tree straight from a projection's rows: latency counts
        dict(op="norm", name="norm_tree", tokens=16, q_heads=64, k_heads=8, width=64, rot=64, layout="pairs", type="bf16", weights=False, train=False),
        # Q and K of a training batch, with the gradients of rows and weights
        dict(op="norm", name="norm_train", tokens=16384, q_heads=32, k_heads=8, width=128, rot=128, layout="halves", type="bf16", weights=True, train=True),
        # a few drafted trees' keys and values into 4 bits: latency counts
        dict(op="store", name="store_tree", tokens=39, kv_heads=8, block=16),
        # a whole context's of one layer
        dict(op="store", name="store_context", tokens=131072, kv_heads=8, block=16),
        # one token that looks back over the last 1024 of a long context
        dict(window, name="window_one_token", seqs=1, nodes=1, ctx=131071, window=1024, sinks=4),
        # a serving batch of single tokens, a window of 4096
        dict(window, name="window_decode_batch", seqs=64, nodes=1, ctx=16384, window=4096, sinks=16),
        # wide trees over a window of long contexts
        dict(window, name="window_tree_large", seqs=8, nodes=64, ctx=32768, window=8192, sinks=128, ragged=False),
        # one token over a long cache in 4 bits, with the log sums for a later merge
        dict(four, name="four_decode_long", seqs=1, nodes=1, ctx=131071, lse=True),
        # one token each for a serving batch of ragged lengths, in 4 bits
        dict(four, name="four_decode_batch", seqs=64, nodes=1, ctx=8200),
        # the front's largest tree for a batch, window and sinks over 4 bits
        dict(four, name="four_tree_batch", seqs=16, nodes=16, ctx=8192, window=6000, sinks=64),
        # a few small trees' accepted paths, every layer's rows
        dict(op="move", name="move_small", seqs=3, nodes=13, path=4, ctx=1500, layers=5, kv_heads=8, block=16, cache="bf16"),
        # a batch of wide trees
        dict(op="move", name="move_batch", seqs=64, nodes=64, path=12, ctx=500, layers=8, kv_heads=8, block=16, cache="bf16"),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "store", "window", "window", "four", "four", "four", "move"])
    if op == "norm":
        q, k = rng.choice([(64, 8), (32, 8), (16, 16), (8, 1), (5, 0), (0, 16), (12, 4)])
        width = rng.choice([64, 64, 128, 128, 96, 256])
        train = rng.random() < 0.5
        tokens = _spread(rng, 1, 16384 * 40 * 128 // ((q + k) * width * 2))
        return dict(op=op, tokens=tokens, q_heads=q, k_heads=k, width=width, rot=rng.choice([32, 64, width]), layout=rng.choice(["pairs", "halves"]),
                    type=rng.choice(["bf16", "bf16", "f32"]), weights=train or rng.random() < 0.5, train=train)
    if op == "store":
        kv = rng.choice([1, 2, 4, 8, 16])
        return dict(op=op, tokens=_spread(rng, 1, 131072 * 8 // (kv * 2)), kv_heads=kv, block=rng.choice([16, 16, 32, 64, 128]))
    if op == "move":
        seqs, nodes, layers, kv = _spread(rng, 1, 64), _spread(rng, 2, 64), rng.choice([1, 3, 4, 5, 8]), rng.choice([1, 2, 8, 16])
        if seqs * nodes * layers * kv > 64 * 64 * 8 * 8:
            kv = 8
        return dict(op=op, seqs=seqs, nodes=nodes, path=_spread(rng, 1, max(1, nodes // 4)), ctx=_spread(rng, 1, 500), layers=layers, kv_heads=kv,
                    block=rng.choice([16, 16, 32, 64]), cache=rng.choice(["bf16", "four"]))
    kv, group = rng.choice([(1, 8), (2, 4), (4, 8), (8, 8), (8, 4), (16, 1), (16, 4), (8, 1), (1, 64), (2, 16)])
    nodes, seqs = _spread(rng, 1, 64), _spread(rng, 1, 64)
    # at most the largest listed case's cache and products (those of the plain form: every key)
    most = min(64 * 8192 * 8 / (seqs * kv), 8 * 32768 * 4096 / (2 * seqs * nodes * kv * group), 131072)
    ctx = _spread(rng, 16, max(17, int(most)))
    window = _spread(rng, 1, 2 * ctx) if op == "window" or rng.random() < 0.5 else 0
    return dict(op=op, seqs=seqs, nodes=nodes, ctx=ctx, kv_heads=kv, group=group, block=rng.choice([16, 16, 16, 32, 64, 128]), window=window,
                sinks=rng.choice([0, 0, 1, 4, 64, 128]) if window else 0, ragged=rng.random() < 0.7, lse=rng.random() < 0.3)


# ------------------------------------------------------------ what is in hand


def _lengths(case):
    """Context lengths of the sequences, from the case alone."""
    n, ctx = case["seqs"], case["ctx"]
    return [ctx - (b * 5 % n) * ctx // (2 * n) if case.get("ragged", True) else ctx for b in range(n)]


def _node_counts(case):
    """Tree sizes of the sequences: the full size, and one less for every other."""
    return [max(1, case["nodes"] - b % 2) for b in range(case["seqs"])]


def _tree(gen, counts):
    """Packed ancestor-or-self bits int64 [rows, words] of random trees."""
    most = max(counts)
    words = -(-most // 64)
    sees = torch.zeros(len(counts), most, most, dtype=torch.bool)
    u = torch.rand(len(counts), most, generator=gen)
    every = torch.arange(len(counts))
    for i in range(most):
        if i:
            parent = i - 1 - (u[:, i] * min(i, 4)).long()
            sees[:, i] = sees[every, parent]
        sees[:, i, i] = True
    bits = torch.zeros(len(counts), most, words, dtype=torch.int64)
    for j in range(most):
        bits[:, :, j // 64] |= sees[:, :, j].long() << (j % 64)
    live = torch.arange(most)[None, :] < torch.tensor(counts)[:, None]
    return bits[live].contiguous()


def _tables(case, host, lens, counts):
    """Block tables int32 [seqs, width] of random blocks, and how many blocks there are."""
    bs = case["block"]
    need = [-(-(c + n) // bs) for c, n in zip(lens, counts)]
    blocks = sum(need) + 3
    order = torch.randperm(blocks, generator=host).to(torch.int32)
    table = torch.zeros(len(need), max(need), dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, blocks


def _codes(x):
    """x [..., 64], two groups of 32: whole numbers -7 .. 7 and the groups' scales.
    A scale is the group's largest size over 7 to four significant bits (to the
    nearest, ties to even), 0 below 2^-100; a number is the nearest to x / scale,
    ties toward zero."""
    g = x.float().unflatten(-1, (-1, GROUP))
    most = g.abs().amax(-1)
    m, e = torch.frexp(most / torch.full_like(most, 7))  # (by a tensor: a quotient, not a product with 1/7)
    scale = torch.ldexp(torch.round(m * 16) / 16, e)
    scale = torch.where(scale < 2.0 ** -100, 0, scale)
    q = g / torch.where(scale > 0, scale, 1)[..., None]
    n = torch.where(scale[..., None] > 0, q.sign() * (q.abs() - 0.5).ceil(), 0)
    return n.flatten(-2), scale


def _packed(n):
    """Whole numbers [..., 2k] as bytes [..., k]: n + 8, the even element in the low half."""
    u = (n + 8).to(torch.uint8)
    return u[..., 0::2] | (u[..., 1::2] << 4)


def _unpacked(b):
    """The whole numbers of bytes, FP32."""
    return torch.stack((b & 15, b >> 4), -1).flatten(-2).float() - 8


def prepare(case, seed):
    dev = torch.device("cuda:0")
    gen = torch.Generator(device=dev).manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    op = case["op"]
    s = dict(op=op, case=case)
    if own:
        import rope_chain_gb300 as rc
        s["rc"] = rc
    if op == "norm":
        T, n, w, rot = case["tokens"], case["q_heads"] + case["k_heads"], case["width"], case["rot"]
        dt = torch.bfloat16 if case["type"] == "bf16" else torch.float32
        most = 131072
        inv = 10000.0 ** (-2.0 * torch.arange(rot // 2, device=dev, dtype=torch.float64) / rot)
        ang = torch.arange(most, device=dev, dtype=torch.float64)[:, None] * inv
        table = torch.cat([ang.cos(), ang.sin()], 1).to(dt)
        # Q and K lead each row of a projection [Q | K | V ...]; rows of uneven size
        rows = (torch.randn(T, (n + 8) * w, generator=gen, device=dev) * torch.rand(T, 1, generator=gen, device=dev).mul_(3).exp_()).to(dt)
        s.update(x=rows[:, : n * w].view(T, n, w), table=table, halves=case["layout"] == "halves", rot=rot, eps=1e-6,
                 positions=torch.randint(0, most, (T,), generator=gen, device=dev))
        for name in ("q", "k"):
            has = case["weights"] and case[name + "_heads"] > 0
            s[name + "_weight"] = (1 + 0.2 * torch.randn(w, generator=gen, device=dev)).to(dt) if has else None
        if case["train"]:
            s["dy"] = torch.randn(T, n, w, generator=gen, device=dev).to(dt)
        return s
    if op == "store":
        T, kv, bs = case["tokens"], case["kv_heads"], case["block"]
        blocks = -(-T // bs) + 3
        order = torch.randperm(blocks, generator=host).to(dev)
        t = torch.arange(T, device=dev)
        # K and V as a projection's columns
        rows = torch.randn(T, 2 * kv * HD, generator=gen, device=dev).to(torch.bfloat16)
        s.update(k=rows[:, : kv * HD].view(T, kv, HD), v=rows[:, kv * HD:].view(T, kv, HD), slots=order[t // bs] * bs + t % bs,
                 cache=torch.zeros(blocks, kv, bs, HD, dtype=torch.uint8, device=dev),
                 scales=torch.zeros(blocks, kv, bs, 4, dtype=torch.bfloat16, device=dev))
        return s
    counts, lens, kv, bs = _node_counts(case), _lengths(case), case["kv_heads"], case["block"]
    start = torch.tensor([0] + counts).cumsum(0).to(torch.int32)
    table, blocks = _tables(case, host, lens, counts)
    s.update(row_start=start.to(dev), rows=int(start[-1]), seqs=len(counts), block_table=table.to(dev),
             context_len=torch.tensor(lens, dtype=torch.int32).to(dev))
    if op == "move":
        # Accepted paths as in a tree in order of depth: the root and perhaps a few
        # more are in place, the others lie beyond the path's length, so that a
        # second pass over the state finds the rows where the first one found them.
        path = torch.zeros(len(counts), case["path"], dtype=torch.int32)
        length = []
        for b, n in enumerate(counts):
            most = min(case["path"], max(1, n // 2))
            m = int(torch.randint(max(1, most // 2), most + 1, (1,), generator=host))
            fixed = int(torch.randint(0, m + 1, (1,), generator=host)) if n == 1 else min(m, 1 + int(torch.randint(0, 2, (1,), generator=host)))
            far = m + torch.randperm(n - m, generator=host)[: m - fixed].sort().values if n > m else torch.zeros(0)
            node = torch.cat([torch.arange(m - far.numel()), far])
            path[b, :m] = node.to(torch.int32)
            length.append(m)
        s.update(path=path.to(dev), path_len=torch.tensor(length, dtype=torch.int32).to(dev))
        caches = []
        for _ in range(case["layers"]):
            if case["cache"] == "bf16":
                caches.append(torch.randn(blocks, kv, bs, 2 * HD, generator=gen, device=dev, dtype=torch.bfloat16))
            else:
                caches.append(torch.randint(0, 256, (blocks, kv, bs, HD), generator=gen, device=dev, dtype=torch.uint8))
                caches.append(torch.rand(blocks, kv, bs, 4, generator=gen, device=dev).to(torch.bfloat16))
        s["caches"] = caches
        return s
    mask = _tree(host, counts)
    group = case["group"]
    s.update(
        tree_mask=mask.to(dev), most_nodes=max(counts), most_keys=max(c + n for c, n in zip(lens, counts)),
        seq_of_row=torch.repeat_interleave(torch.arange(len(counts)), torch.tensor(counts)).to(dev),
        node_of_row=torch.cat([torch.arange(c) for c in counts]).to(dev),
        # Q leads each row of a projection [Q | K | V], as the front writes it
        q=torch.randn(s["rows"], (group + 2) * kv * HD, generator=gen, device=dev).to(torch.bfloat16)[:, : group * kv * HD].view(s["rows"], -1, HD))
    if op == "window":
        s["cache"] = torch.randn(blocks, kv, bs, 2 * HD, generator=gen, device=dev, dtype=torch.bfloat16)
    else:
        s["cache"] = torch.empty(blocks, kv, bs, HD, dtype=torch.uint8, device=dev)
        s["scales"] = torch.empty(blocks, kv, bs, 4, dtype=torch.bfloat16, device=dev)
        step = max(1, 2 ** 20 // (kv * bs))
        for at in range(0, blocks, step):
            rows = torch.randn(min(step, blocks - at), kv, bs, 2 * HD, generator=gen, device=dev).to(torch.bfloat16)
            n, scale = _codes(rows)
            s["cache"][at:at + step], s["scales"][at:at + step] = _packed(n), scale.to(torch.bfloat16)
    if own:
        make = s["rc"].tree_attention_workspace if op == "window" else s["rc"].kv4_attention_workspace
        s["workspace"] = make(s["rows"], s["seqs"], group * kv, kv, dev)
    return s


# ------------------------------------------------------------ one pass


def _columns(s):
    """The pairs' first and second elements."""
    rot = s["rot"]
    return (slice(0, rot // 2), slice(rot // 2, rot)) if s["halves"] else (slice(0, rot, 2), slice(1, rot, 2))


def _turned(s, y, sign):
    """y with its pairs turned by the table's rows (sign -1: back)."""
    cs = s["table"][s["positions"]].float()
    half = s["rot"] // 2
    c, n = cs[:, None, :half], sign * cs[:, None, half:]
    a, b = _columns(s)
    u, v = y[..., a].clone(), y[..., b].clone()
    y[..., a] = u * c - v * n
    y[..., b] = v * c + u * n
    return y


def _weights(s, like):
    """[heads, width] of the heads' weights."""
    case = s["case"]
    w = torch.ones(case["q_heads"] + case["k_heads"], case["width"], **like)
    if s["q_weight"] is not None:
        w[: case["q_heads"]] = s["q_weight"].to(w.dtype)
    if s["k_weight"] is not None:
        w[case["q_heads"]:] = s["k_weight"].to(w.dtype)
    return w


def _norm_plain(s):
    case, x = s["case"], s["x"].float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"])
    w = _weights(s, dict(dtype=torch.float32, device=x.device))
    y = _turned(s, x * r * w, 1).to(s["x"].dtype)
    if "dy" not in s:
        return y
    g = _turned(s, s["dy"].float().clone(), -1)
    n = x * r
    dw = (g * n).double().sum(0)
    g = g * w
    dx = (r * (g - n * (g * n).mean(-1, keepdim=True))).to(s["x"].dtype)
    nq = case["q_heads"]
    return y, dx, [dw[part].sum(0).float() for part, name in ((slice(0, nq), "q"), (slice(nq, None), "k")) if s[name + "_weight"] is not None]


def _store_plain(s):
    bs = s["cache"].shape[2]
    blk, off = s["slots"] // bs, s["slots"] % bs
    n, scale = _codes(torch.cat([s["k"], s["v"]], -1))
    s["cache"][blk, :, off] = _packed(n)
    s["scales"][blk, :, off] = scale.to(torch.bfloat16)
    n, scale = _unpacked(s["cache"][blk, :, off]), s["scales"][blk, :, off].float()
    return (n * scale.repeat_interleave(GROUP, -1)).to(torch.bfloat16)


def _sees(s):
    """Which nodes each row sees: bool [rows, most_nodes]."""
    j = torch.arange(s["most_nodes"], device=s["tree_mask"].device)
    return (s["tree_mask"][:, j // 64] >> (j % 64)) & 1 == 1


def _attention_plain(s):
    case = s["case"]
    kv, g, bs = case["kv_heads"], case["group"], case["block"]
    B, N, S = s["seqs"], s["most_nodes"], s["most_keys"]
    dev = s["q"].device
    p = torch.arange(S, device=dev)
    blocks, off = s["block_table"].long()[:, (p // bs)], (p % bs)[None, :]
    if case["op"] == "window":
        rows = s["cache"][blocks, :, off].float()  # [B, S, kv, 128]
    else:
        rows = _unpacked(s["cache"][blocks, :, off])
        rows.unflatten(-1, (4, GROUP)).mul_(s["scales"][blocks, :, off].float()[..., None])
    k, v = rows[..., :HD].permute(0, 2, 3, 1), rows[..., HD:].permute(0, 2, 1, 3)
    q = torch.zeros(B, N, kv, g, HD, device=dev)
    q[s["seq_of_row"], s["node_of_row"]] = s["q"].float().view(-1, kv, g, HD)
    q = q.permute(0, 2, 1, 3, 4).reshape(B, kv, N * g, HD)
    ctx = s["context_len"].long()
    node = p[None, :] - ctx[:, None]  # [B, S]
    sees = torch.zeros(B, N, N, dtype=torch.bool, device=dev)
    sees[s["seq_of_row"], s["node_of_row"]] = _sees(s)
    inside = (node >= 0) & (node < N)
    pick = node.clamp(0, N - 1)[:, None, :].expand(B, N, S)
    seen = (node < 0)[:, None, :] | (sees.gather(2, pick) & inside[:, None, :])  # [B, N, S]
    if case["window"]:
        # a key's place among those that the row sees
        place = torch.where(node[:, None, :] < 0, p, ctx[:, None, None] + sees.long().cumsum(2).gather(2, pick) - 1)
        total = ctx[:, None] + sees.sum(2)
        seen &= (place < case["sinks"]) | (place >= total[:, :, None] - case["window"])
    seen = seen.repeat_interleave(g, 1)[:, None]  # [B, 1, N * g, S]
    scores = (q @ k).mul_(1 / math.sqrt(HD)).masked_fill_(~seen, float("-inf"))
    top = scores.amax(-1, keepdim=True)
    weight = scores.sub_(top.clamp(min=-3e38)).exp_()
    total = weight.sum(-1, keepdim=True)
    out = (weight @ v) / torch.where(total > 0, total, 1)
    out = out.view(B, kv, N, g, HD).permute(0, 2, 1, 3, 4)[s["seq_of_row"], s["node_of_row"]].reshape(-1, kv * g, HD).to(torch.bfloat16)
    if not case["lse"]:
        return out
    lse = (top + total.log()).view(B, kv, N, g).permute(0, 2, 1, 3)[s["seq_of_row"], s["node_of_row"]].reshape(-1, kv * g)
    return out, lse


def _move_plain(s):
    bs = s["case"]["block"]
    seq, k = (torch.arange(s["path"].shape[1], device=s["path"].device)[None, :] < s["path_len"][:, None]).nonzero(as_tuple=True)
    ctx, table = s["context_len"].long(), s["block_table"].long()
    here, there = ctx[seq] + s["path"][seq, k], ctx[seq] + k
    src, dst = table[seq, here // bs], table[seq, there // bs]
    for c in s["caches"]:
        c[dst, :, there % bs] = c[src, :, here % bs]
    return s["caches"], s["context_len"] + s["path_len"]


def run(s):
    op = s["op"]
    if not own:
        return {"norm": _norm_plain, "store": _store_plain, "window": _attention_plain, "four": _attention_plain, "move": _move_plain}[op](s)
    rc, case = s["rc"], s["case"]
    if op == "norm":
        how = dict(eps=s["eps"], q_weight=s["q_weight"], k_weight=s["k_weight"], q_heads=case["q_heads"],
                   layout=rc.RC_ROPE_HALVES if s["halves"] else rc.RC_ROPE_PAIRS)
        y = rc.head_norm_rope(s["x"], s["positions"], s["table"], **how)
        if "dy" not in s:
            return y
        dx, dq, dk = rc.head_norm_rope_grad(s["dy"], s["x"], s["positions"], s["table"], **how)
        return y, dx, [d for d in (dq, dk) if d is not None]
    if op == "store":
        rc.kv4_store(s["k"], s["v"], s["slots"], s["cache"], s["scales"])
        return rc.kv4_load(s["slots"], s["cache"], s["scales"])
    if op == "move":
        return s["caches"], rc.kv_compact(s["caches"], s["block_table"], s["context_len"], s["row_start"], s["path"], s["path_len"])
    lse = torch.empty(s["rows"], s["q"].shape[1], device=s["q"].device) if case["lse"] else None
    how = dict(tree_mask=s["tree_mask"], lse=lse, workspace=s["workspace"])
    if case["window"]:
        how.update(window=case["window"], sinks=case["sinks"])
    if op == "window":
        out = rc.window_attention(s["q"], s["row_start"], s["context_len"], s["block_table"], s["cache"], **how)
    else:
        out = rc.kv4_attention(s["q"], s["row_start"], s["context_len"], s["block_table"], s["cache"], s["scales"], **how)
    return out if lse is None else (out, lse)


# ------------------------------------------------------------ what it cannot do without


def work(case):
    op = case["op"]
    if op == "norm":
        size = 2 if case["type"] == "bf16" else 4
        heads = case["q_heads"] + case["k_heads"]
        n = case["tokens"] * heads * case["width"]
        once = case["tokens"] * (8 + case["rot"] * size) + 2 * case["width"] * size
        # x in, y out; for the gradients x and dy in, dx out
        return {"bytes": (5 if case["train"] else 2) * n * size + once,
                "flops": (14 if case["train"] else 4) * n + (2 if case["train"] else 1) * 3 * case["tokens"] * heads * case["rot"]}
    if op == "store":
        n = case["tokens"] * case["kv_heads"] * 2 * HD
        # bf16 in, half a byte and the scales out; both read back, bf16 out
        return {"bytes": 4 * n + 2 * (n // 2 + n // GROUP * 2) + 16 * case["tokens"], "flops": 4 * n}
    counts, lens, kv = _node_counts(case), _lengths(case), case["kv_heads"]
    if op == "move":
        # on average three quarters of the longest paths, of which the first rows are in place
        rows = sum(max(0, 3 * min(case["path"], max(1, n // 2)) // 4 - 1) for n in counts)
        row = 2 * HD * 2 if case["cache"] == "bf16" else HD + 8
        return {"bytes": 2 * rows * kv * case["layers"] * row + 8 * len(counts) + 4 * sum(counts), "flops": 0}
    rows, heads = sum(counts), kv * case["group"]
    row = 2 * HD * 2 if op == "window" else HD + 8
    seen = lambda c, m: min(c + m, case["window"] + case["sinks"]) if case["window"] else c + m  # noqa: E731
    keys = sum(min(c + n, seen(c, n) + n) for c, n in zip(lens, counts))
    pairs = sum(n * seen(c, n / 4) for c, n in zip(lens, counts))
    return {"bytes": keys * kv * row + 2 * rows * heads * HD * 2 + (rows * heads * 4 if case["lse"] else 0), "flops": 4 * HD * heads * pairs}


# ------------------------------------------------------------ the definitions in 64 bits


def _exact_norm(s):
    case, f64 = s["case"], torch.float64
    T, rot, nq = case["tokens"], case["rot"], case["q_heads"]
    row = s["table"][s["positions"]].to(f64)
    turn = torch.complex(row[:, : rot // 2], row[:, rot // 2:])[:, None]

    def rotate(x, by):
        if s["halves"]:
            z = torch.complex(x[..., : rot // 2].contiguous(), x[..., rot // 2: rot].contiguous()) * by
            head = torch.cat([z.real, z.imag], -1)
        else:
            z = torch.view_as_complex(x[..., :rot].reshape(T, -1, rot // 2, 2).contiguous()) * by
            head = torch.view_as_real(z).reshape(T, -1, rot)
        return torch.cat([head, x[..., rot:]], -1)

    ys, dxs, dws = [], [], []
    for part, weight in ((slice(0, nq), s["q_weight"]), (slice(nq, nq + case["k_heads"]), s["k_weight"])):
        x = s["x"][:, part].to(f64)
        if x.shape[1] == 0:
            continue
        size = torch.sqrt(x.pow(2).sum(-1, keepdim=True) / case["width"] + s["eps"])
        unit = x / size
        w = 1.0 if weight is None else weight.to(f64)
        ys.append(rotate(unit * w, turn))
        if "dy" in s:
            back = rotate(s["dy"][:, part].to(f64), turn.conj())
            if weight is not None:
                dws.append(torch.einsum("thd,thd->d", back, unit))
            back = back * w
            along = torch.einsum("thd,thd->th", back, x)[..., None] / case["width"]
            dxs.append(back / size - x * along / size ** 3)
    y = torch.cat(ys, 1)
    return (y, torch.cat(dxs, 1), dws) if "dy" in s else y


def _exact_store(s):
    out = []
    for x in (s["k"], s["v"]):
        g = x.to(torch.float64).unflatten(-1, (2, GROUP))
        scale = torch.true_divide(g.abs().amax(-1, keepdim=True), torch.full((1,), 7.0, dtype=torch.float64, device=x.device))
        unit = torch.exp2(torch.floor(torch.log2(scale.clamp(min=2.0 ** -120))) - 3.0)  # four significant bits
        scale = torch.round(scale / unit) * unit
        scale = torch.where(scale < 2.0 ** -100, torch.zeros_like(scale), scale)
        q = torch.where(scale > 0, g / scale, torch.zeros_like(g))
        low = q.abs().floor()
        n = torch.where(q.abs() - low > 0.5, low + 1, low)
        out.append((q.sign() * n * scale).flatten(-2))
    return torch.cat(out, -1)


def _exact_attention(s):
    case, f64 = s["case"], torch.float64
    kv, g, bs = case["kv_heads"], case["group"], case["block"]
    mask, start = s["tree_mask"].cpu(), s["row_start"].tolist()
    outs, lses = [], []
    for b in range(s["seqs"]):
        lo, hi = start[b], start[b + 1]
        ctx, n = int(s["context_len"][b]), hi - lo
        total = ctx + n
        pages = s["block_table"][b, : -(-total // bs)].long()
        rows = s["cache"][pages].permute(0, 2, 1, 3).reshape(len(pages) * bs, kv, -1)[:total]
        if case["op"] == "four":
            scales = s["scales"][pages].permute(0, 2, 1, 3).reshape(-1, kv, 4)[:total].to(f64)
            whole = torch.empty(total, kv, 2 * HD, dtype=f64, device=rows.device)
            whole[..., 0::2], whole[..., 1::2] = (rows % 16).to(f64) - 8, (rows // 16).to(f64) - 8
            rows = (whole.view(total, kv, 4, GROUP) * scales[..., None]).view(total, kv, 2 * HD)
        rows = rows.to(f64)
        see = torch.ones(n, total, dtype=torch.bool)
        for j in range(n):
            see[:, ctx + j] = (mask[lo:hi, j // 64] >> (j % 64)) & 1 == 1
        if case["window"]:
            for i in range(n):
                order = see[i].nonzero().flatten()
                see[i, order[case["sinks"]: max(case["sinks"], len(order) - case["window"])]] = False
        q = s["q"][lo:hi].to(f64).view(n, kv, g, HD)
        for_rows = torch.zeros(n, kv, g, HD, dtype=f64, device=q.device)
        for_sums = torch.zeros(n, kv, g, dtype=f64, device=q.device)
        hidden = ~see.to(q.device)[:, None, :]
        for h in range(kv):
            sc = torch.einsum("ngd,kd->ngk", q[:, h], rows[:, h, :HD]) / 8.0
            sc = sc.masked_fill(hidden, -math.inf)
            for_sums[:, h] = torch.logsumexp(sc, -1)
            for_rows[:, h] = torch.einsum("ngk,kd->ngd", torch.softmax(sc, -1), rows[:, h, HD:])
        outs.append(for_rows.view(n, kv * g, HD))
        lses.append(for_sums.view(n, kv * g))
    out = torch.cat(outs)
    return (out, torch.cat(lses)) if case["lse"] else out


def _exact_move(s):
    caches = [c.clone() for c in s["caches"]]
    bs = s["case"]["block"]
    table, path, lens, ctx = (s[k].tolist() for k in ("block_table", "path", "path_len", "context_len"))
    for b, m in enumerate(lens):
        for k in range(m):
            src, dst = ctx[b] + path[b][k], ctx[b] + k
            for c, old in zip(caches, s["caches"]):
                c[table[b][dst // bs], :, dst % bs] = old[table[b][src // bs], :, src % bs]
    return caches, torch.tensor([c + m for c, m in zip(ctx, lens)], dtype=torch.int32, device=s["path"].device)


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "store": _exact_store, "window": _exact_attention, "four": _exact_attention, "move": _exact_move}[case["op"]](s)
