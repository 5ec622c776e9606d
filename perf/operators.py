"""Cases, plain forms and 64-bit values of the drafted-token operators: tree
attention over the paged cache, rotary positions, and logits adjustment.

`run` computes an operator in elementary torch operations (own = False) or
through the framework's public calls (own = True); both take what `prepare`
makes.  Cache, head and table shapes are those of the context K/V workloads
and of the decode QKV front (8 or 16 KV heads of 64, 64 query heads, pages of
16, tables up to 131072 positions)."""
import math

import torch

own = False

HD = 64  # head width of the paged caches


def listed():
    att = dict(op="attention", kv_heads=8, group=8, block=16, ragged=True, lse=False)
    return [
        # one drafted token over a short context: launch latency counts
        dict(att, name="attn_one_token", seqs=1, nodes=1, ctx=500),
        # one token each for a serving batch of ragged lengths
        dict(att, name="attn_decode_batch", seqs=64, nodes=1, ctx=2049),
        # one token over a long cache, with the log sums for a later merge
        dict(att, name="attn_decode_long", seqs=1, nodes=1, ctx=131071, lse=True),
        # a few small trees of odd sizes
        dict(att, name="attn_tree_small", seqs=3, nodes=13, ctx=1500),
        # the front's largest tree (16 tokens) for a batch
        dict(att, name="attn_tree_batch", seqs=16, nodes=16, ctx=8192, ragged=False),
        # wide trees over long contexts: the largest
        dict(att, name="attn_tree_large", seqs=8, nodes=64, ctx=32768, ragged=False),
        # the store's table of the longest workload, stretched fourfold
        dict(op="table", name="rope_table_long", positions=131072, rot=64, scaling="parts", factor=4.0, type="bf16"),
        # Q and K of one drafted tree straight from a projection's rows
        dict(op="rope", name="rope_tree", tokens=16, heads=72, width=64, rot=64, layout="pairs", type="bf16", train=False),
        # K of a whole context, half the head rotated, with its gradient
        dict(op="rope", name="rope_context_train", tokens=32768, heads=16, width=128, rot=64, layout="halves", type="bf16", train=True),
        # one row before sampling: latency counts
        dict(op="logits", name="logits_one", seqs=1, nodes=1, vocab=32000, history=600, bias=20, type="f32"),
        # small trees over an odd vocabulary and a long history
        dict(op="logits", name="logits_tree_small", seqs=3, nodes=13, vocab=100003, history=9001, bias=300, type="bf16"),
        # every node of a batch of wide trees
        dict(op="logits", name="logits_tree_batch", seqs=16, nodes=64, vocab=131072, history=4096, bias=64, type="f32"),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "rope", "table", "logits", "logits"])
    if op == "attention":
        kv, group = rng.choice([(1, 8), (2, 4), (4, 8), (8, 8), (8, 4), (16, 1), (16, 4), (8, 1), (1, 64), (2, 16)])
        nodes = _spread(rng, 1, 64)
        seqs = _spread(rng, 1, 64)
        # at most the work of the largest listed case, in bytes and in products
        most = min(8 * 32768 * 8 / (seqs * kv), 8 * 32768 * 4096 / (seqs * nodes * kv * group), 131072)
        ctx = _spread(rng, 16, max(17, int(most)))
        return dict(op=op, seqs=seqs, nodes=nodes, ctx=ctx, kv_heads=kv, group=group, block=rng.choice([16, 16, 16, 32, 64, 128]),
                    ragged=rng.random() < 0.7, lse=rng.random() < 0.3)
    if op == "rope":
        heads, width = rng.choice([1, 8, 16, 36, 72]), rng.choice([64, 64, 96, 128])
        rot = rng.choice([32, 64, width])
        tokens = _spread(rng, 1, max(2, 32768 * 16 * 128 // (heads * width * 2)))
        return dict(op=op, tokens=tokens, heads=heads, width=width, rot=rot, layout=rng.choice(["pairs", "halves"]),
                    type=rng.choice(["bf16", "bf16", "f32"]), train=rng.random() < 0.5)
    if op == "table":
        return dict(op=op, positions=_spread(rng, 256, 131072), rot=rng.choice([32, 64, 96, 128]), scaling=rng.choice(["none", "linear", "base", "parts"]),
                    factor=rng.choice([2.0, 4.0, 8.0]), type="bf16")
    vocab = _spread(rng, 1000, 200000)
    seqs, nodes = _spread(rng, 1, 32), _spread(rng, 1, 64)
    nodes = max(1, min(nodes, 1024 * 131072 // (2 * vocab * seqs)))
    return dict(op=op, seqs=seqs, nodes=nodes, vocab=vocab, history=_spread(rng, 1, 32768), bias=rng.choice([0, 1, 50, 300]), type=rng.choice(["f32", "bf16"]))


# ------------------------------------------------------------ what is in hand


def _lengths(case):
    """Context lengths of the sequences, from the case alone."""
    n, ctx = case["seqs"], case["ctx"]
    return [ctx - (b * 5 % n) * ctx // (2 * n) if case["ragged"] else ctx for b in range(n)]


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


def prepare(case, seed):
    dev = torch.device("cuda:0")
    gen = torch.Generator(device=dev).manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    op = case["op"]
    if op == "table":
        # the seed moves the base a little: another model's table
        theta = 10000.0 * (1 + (seed % 1000) / 1000)
        s = dict(op=op, case=case, theta=theta, device=dev)
        if own:
            import rope_chain_gb300 as rc
            s["rc"] = rc
        return s
    if op == "rope":
        T, n, w, rot = case["tokens"], case["heads"], case["width"], case["rot"]
        dt = torch.bfloat16 if case["type"] == "bf16" else torch.float32
        most = 131072
        inv = 10000.0 ** (-2.0 * torch.arange(rot // 2, device=dev, dtype=torch.float64) / rot)
        ang = torch.arange(most, device=dev, dtype=torch.float64)[:, None] * inv
        table = torch.cat([ang.cos(), ang.sin()], 1).to(dt)
        # the heads to rotate lead each row of a wider projection
        rows = torch.randn(T, (n + 8) * w, generator=gen, device=dev).to(dt)
        s = dict(op=op, case=case, x=rows[:, : n * w].view(T, n, w), table=table, halves=case["layout"] == "halves",
                 positions=torch.randint(0, most, (T,), generator=gen, device=dev), rot=rot)
        if case["train"]:
            s["dy"] = torch.randn(T, n, w, generator=gen, device=dev).to(dt)
        if own:
            import rope_chain_gb300 as rc
            s["rc"] = rc
        return s
    counts = _node_counts(case)
    start = torch.tensor([0] + counts).cumsum(0).to(torch.int32)
    mask = _tree(host, counts)
    rows = int(start[-1])
    seq_of_row = torch.repeat_interleave(torch.arange(len(counts)), torch.tensor(counts)).to(dev)
    s = dict(op=op, case=case, row_start=start.to(dev), tree_mask=mask.to(dev), rows=rows, most_nodes=max(counts), seqs=len(counts),
             seq_of_row=seq_of_row, node_of_row=torch.cat([torch.arange(c) for c in counts]).to(dev))
    if op == "attention":
        lens, kv, bs = _lengths(case), case["kv_heads"], case["block"]
        need = [-(-(c + n) // bs) for c, n in zip(lens, counts)]
        width = max(need)
        blocks = sum(need) + 3
        order = torch.randperm(blocks, generator=host).to(torch.int32)
        table = torch.zeros(len(counts), width, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
        s.update(
            context_len=torch.tensor(lens, dtype=torch.int32).to(dev), most_keys=max(c + n for c, n in zip(lens, counts)), block_table=table.to(dev),
            cache=torch.randn(blocks, kv, bs, 2 * HD, generator=gen, device=dev, dtype=torch.bfloat16),
            # Q leads each row of a projection [Q | K | V], as the front writes it
            q=torch.randn(rows, (case["group"] + 2) * kv * HD, generator=gen, device=dev).to(torch.bfloat16)[:, : case["group"] * kv * HD].view(rows, -1, HD))
        if own:
            import rope_chain_gb300 as rc
            s["rc"] = rc
            s["workspace"] = rc.tree_attention_workspace(rows, len(counts), case["group"] * kv, kv, dev)
        return s
    V, hist = case["vocab"], case["history"]
    dt = torch.bfloat16 if case["type"] == "bf16" else torch.float32
    lens = [max(0, hist - b * hist // (2 * len(counts))) for b in range(len(counts))]
    total = sum(lens)
    skew = lambda n: (torch.rand(n, generator=gen, device=dev) ** 4 * V).long().clamp_(max=V - 1).to(torch.int32)  # noqa: E731
    s.update(
        logits=(3 * torch.randn(rows, V, generator=gen, device=dev)).to(dt),
        history=skew(total), history_start=torch.tensor([0] + lens).cumsum(0).to(dev), prompt_len=torch.tensor([n // 2 for n in lens], dtype=torch.int32, device=dev),
        draft_tokens=skew(rows),
        repetition=1 + torch.rand(len(counts), generator=gen, device=dev), frequency=torch.rand(len(counts), generator=gen, device=dev),
        presence=torch.rand(len(counts), generator=gen, device=dev),
        allowed=torch.randint(-2 ** 31, 2 ** 31, (rows, -(-V // 32)), generator=gen, device=dev).to(torch.int32))
    if case["bias"]:
        per = min(case["bias"], V)
        tok = torch.stack([torch.randperm(V, generator=gen, device=dev)[:per] for _ in counts])
        s.update(bias_start=(torch.arange(len(counts) + 1) * per).to(torch.int32).to(dev), bias_tokens=tok.reshape(-1).to(torch.int32),
                 bias_values=2 * torch.randn(per * len(counts), generator=gen, device=dev))
    if own:
        import rope_chain_gb300 as rc
        s["rc"] = rc
    return s


# ------------------------------------------------------------ one pass


def _frequencies(case, theta, like):
    """Angular frequencies of a table [rot / 2], scaled."""
    rot, f = case["rot"], case["factor"]
    j = torch.arange(rot // 2, **like)
    if case["scaling"] == "base":
        theta = theta * f ** (rot / (rot - 2))
    inv = theta ** (-2.0 * j / rot)
    if case["scaling"] == "linear":
        inv = inv / f
    if case["scaling"] == "parts":
        turn = lambda beta: rot * math.log(_original(case) / (beta * 2 * math.pi)) / (2 * math.log(theta))  # noqa: E731
        lo, hi = max(math.floor(turn(32.0)), 0), min(math.ceil(turn(1.0)), rot - 1)
        ramp = ((j - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        inv = inv * (1 - ramp) + inv / f * ramp
    return inv


def _original(case):
    return max(64, int(case["positions"] / case["factor"]))


def _attention_factor(case):
    return 0.1 * math.log(case["factor"]) + 1.0 if case["scaling"] == "parts" else 1.0


def _table_plain(s):
    case = s["case"]
    like = dict(device=s["device"], dtype=torch.float32)
    ang = torch.arange(case["positions"], **like)[:, None] * _frequencies(case, s["theta"], like)
    return (torch.cat([ang.cos(), ang.sin()], 1) * _attention_factor(case)).to(torch.bfloat16)


def _rotate_plain(x, table, positions, rot, halves, sign):
    half = rot // 2
    cs = table[positions].float()
    c, n = cs[:, None, :half], sign * cs[:, None, half:]
    y = x.float().clone()
    a, b = (slice(0, half), slice(half, rot)) if halves else (slice(0, rot, 2), slice(1, rot, 2))
    u, v = y[..., a].clone(), y[..., b].clone()
    y[..., a] = u * c - v * n
    y[..., b] = v * c + u * n
    return y.to(x.dtype)


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
    blocks = s["block_table"].long()[:, (p // bs)]
    rows = s["cache"][blocks, :, (p % bs)[None, :]].float()  # [B, S, kv, 128]
    k, v = rows[..., :HD].permute(0, 2, 3, 1), rows[..., HD:].permute(0, 2, 1, 3)
    q = torch.zeros(B, N, kv, g, HD, device=dev)
    q[s["seq_of_row"], s["node_of_row"]] = s["q"].float().view(-1, kv, g, HD)
    q = q.permute(0, 2, 1, 3, 4).reshape(B, kv, N * g, HD)
    ctx = s["context_len"].long()
    node = p[None, :] - ctx[:, None]  # [B, S]
    sees = torch.zeros(B, N, N, dtype=torch.bool, device=dev)
    sees[s["seq_of_row"], s["node_of_row"]] = _sees(s)
    inside = (node >= 0) & (node < N)
    tree = sees.gather(2, node.clamp(0, N - 1)[:, None, :].expand(B, N, S)) & inside[:, None, :]
    seen = ((node < 0)[:, None, :] | tree).repeat_interleave(g, 1)[:, None]  # [B, 1, N * g, S]
    scores = (q @ k).mul_(1 / math.sqrt(HD)).masked_fill_(~seen, float("-inf"))
    top = scores.amax(-1, keepdim=True)
    weight = (scores - top.clamp(min=-3e38)).exp_()
    total = weight.sum(-1, keepdim=True)
    out = (weight @ v) / torch.where(total > 0, total, 1)
    out = out.view(B, kv, N, g, HD).permute(0, 2, 1, 3, 4)[s["seq_of_row"], s["node_of_row"]].reshape(-1, kv * g, HD).to(torch.bfloat16)
    if not case["lse"]:
        return out
    lse = (top + total.log()).view(B, kv, N, g).permute(0, 2, 1, 3)[s["seq_of_row"], s["node_of_row"]].reshape(-1, kv * g)
    return out, lse


def _logits_plain(s):
    case = s["case"]
    B, V = s["seqs"], case["vocab"]
    dev = s["logits"].device
    start = s["history_start"]
    place = torch.arange(s["history"].numel(), device=dev)
    seq = torch.bucketize(place, start[1:], right=True)
    prompt = place - start[seq] < s["prompt_len"][seq]
    key = seq * V + s["history"].long()
    made = torch.zeros(B * V, device=dev).index_add_(0, key, (~prompt).float()).view(B, V)
    said = torch.zeros(B * V, device=dev).index_add_(0, key, prompt.float()).view(B, V)
    r = s["seq_of_row"]
    count = made[r]
    sees = _sees(s)
    first = s["row_start"].long()[r]
    j = torch.arange(s["most_nodes"], device=dev)
    other = (first[:, None] + j[None, :]).clamp(max=s["rows"] - 1)
    count.scatter_add_(1, s["draft_tokens"].long()[other], sees.float())
    x = s["logits"].float()
    rep = s["repetition"][r][:, None]
    x = torch.where((count > 0) | (said[r] > 0), torch.where(x > 0, x / rep, x * rep), x)
    x = x - s["frequency"][r][:, None] * count - s["presence"][r][:, None] * (count > 0)
    if "bias_start" in s:
        per = case["bias"] if case["bias"] < V else V
        bias = torch.zeros(B, V, device=dev).scatter_(1, s["bias_tokens"].long().view(B, per), s["bias_values"].view(B, per))
        x = x + bias[r]
    t = torch.arange(V, device=dev)
    allowed = (s["allowed"][:, t // 32] >> (t % 32)) & 1 == 1
    return x.masked_fill_(~allowed, float("-inf")).to(s["logits"].dtype)


def run(s):
    op = s["op"]
    if not own:
        if op == "table":
            return _table_plain(s)
        if op == "rope":
            y = _rotate_plain(s["x"], s["table"], s["positions"], s["rot"], s["halves"], 1)
            return (y, _rotate_plain(s["dy"], s["table"], s["positions"], s["rot"], s["halves"], -1)) if "dy" in s else y
        return _attention_plain(s) if op == "attention" else _logits_plain(s)
    rc, case = s["rc"], s["case"]
    if op == "table":
        return rc.rope_table(case["positions"], case["rot"], theta=s["theta"], scaling=case["scaling"], factor=case["factor"],
                             original_max_position=_original(case), attention_factor=_attention_factor(case), dtype=torch.bfloat16, device=s["device"])
    if op == "rope":
        layout = rc.RC_ROPE_HALVES if s["halves"] else rc.RC_ROPE_PAIRS
        y = rc.rope_apply(s["x"], s["positions"], s["table"], layout=layout)
        return (y, rc.rope_apply(s["dy"], s["positions"], s["table"], layout=layout, inverse=True)) if "dy" in s else y
    if op == "attention":
        lse = torch.empty(s["rows"], s["q"].shape[1], device=s["q"].device) if case["lse"] else None
        out = rc.tree_attention(s["q"], s["row_start"], s["context_len"], s["block_table"], s["cache"], tree_mask=s["tree_mask"], lse=lse,
                                workspace=s["workspace"])
        return out if lse is None else (out, lse)
    return rc.logits_adjust(s["logits"], s["row_start"], history=s["history"], history_start=s["history_start"], prompt_len=s["prompt_len"],
                            draft_tokens=s["draft_tokens"], tree_mask=s["tree_mask"], repetition=s["repetition"], frequency=s["frequency"],
                            presence=s["presence"], bias_start=s.get("bias_start"), bias_tokens=s.get("bias_tokens"), bias_values=s.get("bias_values"),
                            allowed=s["allowed"])


# ------------------------------------------------------------ what it cannot do without


def work(case):
    op = case["op"]
    if op == "table":
        n = case["positions"] * case["rot"]
        return {"bytes": 2 * n, "flops": 2 * n}
    if op == "rope":
        size = 2 if case["type"] == "bf16" else 4
        n = case["tokens"] * case["heads"] * case["width"]
        passes = 2 if case["train"] else 1
        # x in, out; positions and their table rows once
        return {"bytes": passes * 2 * n * size + case["tokens"] * (8 + case["rot"] * size), "flops": passes * 3 * case["tokens"] * case["heads"] * case["rot"]}
    counts = _node_counts(case)
    rows = sum(counts)
    if op == "attention":
        lens = _lengths(case)
        heads = case["kv_heads"] * case["group"]
        keys = sum(c + n for c, n in zip(lens, counts))
        seen = sum(n * (c + n / 4) for c, n in zip(lens, counts))
        return {"bytes": keys * case["kv_heads"] * 2 * HD * 2 + 2 * rows * heads * HD * 2 + (rows * heads * 4 if case["lse"] else 0),
                "flops": 4 * HD * heads * seen}
    size = 2 if case["type"] == "bf16" else 4
    hist = sum(max(0, case["history"] - b * case["history"] // (2 * case["seqs"])) for b in range(case["seqs"]))
    return {"bytes": 2 * rows * case["vocab"] * size + rows * (-(-case["vocab"] // 32)) * 4 + hist * 4, "flops": 4 * rows * case["vocab"]}


# ------------------------------------------------------------ the definitions in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    op, f64 = case["op"], torch.float64
    if op == "table":
        rot, f, theta = case["rot"], case["factor"], s["theta"]
        if case["scaling"] == "base":
            theta *= f ** (rot / (rot - 2.0))
        inv = [theta ** (-2.0 * j / rot) for j in range(rot // 2)]
        gain = 1.0
        if case["scaling"] == "linear":
            inv = [x / f for x in inv]
        elif case["scaling"] == "parts":
            gain = 0.1 * math.log(f) + 1.0
            orig = max(64, int(case["positions"] / f))
            where = [rot * math.log(orig / (beta * 2 * math.pi)) / (2 * math.log(theta)) for beta in (32.0, 1.0)]
            lo, hi = max(math.floor(where[0]), 0), min(math.ceil(where[1]), rot - 1)
            mix = [min(1.0, max(0.0, (j - lo) / max(hi - lo, 1e-3))) for j in range(rot // 2)]
            inv = [x * (1 - m) + x / f * m for x, m in zip(inv, mix)]
        turns = torch.outer(torch.arange(case["positions"], dtype=f64, device=s["device"]), torch.tensor(inv, dtype=f64, device=s["device"]))
        return torch.cat([gain * torch.cos(turns), gain * torch.sin(turns)], 1)
    if op == "rope":
        T, n, w, rot = case["tokens"], case["heads"], case["width"], case["rot"]
        row = s["table"][s["positions"]].to(f64)
        turn = torch.complex(row[:, : rot // 2], row[:, rot // 2:])[:, None]

        def rotate(x, by):
            x = x.to(f64)
            if s["halves"]:
                z = torch.complex(x[..., : rot // 2].contiguous(), x[..., rot // 2: rot].contiguous()) * by
                head = torch.cat([z.real, z.imag], -1)
            else:
                z = torch.view_as_complex(x[..., :rot].reshape(T, n, rot // 2, 2).contiguous()) * by
                head = torch.view_as_real(z).reshape(T, n, rot)
            return torch.cat([head, x[..., rot:]], -1)

        y = rotate(s["x"], turn)
        return (y, rotate(s["dy"], turn.conj())) if "dy" in s else y
    mask, start = s["tree_mask"].cpu(), s["row_start"].tolist()
    if op == "attention":
        kv, g, bs = case["kv_heads"], case["group"], case["block"]
        outs, lses = [], []
        for b in range(s["seqs"]):
            lo, hi = start[b], start[b + 1]
            ctx, n = int(s["context_len"][b]), hi - lo
            total = ctx + n
            pages = s["block_table"][b, : -(-total // bs)].long()
            rows = s["cache"][pages].permute(0, 2, 1, 3).reshape(-1, kv, 2 * HD)[:total].to(f64)
            see = torch.ones(n, total, dtype=torch.bool)
            for j in range(n):
                see[:, ctx + j] = (mask[lo:hi, j // 64] >> (j % 64)) & 1 == 1
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
    V = case["vocab"]
    res = torch.empty(s["rows"], V, dtype=f64, device=s["logits"].device)
    hs, pl = s["history_start"].tolist(), s["prompt_len"].tolist()
    bits = torch.arange(32, device=res.device)
    for b in range(s["seqs"]):
        lo, hi = start[b], start[b + 1]
        toks = s["history"][hs[b]:hs[b + 1]].long()
        prompt = torch.bincount(toks[: pl[b]], minlength=V)
        base = torch.bincount(toks[pl[b]:], minlength=V)
        bias = torch.zeros(V, dtype=f64, device=res.device)
        if "bias_start" in s:
            x0, x1 = s["bias_start"][b], s["bias_start"][b + 1]
            bias[s["bias_tokens"][x0:x1].long()] = s["bias_values"][x0:x1].to(f64)
        rep, freq, pres = (float(s[k][b]) for k in ("repetition", "frequency", "presence"))
        drafted = s["draft_tokens"][lo:hi].long()
        for i in range(lo, hi):
            on = torch.tensor([(int(mask[i, j // 64]) >> (j % 64)) & 1 == 1 for j in range(hi - lo)], device=res.device)
            g = base + torch.bincount(drafted[on], minlength=V)
            x = s["logits"][i].to(f64)
            x = torch.where((g > 0) | (prompt > 0), torch.where(x > 0, x / rep, x * rep), x)
            x = x - freq * g - pres * (g > 0) + bias
            ok = ((s["allowed"][i][:, None] >> bits) & 1 == 1).reshape(-1)[:V]
            res[i] = torch.where(ok, x, torch.full_like(x, -math.inf))
    return res
