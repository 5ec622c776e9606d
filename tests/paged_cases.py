"""Operands of attention over paged caches, in bf16 or in 4 bits, with and without a
window, and the formula in 64 bits.

Tolerance, per output with A = sum_p w_p |v_p| / sum_p w_p: the output's rounding
2^-8 |ref|, the weights' rounding 2^-8 A, and 2^-12 A for FP32 scores, exponentials
and sums (scores of 64 products of unit-variance values: 64 * 2^-24 * sum|q k| *
scale < 2^-14, the exponential's 2^-22; what a cache in 4 bits holds is exact).  Log
sums: 64 * 2^-24 times the largest scale * sum|q k|, plus 2^-20 (1 + |lse|)."""
import numpy as np
import torch

import rope_chain_gb300 as rc

DEV = torch.device("cuda:0")
BF, I32 = torch.bfloat16, torch.int32


def random_trees(rng, counts, words, empty=0.0):
    """Ancestor-or-self bits of random trees, bool per sequence, and packed."""
    rows, bits = [], []
    for n in counts:
        m = np.zeros((n, n), dtype=bool)
        for i in range(n):
            if i and rng.random() < 0.9:
                m[i] = m[rng.integers(max(0, i - 4), i)]
            m[i, i] = True
        if empty:
            m[rng.random(n) < empty] = False
        m[:, 64 * words:] = False
        w = np.zeros((n, words), dtype=np.uint64)
        for j in range(min(n, 64 * words)):
            w[:, j // 64] |= m[:, j].astype(np.uint64) << np.uint64(j % 64)
        rows.append(m)
        bits.append(w)
    packed = np.concatenate(bits) if bits else np.zeros((0, words), dtype=np.uint64)
    return rows, torch.from_numpy(packed.view(np.int64)).to(DEV)


class Case:
    """Rows of the cache that are not in use hold NaN (in 4 bits: any bytes, and scales of NaN)."""

    def __init__(self, seed, counts, ctx, H, G, bs, *, four=False, window=None, sinks=0, mask="tree", words=None, spare=3, sigma=1.0,
                 empty=0.0, pad_rows=0):
        rng = np.random.default_rng(seed)
        gen = torch.Generator(device=DEV).manual_seed(seed)
        self.counts, self.ctx, self.H, self.G, self.bs = counts, ctx, H, G, bs
        self.four, self.window, self.sinks = four, window, sinks
        need = [-(-(c + n) // bs) for c, n in zip(ctx, counts)]
        self.nb = nb = sum(need) + spare
        order = rng.permutation(nb)
        table = np.zeros((len(counts), max(need + [1])), dtype=np.int32)
        if four:
            self.cache = torch.randint(0, 256, (nb, H, bs, 64), generator=gen, device=DEV, dtype=torch.uint8)
            self.scales = torch.full((nb, H, bs, 4), float("nan"), dtype=BF, device=DEV)
        else:
            self.cache = torch.full((nb, H, bs, 128), float("nan"), dtype=BF, device=DEV)
        self.kv, at = [], 0
        for b, (c, n) in enumerate(zip(ctx, counts)):
            pages = order[at:at + need[b]]
            at += need[b]
            table[b, :need[b]] = pages
            kv = torch.randn(c + n, H, 128, generator=gen, device=DEV).mul_(sigma).to(BF)
            p = torch.arange(c + n, device=DEV)
            blk = torch.from_numpy(pages.astype(np.int64)).to(DEV)[p // bs]
            if four:
                slots = blk * bs + p % bs
                rc.kv4_store(kv[..., :64], kv[..., 64:], slots, self.cache, self.scales)
                kv = rc.kv4_load(slots, self.cache, self.scales)
            else:
                self.cache[blk, :, p % bs] = kv
            self.kv.append(kv)
        self.table = torch.from_numpy(table).to(DEV)
        self.rows = sum(counts) + pad_rows
        self.q = torch.randn(self.rows, H * G * 64 + 64, generator=gen, device=DEV).mul_(sigma).to(BF)[:, :H * G * 64].view(
            self.rows, H * G, 64)
        self.row_start = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=I32, device=DEV)
        self.context = torch.tensor(ctx, dtype=I32, device=DEV)
        if mask == "tree":
            words = words or max(1, -(-max(counts + [1]) // 64))
            self.sees, self.mask = random_trees(rng, counts, words, empty)
            if pad_rows:
                self.mask = torch.cat([self.mask, torch.zeros(pad_rows, words, dtype=torch.int64, device=DEV)])
        else:
            self.sees, self.mask = [np.tril(np.ones((n, n), dtype=bool)) for n in counts], None
        # keys that are not there, bool per sequence
        self.gone = [np.zeros(c + n, dtype=bool) for c, n in zip(ctx, counts)]

    def visible(self, b):
        """bool [nodes, keys]: which keys count for each row; keys that are gone keep their place."""
        c, n = self.ctx[b], self.counts[b]
        see = np.ones((n, c + n), dtype=bool)
        see[:, c:] = self.sees[b]
        if self.window is not None:
            for i in range(n):
                order = np.flatnonzero(see[i])
                see[i, order[self.sinks:max(self.sinks, len(order) - self.window)]] = False
        see[:, self.gone[b]] = False
        return torch.from_numpy(see).to(DEV)

    def ref(self, scale=0.125):
        """(out, lse, tolerance of out, of lse) in 64 bits."""
        outs, lses, tol, ltol = [], [], [], []
        r = 0
        for b, n in enumerate(self.counts):
            kv, keys = self.kv[b].double(), self.ctx[b] + n
            k, v = torch.nan_to_num(kv[..., :64]), torch.nan_to_num(kv[..., 64:])
            q = self.q[r:r + n].double().view(n, self.H, self.G, 64)
            r += n
            hide = ~self.visible(b)[:, None, None]
            t = torch.einsum("nhgd,phd->nhgp", q, k) * scale
            size = torch.einsum("nhgd,phd->nhgp", q.abs(), k.abs()) * scale
            t = t.masked_fill(hide, -float("inf"))
            lse = torch.logsumexp(t, -1) if keys else torch.full(t.shape[:-1], -float("inf"), device=DEV).double()
            w = torch.nan_to_num(torch.exp(t - torch.nan_to_num(lse, neginf=0.0)[..., None]), nan=0.0)
            out = torch.einsum("nhgp,phd->nhgd", w, v)
            mag = torch.einsum("nhgp,phd->nhgd", w, v.abs())
            outs.append(out.reshape(n, self.H * self.G, 64))
            tol.append((2.0 ** -8 * out.abs() + (2.0 ** -8 + 2.0 ** -12) * mag).reshape(n, self.H * self.G, 64))
            lses.append(lse.reshape(n, self.H * self.G))
            big = size.masked_fill(hide, 0).amax(-1) if keys else torch.zeros_like(lse)
            ltol.append((64 * 2.0 ** -24 * big + 2.0 ** -20 * (1 + torch.nan_to_num(lse, neginf=0.0).abs())).reshape(n, self.H * self.G))
        return torch.cat(outs), torch.cat(lses), torch.cat(tol) + 2.0 ** -30, torch.cat(ltol)

    def workspace(self):
        make = rc.kv4_attention_workspace if self.four else rc.tree_attention_workspace
        return make(self.rows, len(self.counts), self.H * self.G, self.H, DEV)

    def call(self, **kw):
        args = [self.q, self.row_start, self.context, self.table, self.cache] + ([self.scales] if self.four else [])
        if self.window is not None:
            kw.update(window=self.window, sinks=self.sinks)
        attention = rc.kv4_attention if self.four else rc.tree_attention if self.window is None else rc.window_attention
        return attention(*args, tree_mask=self.mask, **kw)

    def run(self, ws=True, **kw):
        lse = torch.full((self.rows, self.H * self.G), 7.0, device=DEV)
        err = torch.zeros(1, dtype=I32, device=DEV)
        out = self.call(lse=lse, err=err, workspace=self.workspace() if ws else None, **kw)
        torch.cuda.synchronize()
        return out, lse, int(err.item())

    def check(self, out, lse, scale=0.125):
        ref, rlse, tol, ltol = self.ref(scale)
        n = ref.shape[0]
        bad = ~((out[:n].double() - ref).abs() <= tol)
        assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()} outside tolerance, first {bad.nonzero()[0].tolist()}"
        got = lse[:n].double()
        same = (got == rlse) | ((got - rlse).abs() <= ltol)
        assert bool(same.all()), f"{int((~same).sum())} log sums outside tolerance"

    def block_out(self, b, page, value):
        """Entry `page` of sequence b's table becomes `value`, its keys are gone."""
        self.table[b, page] = value
        self.gone[b][page * self.bs:(page + 1) * self.bs] = True

    def key_at(self, b, p):
        """(block, offset) of a sequence's key."""
        return int(self.table[b, p // self.bs]), p % self.bs
