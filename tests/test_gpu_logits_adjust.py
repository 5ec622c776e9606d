"""rc_logits_adjust against the formula in 64 bits.  Tolerance: each of the
five FP32 steps rounds once, 2^-24 of the largest magnitude it meets
(|x| after the repetition, freq * g, pres, bias), plus the type's rounding."""
import numpy as np
import pytest
import torch

import rope_chain_gb300 as rc
from tests.test_gpu_tree_attention import random_mask

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    from rope_chain_gb300 import _build
    _build.build()


def make(seed, counts, V, hist, *, parts="hrfpdmba", bias=5, dtype=F32, skew=4, chain=False):
    """Operands; `parts` picks: h history, r f p penalties, d drafted, m tree mask, b bias, a allowed."""
    rng = np.random.default_rng(seed)
    B, rows = len(counts), sum(counts)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    token = lambda n: np.minimum((rng.random(n) ** skew * V).astype(np.int32), V - 1)
    kw = {}
    if "h" in parts:
        lens = [int(rng.integers(0, hist + 1)) for _ in counts]
        kw.update(history=dev(token(sum(lens))), history_start=dev(np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)),
                  prompt_len=dev(np.array([n // 3 for n in lens], dtype=np.int32)))
    for c, name in (("r", "repetition"), ("f", "frequency"), ("p", "presence")):
        if c in parts:
            kw[name] = dev((rng.random(B) + (1 if c == "r" else -0.3)).astype(np.float32))
    if "d" in parts:
        kw["draft_tokens"] = dev(token(rows))
    if "m" in parts:
        sees, kw["tree_mask"] = random_mask(rng, counts, max(1, -(-max(counts) // 64)))
    else:
        sees = [np.tril(np.ones((n, n), dtype=bool)) for n in counts]
    if "b" in parts:
        kw.update(bias_start=dev((np.arange(B + 1) * bias).astype(np.int32)), bias_tokens=dev(token(B * bias)),
                  bias_values=dev(rng.standard_normal(B * bias).astype(np.float32)))
    if "a" in parts:
        kw["allowed"] = dev(rng.integers(-2 ** 31, 2 ** 31, size=(rows, -(-V // 32) + 1)).astype(np.int32))
    logits = dev((3 * rng.standard_normal((rows, V))).astype(np.float32)).to(dtype)
    start = dev(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32))
    return logits, start, kw, sees


def reference(logits, start, kw, sees):
    rows, V = logits.shape
    x = logits.double().cpu().numpy()
    out, tol = np.empty_like(x), np.empty_like(x)
    host = {k: v.cpu().numpy() for k, v in kw.items()}
    st = start.cpu().numpy()
    one = lambda name, b, default: float(host[name][b]) if name in host else default
    for b in range(len(st) - 1):
        made, said, bias = np.zeros(V, np.int64), np.zeros(V, bool), np.zeros(V)
        if "history" in host:
            h = host["history"][host["history_start"][b]:host["history_start"][b + 1]]
            p = host["prompt_len"][b] if "prompt_len" in host else 0
            said[h[:p]] = True
            np.add.at(made, h[p:], 1)
        if "bias_start" in host:
            for e in range(host["bias_start"][b], host["bias_start"][b + 1]):
                bias[host["bias_tokens"][e]] = host["bias_values"][e]
        rep, freq, pres = one("repetition", b, 1.0), one("frequency", b, 0.0), one("presence", b, 0.0)
        for i in range(st[b], st[b + 1]):
            g = made.copy()
            if "draft_tokens" in host:
                np.add.at(g, host["draft_tokens"][st[b]:st[b + 1]][sees[b][i - st[b]]], 1)
            y = x[i]
            y = np.where((g > 0) | said, np.where(y > 0, y / rep, y * rep), y)
            big = np.abs(y) + abs(freq) * g + abs(pres) + np.abs(bias)
            y = y - freq * g - pres * (g > 0) + bias
            if "allowed" in host:
                t = np.arange(V)
                y = np.where((host["allowed"][i][t // 32] >> (t % 32)) & 1, y, -np.inf)
            out[i] = y
            tol[i] = 5 * 2.0 ** -24 * big
    fin = np.where(np.isfinite(out), np.abs(out), 0)
    tol += (2.0 ** -8 if logits.dtype == BF else 0) * fin * (1 + 2.0 ** -7)
    return out, tol


def check(logits, start, kw, sees, got):
    ref, tol = reference(logits, start, kw, sees)
    g = got.double().cpu().numpy()
    assert np.array_equal(np.isneginf(ref), np.isneginf(g))
    m = ~np.isneginf(ref)
    assert (np.abs(g - ref)[m] <= tol[m]).all()


CASES = [([1], 1, 4), ([1], 31, 100), ([1], 32000, 600), ([3, 1], 100003, 3000), ([13, 12], 4097, 50), ([64, 63, 1], 1027, 2000),
         ([2, 0, 3], 129, 40), ([130], 260, 300), ([5] * 20, 5000, 64), ([9, 8], 70001, 0)]


@pytest.mark.parametrize("counts,V,hist", CASES)
@pytest.mark.parametrize("dtype", [F32, BF])
def test_against_formula(counts, V, hist, dtype):
    logits, start, kw, sees = make(V + len(counts), counts, V, hist, dtype=dtype)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = rc.logits_adjust(logits, start, err=err, **kw)
    assert int(err.item()) == 0
    check(logits, start, kw, sees, got)


@pytest.mark.parametrize("parts", ["", "h", "hr", "f", "hfp", "d", "dfp", "dmr", "b", "a", "hdmrfp"])
def test_parts(parts):
    logits, start, kw, sees = make(11, [7, 6], 3001, 500, parts=parts)
    check(logits, start, kw, sees, rc.logits_adjust(logits, start, **kw))


# two and four accesses a row and thread: many sequences over large vocabularies, rows on and off 16-byte boundaries
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("counts,V,hist", [([3] * 40, 40000, 3000), ([3] * 40, 40001, 3000), ([1] * 130, 40000, 200), ([1, 2] * 30, 40003, 20)])
def test_wide_tiles(counts, V, hist, dtype):
    logits, start, kw, sees = make(V + len(counts), counts, V, hist, dtype=dtype)
    check(logits, start, kw, sees, rc.logits_adjust(logits, start, **kw))


def test_empty_tensors_and_masks_without_words():
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)
    empty = torch.zeros(0, dtype=torch.int32, device=DEV)
    assert rc.logits_adjust(torch.zeros(0, 9, device=DEV), i32(0, 0), draft_tokens=empty).shape == (0, 9)
    x = torch.arange(9.0, device=DEV)[None]
    got = rc.logits_adjust(x, i32(0, 1), history=empty, history_start=torch.zeros(2, dtype=torch.int64, device=DEV),
                           bias_start=i32(0, 0), bias_tokens=empty, bias_values=empty.float(),
                           repetition=torch.full((1,), 2.0, device=DEV))
    assert torch.equal(got, x)
    with pytest.raises(ValueError, match="word"):
        rc.logits_adjust(x, i32(0, 1), draft_tokens=i32(3), tree_mask=torch.zeros(1, 0, dtype=torch.int64, device=DEV))


def test_many_drafted_tokens_in_one_tile():
    """More nodes than a tile lists, all of few tokens."""
    logits, start, kw, sees = make(12, [700], 40, 30)
    check(logits, start, kw, sees, rc.logits_adjust(logits, start, **kw))


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("lead,row", [(0, 1500), (1, 1501), (5, 1507), (8, 1504)])
def test_in_place_views_and_slack(dtype, lead, row):
    logits, start, kw, sees = make(5, [4, 5], 1400, 300, dtype=dtype)
    whole = torch.full((9, row), 9.0, dtype=dtype, device=DEV)
    view = whole.as_strided((9, 1400), (row, 1), lead)
    view.copy_(logits)
    other = torch.full((9, 1411), 9.0, dtype=dtype, device=DEV)[:, 2:1402]     # another offset and stride
    check(logits, start, kw, sees, rc.logits_adjust(view, start, out=other, **kw))
    check(logits, start, kw, sees, rc.logits_adjust(view, start, out=view, **kw))
    keep = torch.ones(9, row, dtype=torch.bool, device=DEV).as_strided((9, 1400), (row, 1), lead).logical_not_()
    flat = torch.ones(9 * row, dtype=torch.bool, device=DEV)
    flat.as_strided((9, 1400), (row, 1), lead).fill_(False)
    assert bool((whole.reshape(-1)[flat] == 9).all())


def test_tokens_outside_the_vocabulary_count_and_do_nothing():
    logits, start, kw, sees = make(6, [4], 50, 40)
    bad = {k: v.clone() for k, v in kw.items()}
    bad["history"] = torch.cat([kw["history"], torch.tensor([-1, 50, 2 ** 31 - 1], dtype=torch.int32, device=DEV)])
    bad["history_start"][-1] += 3
    bad["bias_tokens"] = torch.cat([kw["bias_tokens"], torch.tensor([77], dtype=torch.int32, device=DEV)])
    bad["bias_values"] = torch.cat([kw["bias_values"], torch.ones(1, device=DEV)])
    bad["bias_start"][-1] += 1
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = rc.logits_adjust(logits, start, err=err, **bad)
    assert int(err.item()) == 4
    check(logits, start, kw, sees, got)


def test_infinities_nan_and_nothing_allowed():
    logits, start, kw, sees = make(7, [3], 600, 200)
    logits[0, 5], logits[0, 6], logits[1, 7] = float("inf"), -float("inf"), float("nan")
    kw["allowed"][0, 0] = -1
    kw["allowed"][1, 0] = -1
    kw["allowed"][2] = 0
    got = rc.logits_adjust(logits, start, **kw)
    assert float(got[0, 5]) == float("inf") and float(got[0, 6]) == -float("inf") and bool(got[1, 7].isnan())
    assert bool((got[2] == -float("inf")).all())


def test_rows_without_a_sequence_and_stream():
    logits, start, kw, sees = make(8, [3, 4], 999, 100, parts="hrfpdmb")
    more = torch.cat([logits, logits[:2]])
    kw2 = dict(kw, draft_tokens=torch.cat([kw["draft_tokens"], kw["draft_tokens"][:2]]),
               tree_mask=torch.cat([kw["tree_mask"], kw["tree_mask"][:2]]))
    out = torch.full_like(more, 4.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    rc.logits_adjust(more, start, out=out, stream=side, **kw2)
    torch.cuda.synchronize()
    check(logits, start, kw, sees, out[:7])
    assert bool((out[7:] == 4).all())


@pytest.mark.parametrize("dtype", [F32, BF])
def test_infinite_penalties_touch_what_was_generated_only(dtype):
    """A frequency or presence of infinity forbids what was generated; what the prompt, a bias or another node of
    the tree names, but the row's own past does not (g = 0), has no penalty to multiply."""
    logits, start, kw, sees = make(21, [6, 5], 900, 200, dtype=dtype, parts="hrdmb")
    plain = rc.logits_adjust(logits, start, **kw)
    ref, tol = reference(logits, start, kw, sees)
    host = {k: v.cpu().numpy() for k, v in kw.items()}
    made = np.zeros(ref.shape, bool)
    for b in range(2):
        h = host["history"][host["history_start"][b]:host["history_start"][b + 1]][host["prompt_len"][b]:]
        for i in range(*start.cpu().numpy()[b:b + 2]):
            made[i, h] = True
            r0 = int(start[b])
            made[i, host["draft_tokens"][r0:int(start[b + 1])][sees[b][i - r0]]] = True
    assert made.any() and not made.all()
    for name in ("frequency", "presence"):
        got = rc.logits_adjust(logits, start, **kw, **{name: torch.full((2,), float("inf"), device=DEV)}).double().cpu().numpy()
        assert np.isneginf(got[made]).all(), name
        assert np.array_equal(got[~made], plain.double().cpu().numpy()[~made]), name


@pytest.mark.parametrize("n", [63, 64, 65])
@pytest.mark.parametrize("V,skew", [(40, 1), (40, 30), (9000, 1)])
def test_trees_as_large_as_the_listed_ones(n, V, skew):
    """64 nodes is the largest tree whose tokens are listed; one more is walked node by node."""
    logits, start, kw, sees = make(n, [n, 2, n], V, 30, skew=skew)
    check(logits, start, kw, sees, rc.logits_adjust(logits, start, **kw))
