"""What a call writes into a tensor that was there before shows as one of torch's
in-place operations does: a backward pass that has saved the tensor raises instead of
taking what was written over it."""
import pytest
import torch

import rope_chain_gb300 as rc
from tests import paged_cases

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, F32, I32, I64 = torch.bfloat16, torch.float32, torch.int32, torch.int64


@pytest.fixture(scope="module", autouse=True)
def built():
    from rope_chain_gb300 import _build
    _build.build()


def rows(*shape, dtype=BF):
    return torch.randn(*shape, device=DEV).to(dtype)


def rope_table():
    out = rows(32, 64)
    return [out], lambda: rc.rope_table(32, 64, out=out)


def norm_operands():
    return rows(5, 8, 64), torch.arange(5, device=DEV), rc.rope_table(16, 64, device=DEV)


def rope_apply():
    x, pos, table = norm_operands()
    return [x], lambda: rc.rope_apply(x, pos, table, out=x)


def head_norm_rope():
    x, pos, table = norm_operands()
    return [x], lambda: rc.head_norm_rope(x, pos, table, eps=1e-6, out=x)


def head_norm_rope_grad():
    x, pos, table = norm_operands()
    dy = rows(5, 8, 64)
    return [dy], lambda: rc.head_norm_rope_grad(dy, x, pos, table, eps=1e-6, out=dy)


def attention(**kw):
    def make():
        c = paged_cases.Case(3, [3, 1], [40, 17], 2, 4, 16, **kw)
        out, lse = torch.empty_like(c.q), torch.empty(c.rows, 8, device=DEV)
        return [out, lse], lambda: c.call(out=out, lse=lse)
    return make


def logits_adjust():
    logits = rows(4, 100, dtype=F32)
    start = torch.tensor([0, 4], dtype=I32, device=DEV)
    return [logits], lambda: rc.logits_adjust(logits, start, out=logits)


def kv4_store():
    cache, scales = rc.new_kv4_cache(3, 2, 16, DEV)
    k, v, slots = rows(5, 2, 64), rows(5, 2, 64), torch.arange(5, device=DEV)
    return [cache, scales], lambda: rc.kv4_store(k, v, slots, cache, scales)


def kv4_load():
    cache, scales = rc.new_kv4_cache(3, 2, 16, DEV)
    out, slots = rows(5, 2, 128), torch.arange(5, device=DEV)
    return [out], lambda: rc.kv4_load(slots, cache, scales, out=out)


def kv_compact():
    ints = lambda *v: torch.tensor(v, dtype=I32, device=DEV)  # noqa: E731
    caches, new_len = [rows(4, 2, 16, 128), rows(4, 2, 16, 4)], ints(0)
    return caches + [new_len], lambda: rc.kv_compact(caches, ints(0, 1)[None], ints(9), ints(0, 6), ints(1, 4)[None], ints(2), new_len=new_len)


CALLS = dict(rope_table=rope_table, rope_apply=rope_apply, head_norm_rope=head_norm_rope, head_norm_rope_grad=head_norm_rope_grad,
             tree_attention=attention(), window_attention=attention(window=9), kv4_attention=attention(four=True), logits_adjust=logits_adjust,
             kv4_store=kv4_store, kv4_load=kv4_load, kv_compact=kv_compact)


@pytest.mark.parametrize("call", CALLS)
def test_versions_move_on(call):
    tensors, run = CALLS[call]()
    for _ in range(2):
        before = [t._version for t in tensors]
        run()
        assert all(t._version > v for t, v in zip(tensors, before))
    torch.cuda.synchronize()


@pytest.mark.parametrize("call,which", [(c, i) for c, n in [("rope_table", 1), ("rope_apply", 1), ("head_norm_rope", 1), ("head_norm_rope_grad", 1),
                                                             ("tree_attention", 2), ("kv4_attention", 2), ("logits_adjust", 1), ("kv4_load", 1),
                                                             ("kv_compact", 2)] for i in range(n)])
def test_a_backward_pass_finds_what_it_saved_overwritten(call, which):
    tensors, run = CALLS[call]()
    t = tensors[which]
    w = torch.ones(t.shape[-1], device=DEV, dtype=t.dtype, requires_grad=True)
    y = (t * w).sum()                                    # saves t for the gradient of w
    run()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


def test_through_a_view_of_it():
    """Q's columns of a projection's rows, turned in place: the rows are changed."""
    projected = rows(5, 12 * 64)
    w = torch.ones(12 * 64, device=DEV, dtype=BF, requires_grad=True)
    y = (projected * w).sum()
    q = projected[:, :8 * 64].view(5, 8, 64)
    rc.head_norm_rope(q, torch.arange(5, device=DEV), rc.rope_table(16, 64, device=DEV), eps=1e-6, out=q)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


def test_what_is_read_keeps_its_version():
    c = paged_cases.Case(3, [3, 1], [40, 17], 2, 4, 16)
    tensors = [c.q, c.cache, c.mask, c.table, c.context, c.row_start]
    before = [t._version for t in tensors]
    c.call()
    assert [t._version for t in tensors] == before
    x, pos, table = norm_operands()
    before = [t._version for t in (x, pos, table)]
    rc.head_norm_rope(x, pos, table, eps=1e-6)
    rc.head_norm_rope_grad(x.clone(), x, pos, table, eps=1e-6)
    assert [t._version for t in (x, pos, table)] == before


def test_refused_calls_change_no_version():
    x, pos, table = norm_operands()
    before = x._version
    with pytest.raises(rc.RopeChainError):
        rc.head_norm_rope(x, pos, table, eps=-1.0, out=x)
    assert x._version == before


@pytest.mark.parametrize("call", CALLS)
def test_tensors_of_inference_mode_are_written_in_it_and_after_it(call):
    with torch.inference_mode():
        tensors, run = CALLS[call]()
        run()
    run()
    torch.cuda.synchronize()
