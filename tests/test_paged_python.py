"""Refusals of the calls around the drafted tokens' step in their Python module
(no GPU needed): the operands are tensors with a device, a shape and a type but
no memory, and every refusal comes before CUDA is asked for anything."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import rope_chain_gb300 as rc

BF, F32, I32, I64, U8 = torch.bfloat16, torch.float32, torch.int32, torch.int64, torch.uint8


@pytest.fixture(scope="module", autouse=True)
def built():
    from rope_chain_gb300 import _build
    _build.build()


def fake(*shape, dtype=BF, device="cuda:0", **kw):
    with FakeTensorMode():
        return torch.empty(*shape, dtype=dtype, device=device, **kw)


def norm_operands():
    return dict(x=fake(4, 8, 64), positions=fake(4, dtype=I64), cos_sin=fake(16, 64), q_weight=fake(64), k_weight=fake(64),
                out=fake(4, 8, 64), err=fake(1, dtype=I32), eps=1e-6, q_heads=5)


def norm_grad_operands():
    return dict(norm_operands(), grad=fake(4, 8, 64), workspace=fake(1 << 24, dtype=U8))


def store_operands():
    return dict(k=fake(4, 8, 64), v=fake(4, 8, 64), slots=fake(4, dtype=I64), cache=fake(9, 8, 16, 64, dtype=U8),
                scales=fake(9, 8, 16, 4), err=fake(1, dtype=I32))


def load_operands():
    return dict(slots=fake(4, dtype=I64), cache=fake(9, 8, 16, 64, dtype=U8), scales=fake(9, 8, 16, 4), out=fake(4, 8, 128),
                err=fake(1, dtype=I32))


def compact_operands():
    return dict(block_table=fake(2, 5, dtype=I32), caches=[fake(9, 8, 16, 128)], context_len=fake(2, dtype=I32),
                row_start=fake(3, dtype=I32), path=fake(2, 4, dtype=I32), path_len=fake(2, dtype=I32), new_len=fake(2, dtype=I32),
                err=fake(1, dtype=I32))


def window_operands():
    return dict(q=fake(4, 8, 64), row_start=fake(3, dtype=I32), context_len=fake(2, dtype=I32), block_table=fake(2, 5, dtype=I32),
                cache=fake(9, 2, 16, 128), tree_mask=fake(4, 1, dtype=I64), out=fake(4, 8, 64), lse=fake(4, 8, dtype=F32),
                err=fake(1, dtype=I32), workspace=fake(1 << 24, dtype=U8), window=5, sinks=1)


def kv4_attention_operands():
    return dict(window_operands(), cache=fake(9, 2, 16, 64, dtype=U8), scales=fake(9, 2, 16, 4))


CALLS = {"window_attention": window_operands, "kv4_attention": kv4_attention_operands, "head_norm_rope": norm_operands, "head_norm_rope_grad": norm_grad_operands, "kv4_store": store_operands,
         "kv4_load": load_operands, "kv_compact": compact_operands}
TENSORS = [(c, n) for c, make in CALLS.items() for n, t in make().items() if isinstance(t, torch.Tensor)]
# (a tensor without memory sets up the context of its GPU where there are any)
two_gpus = pytest.mark.skipif(torch.cuda.device_count() == 1, reason="no GPU or two")


@two_gpus
@pytest.mark.parametrize("call,name", TENSORS)
def test_operands_of_two_gpus_are_refused(call, name):
    args = CALLS[call]()
    first = next(iter(args))
    if name == first:
        pytest.skip("the others lie beside it")
    with FakeTensorMode():
        args[name] = torch.empty_strided(args[name].shape, args[name].stride(), dtype=args[name].dtype, device="cuda:1")
    with pytest.raises(ValueError, match="is on device cuda:"):
        getattr(rc, call)(**args)


@pytest.mark.parametrize("call,name", [(c, n) for c, n in TENSORS if CALLS[c]()[n].is_floating_point()])
def test_gradients_are_not_dropped_silently(call, name):
    """What requires a gradient, where the call gives none (here: with an output), is refused while gradients are recorded."""
    args = CALLS[call]()
    args[name] = fake(*args[name].shape, dtype=args[name].dtype, requires_grad=True)
    with pytest.raises(ValueError, match="requires a gradient"):
        getattr(rc, call)(**args)


@pytest.mark.parametrize("call,name", TENSORS)
def test_tensors_of_the_host_are_refused(call, name):
    args = CALLS[call]()
    args[name] = fake(*args[name].shape, dtype=args[name].dtype, device="cpu")
    with pytest.raises((TypeError, ValueError)):
        getattr(rc, call)(**args)


@pytest.mark.parametrize("call", ["head_norm_rope", "head_norm_rope_grad"])
@pytest.mark.parametrize("change", [
    dict(x=fake(4, 512)), dict(x=fake(4, 8, 64, dtype=torch.float16)), dict(x=fake(4, 64, 8).transpose(1, 2)),
    dict(positions=fake(3, dtype=I64)), dict(positions=fake(4, dtype=I32)), dict(positions=None), dict(cos_sin=fake(16, 128)[:, :64]),
    dict(cos_sin=fake(16)), dict(q_weight=fake(32)), dict(k_weight=fake(64, dtype=F32)), dict(q_weight=fake(8, 64)),
    dict(q_heads=None), dict(q_heads=2 ** 40), dict(out=fake(4, 8, 32)), dict(out=fake(4, 8, 64, dtype=F32)),
    dict(out=fake(4, 64, 8).transpose(1, 2)), dict(eps="small"), dict(err=fake(1, dtype=I64))])
def test_head_norm_shapes_and_types(call, change):
    with pytest.raises((TypeError, ValueError)):
        getattr(rc, call)(**{**CALLS[call](), **change})


def test_head_norm_gradient_like_x():
    for grad in (fake(4, 8, 32), fake(4, 8, 64, dtype=F32), fake(4, 64, 8).transpose(1, 2), fake(3, 8, 64)):
        with pytest.raises((TypeError, ValueError)):
            rc.head_norm_rope_grad(**dict(norm_grad_operands(), grad=grad))


@pytest.mark.parametrize("call", ["kv4_store", "kv4_load"])
@pytest.mark.parametrize("change", [
    dict(cache=fake(9, 8, 16, 128, dtype=U8)), dict(cache=fake(9, 8, 16, 64)), dict(cache=fake(9, 8, 64, 16, dtype=U8).transpose(2, 3)),
    dict(scales=fake(9, 8, 16, 4, dtype=F32)), dict(scales=fake(9, 8, 16, 2)), dict(scales=fake(8, 8, 16, 4)), dict(slots=None),
    dict(slots=fake(4, dtype=I32)), dict(slots=fake(8, dtype=I64)[::2]), dict(err=fake(0, dtype=I32))])
def test_kv4_shapes_and_types(call, change):
    with pytest.raises((TypeError, ValueError)):
        getattr(rc, call)(**{**CALLS[call](), **change})


@pytest.mark.parametrize("change", [dict(k=fake(4, 7, 64)), dict(k=fake(4, 8, 32)), dict(v=fake(3, 8, 64)), dict(v=fake(4, 8, 64, dtype=F32)),
                                    dict(k=fake(4, 64, 8).transpose(1, 2)), dict(slots=fake(3, dtype=I64)),
                                    dict(k=fake(4, 2, 64), v=fake(4, 2, 64))])
def test_kv4_rows(change):
    with pytest.raises((TypeError, ValueError)):
        rc.kv4_store(**{**store_operands(), **change})


@pytest.mark.parametrize("change", [dict(out=fake(4, 8, 64)), dict(out=fake(3, 8, 128)), dict(out=fake(4, 8, 128, dtype=F32))])
def test_kv4_output(change):
    with pytest.raises((TypeError, ValueError)):
        rc.kv4_load(**{**load_operands(), **change})


@pytest.mark.parametrize("change", [
    dict(caches=[]), dict(caches=3), dict(caches=[None]), dict(caches=[fake(9, 8, 16, 128)] * 65), dict(caches=[fake(9, 8, 16)]),
    dict(caches=[fake(9, 8, 16, 128), fake(9, 8, 15, 4)]), dict(caches=[fake(9, 8, 128, 16).transpose(2, 3)]),
    dict(caches=[fake(9, 8, 16, 128, requires_grad=True)]), dict(caches=[fake(9, 8, 16, 128, device="cpu")]),
    dict(block_table=fake(2, 5, dtype=I64)), dict(block_table=fake(2, 10, dtype=I32)[:, ::2]), dict(path=fake(3, 4, dtype=I32)),
    dict(path=fake(2, 4, dtype=I64)), dict(path=fake(4, 2, dtype=I32).t()), dict(context_len=fake(1, dtype=I32)),
    dict(row_start=fake(2, dtype=I32)), dict(path_len=None), dict(path_len=fake(2, dtype=I64)), dict(new_len=fake(1, dtype=I32))])
def test_compact_shapes_and_types(change):
    with pytest.raises((TypeError, ValueError)):
        rc.kv_compact(**{**compact_operands(), **change})


@pytest.mark.parametrize("call", ["window_attention", "kv4_attention"])
@pytest.mark.parametrize("change", [
    dict(q=fake(4, 8, 32)), dict(q=fake(4, 8, 64, dtype=F32)), dict(q=fake(4, 512)), dict(q=fake(8, 4, 64).transpose(0, 1)),
    dict(row_start=fake(2, dtype=I32)), dict(row_start=None), dict(context_len=fake(2, dtype=I64)), dict(block_table=fake(2, 5, dtype=I64)),
    dict(block_table=fake(2, 10, dtype=I32)[:, ::2]), dict(cache=fake(9, 2, 16, 32)), dict(cache=fake(9, 2, 16)),
    dict(tree_mask=fake(3, 1, dtype=I64)), dict(tree_mask=fake(4, 0, dtype=I64)), dict(tree_mask=fake(4, 1, dtype=I32)),
    dict(out=fake(4, 8, 32)), dict(out=fake(8, 4, 64).transpose(0, 1)), dict(lse=fake(4, 7, dtype=F32)), dict(lse=fake(4, 8)),
    dict(workspace=fake(64, 2, dtype=U8).t()), dict(window="wide"), dict(window=2 ** 31), dict(sinks=2 ** 31), dict(sinks=None)])
def test_attention_shapes_and_types(call, change):
    with pytest.raises((TypeError, ValueError)):
        getattr(rc, call)(**{**CALLS[call](), **change})


@pytest.mark.parametrize("change", [dict(scales=fake(9, 2, 16, 2)), dict(scales=fake(9, 2, 16, 4, dtype=F32)), dict(scales=fake(9, 2, 15, 4)),
                                    dict(window=0), dict(window=-1), dict(sinks=-1), dict(window=None)])
def test_kv4_attention_operands(change):
    with pytest.raises((TypeError, ValueError)):
        rc.kv4_attention(**{**kv4_attention_operands(), **change})


@pytest.mark.parametrize("change", [dict(window=0), dict(window=-3), dict(sinks=-1)])
def test_windows(change):
    with pytest.raises(ValueError):
        rc.window_attention(**{**window_operands(), **change})
