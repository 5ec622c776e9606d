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


CALLS = {"head_norm_rope": norm_operands, "head_norm_rope_grad": norm_grad_operands}
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
