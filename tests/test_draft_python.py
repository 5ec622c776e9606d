"""Refusals of the drafted tokens' calls in their Python module (no GPU
needed): the operands are tensors with a device, a shape and a type but no
memory, and every refusal comes before CUDA is asked for anything."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import rope_chain_gb300 as rc

BF, F32, I32, I64 = torch.bfloat16, torch.float32, torch.int32, torch.int64


@pytest.fixture(scope="module", autouse=True)
def built():
    from rope_chain_gb300 import _build
    _build.build()


def fake(*shape, dtype=BF, device="cuda:0", **kw):
    with FakeTensorMode():
        return torch.empty(*shape, dtype=dtype, device=device, **kw)


def rope_operands():
    return dict(x=fake(4, 8, 64), positions=fake(4, dtype=I64), cos_sin=fake(16, 64), out=fake(4, 8, 64),
                err=fake(1, dtype=I32))


def attention_operands():
    return dict(q=fake(4, 8, 64), row_start=fake(3, dtype=I32), context_len=fake(2, dtype=I32),
                block_table=fake(2, 5, dtype=I32), cache=fake(9, 2, 16, 128), tree_mask=fake(4, 1, dtype=I64),
                out=fake(4, 8, 64), lse=fake(4, 8, dtype=F32), err=fake(1, dtype=I32),
                workspace=fake(1 << 24, dtype=torch.uint8))


def logits_operands():
    return dict(logits=fake(4, 100, dtype=F32), row_start=fake(3, dtype=I32), history=fake(50, dtype=I32),
                history_start=fake(3, dtype=I64), prompt_len=fake(2, dtype=I32), draft_tokens=fake(4, dtype=I32),
                tree_mask=fake(4, 1, dtype=I64), repetition=fake(2, dtype=F32), frequency=fake(2, dtype=F32),
                presence=fake(2, dtype=F32), bias_start=fake(3, dtype=I32), bias_tokens=fake(6, dtype=I32),
                bias_values=fake(6, dtype=F32), allowed=fake(4, 4, dtype=I32), out=fake(4, 100, dtype=F32),
                err=fake(1, dtype=I32))


# (a tensor without memory sets up the context of its GPU where there are any)
two_gpus = pytest.mark.skipif(torch.cuda.device_count() == 1, reason="no GPU or two")
CALLS = {"rope_apply": rope_operands, "tree_attention": attention_operands, "logits_adjust": logits_operands}


@two_gpus
@pytest.mark.parametrize("call,name", [(c, n) for c, make in CALLS.items() for n in make()])
def test_operands_of_two_gpus_are_refused(call, name):
    args = CALLS[call]()
    with FakeTensorMode():
        args[name] = torch.empty_strided(args[name].shape, args[name].stride(), dtype=args[name].dtype, device="cuda:1")
    with pytest.raises(ValueError, match="is on device cuda:"):
        getattr(rc, call)(**args)


@two_gpus
def test_a_table_on_another_gpu_than_its_output_is_refused():
    with pytest.raises(ValueError, match="is on device cuda:"):
        rc.rope_table(16, 64, device="cuda:0", out=fake(16, 64, device="cuda:1"))


def test_scaling_by_parts_needs_the_trained_positions():
    """Without them every column but the first would be divided by the factor."""
    with pytest.raises(ValueError, match="original_max_position"):
        rc.rope_table(16, 64, scaling="parts", factor=4.0, out=fake(16, 64))


FLOATS = [("rope_apply", n) for n in ("x", "cos_sin", "out")] + [("tree_attention", n) for n in ("q", "cache", "out", "lse")] + \
    [("logits_adjust", n) for n in ("logits", "repetition", "frequency", "presence", "bias_values", "out")]


@pytest.mark.parametrize("call,name", FLOATS)
def test_gradients_are_not_dropped_silently(call, name):
    """What requires a gradient, where the call gives none, is refused while gradients are recorded."""
    args = CALLS[call]()
    args[name] = fake(*args[name].shape, dtype=args[name].dtype, requires_grad=True)
    with pytest.raises(ValueError, match=f"{name} requires a gradient"):
        getattr(rc, call)(**args)


def test_an_inverse_without_a_truth_value_is_refused():
    class Neither:
        def __bool__(self):
            raise ArithmeticError("neither")
    args = rope_operands()
    with pytest.raises(ArithmeticError, match="neither"):
        rc.rope_apply(**args, inverse=Neither())
