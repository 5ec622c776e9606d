"""Tangents of forward-mode differentiation are refused, not dropped, by the calls that
carry none on (no GPU needed: tensors without memory, refused before CUDA is asked for
anything)."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode
from torch.autograd import forward_ad

import rope_chain_gb300 as rc
from tests import test_draft_python as drafted
from tests import test_paged_python as paged

CALLS = {**drafted.CALLS, **paged.CALLS}


@pytest.fixture(scope="module", autouse=True)
def built():
    from rope_chain_gb300 import _build
    _build.build()


def has_tangent(t):
    """Such a tensor like t (one mode for both of its parts)."""
    with FakeTensorMode():
        made = [torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device=t.device) for _ in range(2)]
        return forward_ad.make_dual(made[0].requires_grad_(t.requires_grad), made[1])


FLOATS = [(c, n) for c, make in CALLS.items() for n, t in make().items() if isinstance(t, torch.Tensor) and t.is_floating_point()]


@pytest.mark.parametrize("call,name", FLOATS)
@pytest.mark.parametrize("grad_mode", [True, False])
def test_tangents_are_not_dropped(call, name, grad_mode):
    args = CALLS[call]()
    with forward_ad.dual_level(), torch.set_grad_enabled(grad_mode):
        args[name] = has_tangent(args[name])
        with pytest.raises(ValueError, match=f"{name} has a tangent"):
            getattr(rc, call)(**args)


@pytest.mark.parametrize("call,name", [("rope_apply", "x"), ("head_norm_rope", "x"), ("head_norm_rope", "q_weight"), ("head_norm_rope", "k_weight")])
@pytest.mark.parametrize("recorded", [True, False])
def test_tangents_of_what_is_recorded(call, name, recorded):
    """Without an output, where the reverse mode has a gradient."""
    args = dict(CALLS[call](), out=None)
    args["x"] = drafted.fake(4, 8, 64, requires_grad=recorded)
    with forward_ad.dual_level():
        args[name] = has_tangent(args[name])
        with pytest.raises(ValueError, match=f"{name} has a tangent"):
            getattr(rc, call)(**args)


def test_tangents_of_caches():
    args = paged.compact_operands()
    with forward_ad.dual_level():
        args["caches"] = [has_tangent(args["caches"][0])]
        with pytest.raises(ValueError, match="a cache has a tangent"):
            rc.kv_compact(**args)


def test_a_tangent_does_not_outlive_its_level():
    """Refused for another reason then: the shape."""
    args = dict(paged.norm_operands(), positions=paged.fake(3, dtype=torch.int64))
    with forward_ad.dual_level():
        args["q_weight"] = has_tangent(args["q_weight"])
    with pytest.raises(ValueError, match="positions needs"):
        rc.head_norm_rope(**args)
