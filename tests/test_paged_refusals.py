"""Refusals of the operators around the drafted tokens' step, on the host before
any CUDA call (no GPU needed): malformed arguments are rejected, empty calls
succeed."""
import ctypes

import pytest

import rope_chain_gb300 as rc

BAD, UNSUPPORTED, OK = rc.RC_ERR_INVALID_ARG, rc.RC_ERR_UNSUPPORTED, rc.RC_OK


@pytest.fixture(scope="module")
def lib():
    from rope_chain_gb300 import _build
    _build.build()
    return rc.lib()


def A(v):
    return None if v is None else ctypes.c_void_p(v)


X, DY, POS, TAB, OUT, QW, KW = 0x100000, 0x140000, 0x200000, 0x300000, 0x8000000, 0x400000, 0x410000
DQ, DK, WS, ERR = 0x420000, 0x430000, 0x40000000, 0x440000
NORM = dict(x=X, dtype=rc.RC_BF16, xr=512, xh=64, T=4, heads=8, dim=64, nq=6, qw=QW, kw=KW, wdt=rc.RC_BF16, eps=1e-6, pos=POS,
            tab=TAB, tdt=rc.RC_BF16, maxpos=128, rot=64, layout=0, out=OUT, orow=512, oh=64, err=ERR, params=True)


def params_of(a):
    return ctypes.byref(rc.HeadNormParams(a["nq"], A(a["qw"]), A(a["kw"]), a["wdt"], a["eps"])) if a["params"] else None


def norm(lib, **over):
    a = {**NORM, **over}
    return lib.rc_head_norm_rope(A(a["x"]), a["dtype"], a["xr"], a["xh"], a["T"], a["heads"], a["dim"], params_of(a), A(a["pos"]),
                                 A(a["tab"]), a["tdt"], a["maxpos"], a["rot"], a["layout"], A(a["out"]), a["orow"], a["oh"],
                                 A(a["err"]), None)


def norm_grad(lib, **over):
    a = {**NORM, **dict(dy=DY, dr=512, dh=64, dq=DQ, dk=DK, ws=WS, wb=1 << 30), **over}
    return lib.rc_head_norm_rope_grad(A(a["dy"]), a["dr"], a["dh"], A(a["x"]), a["dtype"], a["xr"], a["xh"], a["T"], a["heads"],
                                      a["dim"], params_of(a), A(a["pos"]), A(a["tab"]), a["tdt"], a["maxpos"], a["rot"],
                                      a["layout"], A(a["out"]), a["orow"], a["oh"], A(a["dq"]), A(a["dk"]), A(a["ws"]), a["wb"],
                                      A(a["err"]), None)


@pytest.mark.parametrize("call", [norm, norm_grad])
def test_head_norm_refusals(lib, call):
    for over in (dict(dtype=0), dict(tdt=3), dict(wdt=0), dict(layout=2), dict(T=-1), dict(heads=0), dict(T=1 << 28), dict(xr=-64),
                 dict(oh=-64), dict(xh=1 << 41), dict(x=None), dict(out=None), dict(x=X + 1), dict(dtype=rc.RC_F32, x=X + 2),
                 dict(pos=None), dict(pos=POS + 4), dict(tab=None), dict(maxpos=0), dict(out=OUT + 1), dict(out=X, orow=576),
                 dict(orow=0), dict(oh=0), dict(orow=64, oh=64), dict(nq=-1), dict(nq=9), dict(eps=-1e-6), dict(eps=float("nan")),
                 dict(eps=float("inf")), dict(qw=QW + 1), dict(wdt=rc.RC_F32, kw=KW + 2), dict(err=ERR + 1), dict(params=False),
                 dict(pos=OUT), dict(tab=OUT), dict(qw=OUT + 64), dict(kw=OUT + 4 * 512 * 2 - 2), dict(err=OUT)):
        assert call(lib, **over) == BAD, over
        assert lib.rc_last_error()
    for over in (dict(rot=63), dict(rot=66), dict(rot=0), dict(dim=65), dict(dim=1), dict(dim=514), dict(dim=0)):
        assert call(lib, **over) == UNSUPPORTED, over
    # (65 elements in halves are fine as far as the host goes: the next check speaks)
    assert call(lib, dim=65, layout=1, x=None) == BAD


def test_head_norm_grad_refusals(lib):
    for over in (dict(dy=None), dict(dy=DY + 1), dict(dr=-1), dict(dh=1 << 41), dict(dq=DQ + 2), dict(ws=None), dict(ws=WS + 8),
                 dict(out=DY, orow=576, dr=512), dict(out=DY + 64), dict(dq=X), dict(dk=DY), dict(dq=OUT), dict(dq=DK),
                 dict(dq=QW), dict(dk=TAB), dict(dk=POS)):
        assert norm_grad(lib, **over) == BAD, over


def test_empty_head_norms(lib):
    assert norm(lib, T=0, x=None, out=None, pos=None) == OK
    assert norm_grad(lib, T=0, x=None, out=None, pos=None, dy=None, dq=None, dk=None, ws=None, wb=0) == OK
    assert lib.rc_last_error() == b""
    for dim in (0, 1, 513):
        assert lib.rc_head_norm_rope_grad_workspace_size(dim) == 0
