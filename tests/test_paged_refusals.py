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


K, V, SLOTS, C4, SC = 0x100000, 0x180000, 0x200000, 0x8000000, 0x9000000
KV4 = dict(k=K, kr=512, kh=64, v=V, vr=512, vh=64, T=4, heads=8, slots=SLOTS, cache=C4, scales=SC, nb=8, bs=16, err=ERR, out=OUT + 0x4000000)


def kv4_store(lib, **over):
    a = {**KV4, **over}
    return lib.rc_kv4_store(A(a["k"]), a["kr"], a["kh"], A(a["v"]), a["vr"], a["vh"], a["T"], a["heads"], A(a["slots"]),
                            A(a["cache"]), A(a["scales"]), a["nb"], a["bs"], A(a["err"]), None)


def kv4_load(lib, **over):
    a = {**KV4, **over}
    return lib.rc_kv4_load(A(a["slots"]), a["T"], a["heads"], A(a["cache"]), A(a["scales"]), a["nb"], a["bs"], A(a["out"]),
                           A(a["err"]), None)


COMMON4 = [dict(T=-1), dict(T=1 << 28), dict(heads=0), dict(nb=0), dict(bs=0), dict(nb=1 << 20, bs=1 << 11), dict(slots=None),
           dict(slots=SLOTS + 4), dict(cache=None), dict(cache=C4 + 8), dict(scales=None), dict(scales=SC + 4), dict(err=ERR + 2)]


def test_kv4_refusals(lib):
    for over in COMMON4 + [dict(k=None), dict(v=None), dict(k=K + 8), dict(v=V + 2), dict(kr=516), dict(vh=60), dict(kr=-512),
                           dict(vr=1 << 41), dict(cache=K), dict(scales=V), dict(scales=C4 + 64), dict(slots=C4), dict(err=SC)]:
        assert kv4_store(lib, **over) == BAD, over
    for over in COMMON4 + [dict(out=None), dict(out=KV4["out"] + 8), dict(out=C4), dict(out=SC), dict(slots=KV4["out"]), dict(err=KV4["out"])]:
        assert kv4_load(lib, **over) == BAD, over
    assert kv4_store(lib, T=0, k=None, v=None, slots=None) == OK and kv4_load(lib, T=0, out=None, slots=None) == OK


TABLE, LENS, START, PATH, COUNT, NEW = 0x30000, 0x20000, 0x10000, 0x40000, 0x50000, 0x60000
MOVE = dict(caches=(0x10000000, 0x20000000), bytes=(256, 8), nb=8, heads=4, bs=16, bt=TABLE, ts=4, tw=4, ctx=LENS, rs=START, seqs=2,
            rows=26, path=PATH, ps=5, pw=5, count=COUNT, new=NEW, err=ERR)


def compact(lib, **over):
    a = {**MOVE, **over}
    n = len(a["caches"]) if a["caches"] else 0
    caches = (ctypes.c_void_p * n)(*a["caches"]) if n else None
    sizes = (ctypes.c_int32 * len(a["bytes"]))(*a["bytes"]) if a["bytes"] else None
    return lib.rc_kv_compact(caches, sizes, n, a["nb"], a["heads"], a["bs"], A(a["bt"]), a["ts"], a["tw"], A(a["ctx"]), A(a["rs"]),
                             a["seqs"], a["rows"], A(a["path"]), a["ps"], a["pw"], A(a["count"]), A(a["new"]), A(a["err"]), None)


def test_compact_refusals(lib):
    first = MOVE["caches"][0]
    size = 8 * 4 * 16 * 256
    for over in (dict(caches=()), dict(bytes=()), dict(caches=(first,) * 65, bytes=(256,) * 65), dict(nb=0), dict(bs=0), dict(heads=0),
                 dict(heads=65537), dict(nb=1 << 20, bs=1 << 11), dict(seqs=0), dict(seqs=1 << 24), dict(rows=-1), dict(rows=1 << 31),
                 dict(tw=-1), dict(ts=-1), dict(tw=1 << 20, bs=1 << 11), dict(pw=-1), dict(ps=-1), dict(ps=1 << 41), dict(rs=None),
                 dict(ctx=None), dict(count=None), dict(path=None), dict(bt=None), dict(rs=START + 2), dict(ctx=LENS + 1),
                 dict(count=COUNT + 2), dict(path=PATH + 2), dict(bt=TABLE + 2), dict(new=NEW + 2), dict(err=ERR + 2),
                 dict(bytes=(12, 8)), dict(bytes=(0, 8)), dict(bytes=(256, 4104)), dict(bytes=(-8, 8)), dict(caches=(None, 0x20000000)),
                 dict(caches=(first + 8, 0x20000000)), dict(caches=(first, 0x20000004)), dict(caches=(first, first + size - 8)),
                 dict(caches=(first, first)), dict(bt=first), dict(path=first + size - 4), dict(ctx=first), dict(rs=first), dict(count=first),
                 dict(new=first), dict(err=first), dict(new=LENS), dict(new=PATH), dict(new=START), dict(new=COUNT), dict(new=TABLE),
                 dict(new=ERR)):
        assert compact(lib, **over) == BAD, over


Q, RS, CL, BT, TM, CA, S4 = 0x1000000, 0x10000, 0x20000, 0x30000, 0x40000, 0x2000000, 0x3000000
ATTEND = dict(q=Q, qs=512, rows=4, heads=8, kv=2, rs=RS, seqs=2, cl=CL, bt=BT, ts=4, tw=4, tm=TM, mw=1, ca=CA, sc=S4, nb=8, bs=16,
              window=5, sinks=1, scale=0.125, out=OUT, os=512, lse=None, ws=None, wb=0)


def window(lib, **over):
    a = {**ATTEND, **over}
    return lib.rc_window_attention(A(a["q"]), a["qs"], a["rows"], a["heads"], a["kv"], A(a["rs"]), a["seqs"], A(a["cl"]), A(a["bt"]),
                                   a["ts"], a["tw"], A(a["tm"]), a["mw"], A(a["ca"]), a["nb"], a["bs"], a["window"], a["sinks"],
                                   a["scale"], A(a["out"]), a["os"], A(a["lse"]), None, A(a["ws"]), a["wb"], None)


def attend4(lib, **over):
    a = {**ATTEND, **over}
    return lib.rc_kv4_attention(A(a["q"]), a["qs"], a["rows"], a["heads"], a["kv"], A(a["rs"]), a["seqs"], A(a["cl"]), A(a["bt"]),
                                a["ts"], a["tw"], A(a["tm"]), a["mw"], A(a["ca"]), A(a["sc"]), a["nb"], a["bs"], a["window"],
                                a["sinks"], a["scale"], A(a["out"]), a["os"], A(a["lse"]), None, A(a["ws"]), a["wb"], None)


@pytest.mark.parametrize("call", [window, attend4])
def test_attention_refusals(lib, call):
    for over in (dict(heads=7), dict(kv=0), dict(heads=1, kv=2), dict(rows=-1), dict(rows=1 << 29), dict(seqs=0), dict(seqs=1 << 24),
                 dict(nb=0), dict(bs=0), dict(nb=1 << 20, bs=1 << 11), dict(tw=-1), dict(ts=-1), dict(tw=1 << 20, bs=1 << 11),
                 dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(q=None), dict(q=Q + 8),
                 dict(out=None), dict(out=OUT + 2), dict(ca=None), dict(ca=CA + 4), dict(rs=None), dict(cl=None), dict(bt=None),
                 dict(tm=TM + 4), dict(mw=0), dict(qs=516), dict(qs=-512), dict(os=448), dict(os=516), dict(lse=0x50002),
                 dict(ws=WS + 8, wb=1 << 30), dict(out=Q), dict(out=Q + 512), dict(out=CA), dict(lse=OUT), dict(window=-1),
                 dict(sinks=-1), dict(window=0, sinks=1), dict(out=CL & ~15), dict(lse=TM)):
        assert call(lib, **over) == BAD, over
    assert call(lib, rows=0, q=None, out=None, tm=None, bt=None, tw=0) == OK
    rows = (1 << 31) - 1
    assert call(lib, rows=rows, heads=1, kv=1, seqs=1, qs=0, os=64, out=1 << 60, tm=None) == BAD


def test_attention_of_each_format(lib):
    assert window(lib, window=0, sinks=0) == BAD
    for over in (dict(sc=None), dict(sc=S4 + 4), dict(out=S4), dict(lse=S4)):
        assert attend4(lib, **over) == BAD, over
    assert attend4(lib, rows=0, window=0, sinks=0) == OK
    for sizes in ((0, 1, 8, 8), (4, 0, 8, 8), (4, 1, 8, 3), (4, 1, 0, 0), (1 << 30, 1, 8, 8)):
        assert lib.rc_kv4_attention_workspace_size(*sizes) == 0
