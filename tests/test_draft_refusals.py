"""Refusals of the drafted tokens' operators, on the host before any CUDA
call (no GPU needed): malformed arguments are rejected, empty calls succeed."""
import ctypes

import pytest
import torch

import rope_chain_gb300 as rc

X, POS, TAB, OUT = 0x100000, 0x200000, 0x300000, 0x8000000


@pytest.fixture(scope="module")
def lib():
    from rope_chain_gb300 import _build
    _build.build()
    return rc.lib()


def A(v):
    return None if v is None else ctypes.c_void_p(v)


def table(lib, scaling=None, **over):
    a = dict(out=OUT, dtype=rc.RC_BF16, n=16, rot=64, theta=1e4)
    a.update(over)
    sc = rc.RopeScaling(*scaling) if scaling else None
    return lib.rc_rope_table(A(a["out"]), a["dtype"], a["n"], a["rot"], a["theta"],
                             ctypes.byref(sc) if sc else None, None)


def test_rope_table_refusals(lib):
    bad = rc.RC_ERR_INVALID_ARG
    assert table(lib, dtype=3) == bad
    assert table(lib, n=-1) == bad and table(lib, n=1 << 31) == bad
    for rot in (0, 3, 514):
        assert table(lib, rot=rot) == rc.RC_ERR_UNSUPPORTED
    for theta in (1.0, 0.0, -2.0, float("inf"), float("nan")):
        assert table(lib, theta=theta) == bad
    assert table(lib, out=None) == bad and table(lib, out=OUT + 8) == bad
    good = (1, 2.0, 1.0, 32.0, 1.0, 1.0)
    for at, v in ((0, 4), (0, -1), (1, 0.0), (1, float("nan")), (5, float("inf"))):
        assert table(lib, scaling=good[:at] + (v,) + good[at + 1:]) == bad
    parts = (3, 2.0, 4096.0, 32.0, 1.0, 1.0)
    for at, v in ((2, 0.0), (3, 1.0), (4, 0.0), (4, 32.0)):
        assert table(lib, scaling=parts[:at] + (v,) + parts[at + 1:]) == bad
    assert table(lib, scaling=(2, 2.0, 1.0, 32.0, 1.0, 1.0), rot=2) == rc.RC_ERR_UNSUPPORTED
    assert table(lib, n=0, scaling=parts) == rc.RC_OK
    assert lib.rc_last_error() == b""


def apply(lib, **over):
    a = dict(x=X, dtype=rc.RC_BF16, xr=512, xh=64, T=4, heads=8, dim=64, pos=POS, tab=TAB,
             tdt=rc.RC_BF16, maxpos=128, rot=64, layout=0, inv=0, out=OUT, orow=512, oh=64)
    a.update(over)
    return lib.rc_rope_apply(A(a["x"]), a["dtype"], a["xr"], a["xh"], a["T"], a["heads"], a["dim"],
                             A(a["pos"]), A(a["tab"]), a["tdt"], a["maxpos"], a["rot"], a["layout"],
                             a["inv"], A(a["out"]), a["orow"], a["oh"], None, None)


def test_rope_apply_refusals(lib):
    bad = rc.RC_ERR_INVALID_ARG
    for over in (dict(dtype=0), dict(tdt=3), dict(layout=2), dict(T=-1), dict(heads=0), dict(T=1 << 28),
                 dict(xr=-64), dict(oh=-64), dict(x=None), dict(out=None), dict(x=X + 1),
                 dict(dtype=rc.RC_F32, x=X + 2), dict(pos=None), dict(pos=POS + 4), dict(tab=None),
                 dict(maxpos=0), dict(out=X + 2), dict(out=X, orow=576), dict(orow=0), dict(oh=0),
                 dict(orow=64, oh=64)):
        assert apply(lib, **over) == bad, over
    for over in (dict(rot=63), dict(rot=66), dict(rot=0), dict(dim=65, rot=64), dict(dim=1 << 17),
                 dict(dim=1024, rot=514)):
        assert apply(lib, **over) == rc.RC_ERR_UNSUPPORTED, over
    assert apply(lib, T=0) == rc.RC_OK


Q, RS, CL, BT, TM, CA, WS = 0x1000000, 0x10000, 0x20000, 0x30000, 0x40000, 0x2000000, 0x40000000


def attend(lib, **over):
    a = dict(q=Q, qs=512, rows=4, heads=8, kv=2, rs=RS, seqs=2, cl=CL, bt=BT, ts=4, tw=4, tm=TM, mw=1,
             ca=CA, nb=8, bs=16, scale=0.125, out=OUT, os=512, lse=None, ws=None, wb=0)
    a.update(over)
    return lib.rc_tree_attention(A(a["q"]), a["qs"], a["rows"], a["heads"], a["kv"], A(a["rs"]),
                                 a["seqs"], A(a["cl"]), A(a["bt"]), a["ts"], a["tw"], A(a["tm"]),
                                 a["mw"], A(a["ca"]), a["nb"], a["bs"], a["scale"], A(a["out"]),
                                 a["os"], A(a["lse"]), None, A(a["ws"]), a["wb"], None)


def test_tree_attention_refusals(lib):
    for over in (dict(heads=7), dict(kv=0), dict(heads=1, kv=2), dict(rows=-1), dict(rows=1 << 29),
                 dict(seqs=0), dict(seqs=1 << 24), dict(nb=0), dict(bs=0), dict(nb=1 << 20, bs=1 << 11),
                 dict(tw=-1), dict(ts=-1), dict(tw=1 << 20, bs=1 << 11), dict(scale=0.0), dict(scale=-1.0),
                 dict(scale=float("nan")), dict(scale=float("inf")), dict(q=None), dict(q=Q + 8),
                 dict(out=None), dict(out=OUT + 2), dict(ca=None), dict(ca=CA + 4), dict(rs=None),
                 dict(cl=None), dict(bt=None), dict(tm=TM + 4), dict(mw=0), dict(qs=516), dict(qs=-512),
                 dict(os=448), dict(os=516), dict(lse=0x50002), dict(ws=WS + 8, wb=1 << 30),
                 dict(out=Q), dict(out=Q + 512), dict(out=CA), dict(lse=OUT)):
        assert attend(lib, **over) == rc.RC_ERR_INVALID_ARG, over
    assert attend(lib, rows=0) == rc.RC_OK
    for sizes in ((0, 1, 8, 8), (4, 0, 8, 8), (4, 1, 8, 3), (4, 1, 0, 0), (1 << 30, 1, 8, 8)):
        assert lib.rc_tree_attention_workspace_size(*sizes) == 0


def adjust(lib, params=None, **over):
    a = dict(x=Q, dtype=rc.RC_F32, stride=100, rows=4, vocab=100, rs=RS, seqs=2, out=OUT, os=100)
    a.update(over)
    p = rc.LogitsParams(**{k: v for k, v in (params or {}).items()})
    return lib.rc_logits_adjust(A(a["x"]), a["dtype"], a["stride"], a["rows"], a["vocab"], A(a["rs"]),
                                a["seqs"], None if params == "none" else ctypes.byref(p), A(a["out"]),
                                a["os"], None, None)


def test_logits_refusals(lib):
    bad = rc.RC_ERR_INVALID_ARG
    for over in (dict(dtype=0), dict(rows=-1), dict(rows=(1 << 30) + 1), dict(vocab=0), dict(seqs=0),
                 dict(seqs=65536), dict(x=None), dict(out=None), dict(rs=None), dict(x=Q + 2),
                 dict(stride=-1), dict(os=99), dict(out=Q + 4), dict(out=Q, os=104)):
        assert adjust(lib, **over) == bad, over
    for params in (dict(history=0x1000), dict(history=0x1000, history_start=0x2000, history_size=-1),
                   dict(history=0x1000, history_start=0x2000, history_size=1 << 28),
                   dict(history=0x1002, history_start=0x2000), dict(history=0x1000, history_start=0x2004),
                   dict(bias_start=0x1000), dict(bias_tokens=0x1000),
                   dict(bias_start=0x1000, bias_tokens=0x1000, bias_values=0x1000, bias_size=-1),
                   dict(tree_mask=0x1000), dict(tree_mask=0x1004, mask_words=1), dict(repetition=0x1002),
                   dict(allowed=0x1000, allowed_stride=3), dict(prompt_len=0x1001)):
        assert adjust(lib, params=params) == bad, params
    assert adjust(lib, rows=0) == rc.RC_OK


def test_empty_calls_need_no_addresses(lib):
    assert table(lib, n=0, out=None) == rc.RC_OK
    assert apply(lib, T=0, x=None, out=None, pos=None) == rc.RC_OK
    assert attend(lib, rows=0, q=None, out=None, tm=None, bt=None, tw=0) == rc.RC_OK
    assert adjust(lib, rows=0, x=None, out=None) == rc.RC_OK


def test_python_checks_shapes_and_types():
    cpu = torch.zeros(4, 8, 64, dtype=torch.bfloat16)
    with pytest.raises((TypeError, ValueError)):
        rc.rope_apply(cpu, torch.zeros(4, dtype=torch.int64), torch.zeros(16, 64, dtype=torch.bfloat16))
    with pytest.raises((TypeError, ValueError)):
        rc.tree_attention(cpu, None, None, None, None)
    with pytest.raises((TypeError, ValueError)):
        rc.logits_adjust(torch.zeros(4, 100), torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="scaling"):
        rc.rope_table(16, scaling="other")


def test_outputs_over_what_is_still_read(lib):
    """Other CTAs read positions, tables, lists and masks while one writes its outputs."""
    bad = rc.RC_ERR_INVALID_ARG
    end = OUT + 2 * 4 * 512                            # of out: [4, 8, 64] bf16
    for at in (OUT, OUT + 512, end - 16):
        for name in ("pos", "tab"):
            assert apply(lib, **{name: at}) == bad, (name, at)
        for name in ("rs", "cl", "bt", "tm"):
            assert attend(lib, **{name: at}) == bad, (name, at)
    assert attend(lib, tm=OUT - 24) == bad             # the mask's last row
    assert attend(lib, bt=OUT - 28) == bad             # the table's last
    lse = 0x5000000
    for name in ("q", "ca", "rs", "cl", "bt", "tm"):
        assert attend(lib, lse=lse, **{name: lse}) == bad, name
    last = OUT + 4 * 399                               # of out: [4, 100] FP32
    assert adjust(lib, rs=last) == bad
    for at in (OUT & ~7, last & ~7):
        for params in (dict(history=at, history_size=1, history_start=0x2000),
                       dict(history=0x1000, history_size=1, history_start=at), dict(prompt_len=at),
                       dict(draft_tokens=at), dict(tree_mask=at, mask_words=1), dict(repetition=at),
                       dict(frequency=at), dict(presence=at), dict(allowed=at, allowed_stride=4),
                       dict(bias_start=at, bias_tokens=0x1000, bias_values=0x2000, bias_size=2),
                       dict(bias_start=0x1000, bias_tokens=at, bias_values=0x2000, bias_size=2),
                       dict(bias_start=0x1000, bias_tokens=0x2000, bias_values=at, bias_size=2)):
            assert adjust(lib, params=params) == bad, params
    assert adjust(lib, params=dict(allowed=OUT - 48, allowed_stride=4)) == bad


def test_rows_whose_last_tile_ends_past_32_bits(lib):
    """2^31 - 1 rows of a KV head: the last tile of 16 to 256 rows would end past 2^31."""
    rows = (1 << 31) - 1
    far = 1 << 60
    for n in (rows, rows - 15, rows - 255):
        assert attend(lib, rows=n, heads=1, kv=1, seqs=1, qs=0, os=64, out=far, tm=None) == rc.RC_ERR_INVALID_ARG, n
        assert lib.rc_last_error().decode().find("2^31") > 0
        assert lib.rc_tree_attention_workspace_size(n, 1, 1, 1) == 0


def test_the_stride_of_one_row_is_not_looked_at(lib):
    for over in (dict(qs=516), dict(qs=-512), dict(os=448), dict(os=516)):
        assert attend(lib, rows=0, **over) == rc.RC_OK, over
        assert attend(lib, rows=2, **over) == rc.RC_ERR_INVALID_ARG, over
