"""The per-head-decay and beam-search entry points on a host without a GPU:
libgdr exports what include/gdr_ops.h declares, and bad arguments are refused
with the documented status before any HIP call (no call here passes)."""
import ctypes
import os
import re

import pytest
import torch

import gated_delta_rule_26_amd as gdr

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "gdr_ops.h")

pytestmark = pytest.mark.skipif(not os.path.exists(gdr.library_path), reason="libgdr.so not built")

E = {name: code for code, name in gdr.STATUS.items()}
BASE = 1 << 40


def P(i, off=0):
    return ctypes.c_void_p(BASE + i * (1 << 36) + off)


def desc(B=2, T=600, H=4, Hk=2, Dk=64, Dv=96, dtype=torch.bfloat16, **kw):
    return gdr.make_head_decay_desc(B, T, H, Hk, Dk, Dv, dtype=dtype, **kw)


def test_exports_and_desc_layout():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    lib = gdr.load_library()
    names = sorted(set(re.findall(r"\b(gdr_[a-z_0-9]+)\s*\(", text)))
    assert len(names) == 8
    for n in names:
        assert hasattr(lib, n), n
    body = text[text.index("typedef struct gdr_head_decay_desc"):text.index("} gdr_head_decay_desc;")]
    fields = re.findall(r"(int32_t|float|int64_t)\s+(\w+)(\[3\])?;", body)
    assert [f[1] for f in fields] == [f for f, _ in gdr.HeadDecayDesc._fields_]
    assert ctypes.sizeof(gdr.HeadDecayDesc) == 8 * 4 + 4 * 3 * 8


def size(d, packed=0, dg=None):
    n = ctypes.c_size_t(0)
    lib = gdr.load_library()
    if dg is None:
        return lib.gdr_head_decay_fwd_workspace_size(ctypes.byref(d), packed, ctypes.byref(n)), n.value
    return lib.gdr_head_decay_bwd_workspace_size(ctypes.byref(d), packed, dg, ctypes.byref(n)), n.value


def test_workspace_queries():
    assert size(desc(T=64)) == (0, 0)                      # one segment: nothing to keep
    assert size(desc(T=2000, B=1))[1] > 0
    assert size(desc(), dg=0)[0] == 0
    assert size(desc(), dg=1)[1] > size(desc(), dg=0)[1]
    assert size(desc(Hk=4), dg=0)[1] < size(desc(), dg=0)[1]  # shared heads need partial sums
    for kw, want in ((dict(B=-1), "GDR_E_SHAPE"), (dict(T=-1), "GDR_E_SHAPE"), (dict(H=5), "GDR_E_SHAPE"),
                     (dict(Hk=0), "GDR_E_SHAPE"), (dict(Dk=12), "GDR_E_UNSUPPORTED"), (dict(Dk=264), "GDR_E_UNSUPPORTED"),
                     (dict(Dv=0), "GDR_E_UNSUPPORTED"), (dict(scale=float("nan")), "GDR_E_MODE"),
                     (dict(B=2 ** 30, T=2 ** 30, H=1024, Hk=1024), "GDR_E_SHAPE")):
        assert size(desc(**kw))[0] == E[want], kw
        assert size(desc(**kw), dg=1)[0] == E[want], kw
    d = desc()
    d.dtype = 7
    assert size(d)[0] == E["GDR_E_MODE"]
    lib = gdr.load_library()
    assert lib.gdr_head_decay_fwd_workspace_size(None, 0, ctypes.byref(ctypes.c_size_t())) == E["GDR_E_NULL"]
    assert lib.gdr_head_decay_fwd_workspace_size(ctypes.byref(d), 0, None) == E["GDR_E_NULL"]


def fwd(d, cu=None, q=P(1), k=P(2), v=P(3), g=P(4), s0=P(5), o=P(6), sf=P(7), ws=P(8), n=None):
    n = size(d, int(cu is not None))[1] if n is None else n
    return gdr.load_library().gdr_head_decay_fwd(ctypes.byref(d), cu, q, k, v, g, s0, o, sf, ws, n, None)


def test_forward_refusals():
    d = desc(T=2000, B=1)
    for kw in (dict(q=None), dict(k=None), dict(v=None), dict(g=None), dict(o=None)):
        assert fwd(d, **kw) == E["GDR_E_NULL"], kw
    assert fwd(d, ws=None) == E["GDR_E_WORKSPACE"]
    assert fwd(d, n=size(d)[1] - 1) == E["GDR_E_WORKSPACE"]
    for kw in (dict(q=P(1, 8)), dict(k=P(2, 2)), dict(v=P(3, 4)), dict(g=P(4, 2)), dict(s0=P(5, 4)), dict(o=P(6, 8)),
               dict(sf=P(7, 8)), dict(ws=P(8, 8)), dict(cu=P(9, 2))):
        assert fwd(d, **kw) == E["GDR_E_ALIGN"], kw
    assert fwd(d, o=P(1)) == E["GDR_E_ALIAS"]
    assert fwd(d, o=P(6), sf=P(6, 1024)) == E["GDR_E_ALIAS"]
    assert fwd(d, sf=P(5, 16)) == E["GDR_E_ALIAS"]          # s0 and s_final overlap in part
    assert fwd(d, ws=P(2, 4096)) == E["GDR_E_ALIAS"]
    assert fwd(d, cu=P(6)) == E["GDR_E_ALIAS"]
    # strides: negative, rows off 16 bytes, the reach of a view counted in the overlaps
    assert fwd(desc(T=2000, B=1, q_stride=(0, -256, 64))) == E["GDR_E_SHAPE"]
    assert fwd(desc(T=2000, B=1, k_stride=(0, 132, 64))) == E["GDR_E_ALIGN"]
    far = desc(T=2000, B=1, v_stride=(0, 1 << 20, 96))
    assert fwd(far, o=P(3, 2 * (1 << 20) * 1000)) == E["GDR_E_ALIAS"]
    assert fwd(desc(T=2000, B=1, v_stride=(0, 1 << 60, 96))) == E["GDR_E_SHAPE"]
    assert fwd(desc(H=5)) == E["GDR_E_SHAPE"]


def bwd(d, cu=None, q=P(1), k=P(2), v=P(3), g=P(4), s0=P(5), do=P(6), dsf=P(7), dq=P(8), dk=P(9), dv=P(10), dg=P(11),
        ds0=P(12), ws=P(13), n=None):
    n = size(d, int(cu is not None), int(dg is not None))[1] if n is None else n
    return gdr.load_library().gdr_head_decay_bwd(ctypes.byref(d), cu, q, k, v, g, s0, do, dsf, dq, dk, dv, dg, ds0, ws,
                                                 n, None)


def test_backward_refusals():
    d = desc()
    for kw in (dict(q=None), dict(k=None), dict(v=None), dict(g=None), dict(do=None), dict(dq=None), dict(dk=None),
               dict(dv=None)):
        assert bwd(d, **kw) == E["GDR_E_NULL"], kw
    assert bwd(d, ws=None) == E["GDR_E_WORKSPACE"]
    assert bwd(d, n=size(d, dg=0)[1]) == E["GDR_E_WORKSPACE"]  # without the chunk states that dg needs
    for kw in (dict(do=P(6, 8)), dict(dsf=P(7, 8)), dict(dq=P(8, 8)), dict(dk=P(9, 8)), dict(dv=P(10, 8)),
               dict(dg=P(11, 2)), dict(ds0=P(12, 8)), dict(ws=P(13, 8))):
        assert bwd(d, **kw) == E["GDR_E_ALIGN"], kw
    for kw in (dict(dq=P(1)), dict(dk=P(8)), dict(dv=P(6)), dict(dg=P(4)), dict(ds0=P(7)), dict(ws=P(5)),
               dict(ds0=P(5))):
        assert bwd(d, **kw) == E["GDR_E_ALIAS"], kw
    assert bwd(desc(do_stride=(4 * 96, 4, 96))) == E["GDR_E_ALIGN"]


def step(d, M=2, q=P(1), k=P(2), v=P(3), g=P(4), st=P(5), slots=None, parents=None, out=None, o=P(6)):
    return gdr.load_library().gdr_head_decay_step(ctypes.byref(d), q, k, v, g, st, M, slots, parents, out, o, None)


def test_step_refusals():
    d = desc(T=1)
    for kw in (dict(q=None), dict(k=None), dict(v=None), dict(g=None), dict(st=None), dict(o=None)):
        assert step(d, **kw) == E["GDR_E_NULL"], kw
    assert step(d, M=3) == E["GDR_E_SHAPE"]                    # in place, one state per row
    assert step(d, M=-1, slots=P(7)) == E["GDR_E_SHAPE"]
    assert step(d, M=1, out=P(7)) == E["GDR_E_SHAPE"]
    assert step(d, parents=P(7)) == E["GDR_E_MODE"]            # parents without state_out
    assert step(d, slots=P(7), out=P(8)) == E["GDR_E_MODE"]    # slots with it
    assert step(d, st=P(5, 8)) == E["GDR_E_ALIGN"]
    assert step(d, slots=P(7, 2)) == E["GDR_E_ALIGN"]
    assert step(d, out=P(7, 8)) == E["GDR_E_ALIGN"]
    assert step(d, out=P(5, 1024)) == E["GDR_E_ALIAS"]
    assert step(d, o=P(5)) == E["GDR_E_ALIAS"]
    assert step(d, parents=P(7), out=P(7)) == E["GDR_E_ALIAS"]
    assert step(desc(Dv=100)) == E["GDR_E_UNSUPPORTED"]


def select(B=2, K=4, V=1000, dt=0, x=P(1), stride=1000, s=P(2), done=P(3), eos=1, pad=0, os=P(4), ot=P(5), op=P(6),
           od=P(7), ws=P(8), n=None):
    lib = gdr.load_library()
    need = ctypes.c_size_t(0)
    lib.gdr_beam_select_workspace_size(B, K, V, ctypes.byref(need))
    return lib.gdr_beam_select(B, K, V, dt, x, stride, s, done, eos, pad, os, ot, op, od, ws,
                               need.value if n is None else n, None)


def test_select_refusals():
    for kw, want in ((dict(B=-1), "SHAPE"), (dict(K=0), "SHAPE"), (dict(V=0), "SHAPE"), (dict(K=33), "UNSUPPORTED"),
                     (dict(V=2 ** 30 + 1, K=1), "UNSUPPORTED"), (dict(V=2 ** 28, K=8), "SHAPE"),
                     (dict(B=2 ** 30), "SHAPE"), (dict(dt=5), "MODE"), (dict(pad=1000), "MODE"), (dict(pad=-1), "MODE"),
                     (dict(stride=-1), "SHAPE"), (dict(x=None), "NULL"), (dict(s=None), "NULL"), (dict(os=None), "NULL"),
                     (dict(ot=None), "NULL"), (dict(op=None), "NULL"), (dict(od=None), "NULL"),
                     (dict(ws=None), "WORKSPACE"), (dict(n=8), "WORKSPACE"), (dict(x=P(1, 2)), "ALIGN"),
                     (dict(x=P(1, 1), dt=1), "ALIGN"), (dict(ot=P(5, 1)), "ALIGN"), (dict(ws=P(8, 8)), "ALIGN"),
                     (dict(os=P(2)), "ALIAS"), (dict(od=P(3)), "ALIAS"), (dict(ws=P(1, 16)), "ALIAS"),
                     (dict(ot=P(6)), "ALIAS")):
        assert select(**kw) == E["GDR_E_" + want], kw


def test_reorder_refusals():
    lib = gdr.load_library()

    def call(L=1, B=2, K=4, row=1024, st=P(1), p=P(2), out=P(1)):
        return lib.gdr_beam_reorder(L, B, K, row, st, p, out, None)

    for kw, want in ((dict(L=-1), "SHAPE"), (dict(B=-1), "SHAPE"), (dict(K=0), "SHAPE"), (dict(K=33), "UNSUPPORTED"),
                     (dict(row=-16), "SHAPE"), (dict(row=24), "ALIGN"), (dict(row=2 ** 60), "SHAPE"),
                     (dict(st=None), "NULL"), (dict(p=None), "NULL"), (dict(out=None), "NULL"),
                     (dict(st=P(1, 8)), "ALIGN"), (dict(p=P(2, 2)), "ALIGN"), (dict(out=P(1, 1024)), "ALIAS"),
                     (dict(p=P(1, 64)), "ALIAS")):
        assert call(**kw) == E["GDR_E_" + want], kw


def test_python_checks():
    x = torch.zeros(1, 4, 2, 8)
    with pytest.raises(ValueError, match="GPU tensor"):
        gdr.head_decay_fwd(x, x, x, torch.zeros(2))
    with pytest.raises(TypeError):
        gdr.head_decay_fwd(None, x, x, torch.zeros(2))
    with pytest.raises(TypeError):
        gdr.head_decay_fwd_varlen(x[0], x[0], x[0], torch.zeros(2), None)
    with pytest.raises(ValueError, match="GPU tensor"):
        gdr.head_decay_step(x[0], x[0], x[0], torch.zeros(2), torch.zeros(4, 2, 8, 8))
    with pytest.raises(ValueError, match="GPU tensor"):
        gdr.beam_select(torch.zeros(1, 2, 3), torch.zeros(1, 2))
    with pytest.raises(ValueError, match="GPU tensor"):
        gdr.beam_reorder(torch.zeros(1, 2, 8), torch.zeros(1, 2, dtype=torch.int32))
