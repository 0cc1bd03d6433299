"""The paged 8-bit cache's C entry points without a GPU: descriptor layouts,
workspace sizes, and the refusals, each of which happens on the host before
anything is launched; and the binding's own argument checks."""
import ctypes
import os
import re

import pytest
import torch

import graph_community_sparse_b200 as ckv
from test_abi import CAPACITY, CUDA, FAKE, HEADER, INVALID, MISALIGNED, OK, UNSUPPORTED, WORKSPACE, _graph, _sel


def test_struct_layouts_match_header_order():
    src = open(HEADER).read()
    for cls, tag in [(ckv.TableDesc, "ckv_table_desc"), (ckv.Q8Desc, "ckv_q8_desc"), (ckv.PlanDesc, "ckv_plan_desc")]:
        body = re.search(r"typedef struct \{([^{}]*)\}\s*" + tag + ";", src).group(1)
        body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
        assert [f[0] for f in cls._fields_] == re.findall(r"\**\s*(\w+)\s*(?=[,;])", body), tag


def test_constants_match_header():
    src = open(HEADER).read()
    for name, val in [("CKV_DEVERR_PLAN", ckv.DEVERR_PLAN), ("CKV_DEVERR_BLOCK", ckv.DEVERR_BLOCK)]:
        assert int(re.search(rf"#define {name} (\d+)", src).group(1)) == val
    for name, val in [("CKV_Q8_INT8", ckv.Q8_INT8), ("CKV_Q8_E4M3", ckv.Q8_E4M3)]:
        assert int(re.search(rf"\b{name} = (\d+)", src).group(1)) == val


def _table(**kw):
    t = dict(B=2, block=64, n_blocks=100, max_blocks=64)
    for i, f in enumerate(["table", "len", "free_list", "n_free", "dev_err"]):
        t[f] = FAKE + (i + 1) * (1 << 20)
    t.update(kw)
    return ckv.TableDesc(**t)


def _q8(table=None, **kw):
    c = dict(format=0, dtype=1, Hkv=8, Hq=32, d=128)
    for i, f in enumerate(["k", "v", "k_scale", "v_scale"]):
        c[f] = FAKE + (i + 1) * (1 << 28)
    c.update(kw)
    return ckv.Q8Desc(blocks=table or _table(), **c)


def _pl(**kw):
    p = dict(n_rows=10, start=FAKE, slot=FAKE, granted=FAKE)
    p.update(kw)
    return ckv.PlanDesc(**p)


R = ctypes.byref


def _plan(table=None, plan=None, add=FAKE):
    return ckv.lib.ckv_plan_blocks(R(table or _table()), add, R(plan or _pl()), None)


def _append(cache=None, plan=None, k=FAKE, v=FAKE, T_rows=0, sb=0, st=1024, sh=128):
    return ckv.lib.ckv_quant_append(R(cache or _q8()), R(plan or _pl()), k, v, T_rows, sb, st, sh, None)


def _read(cache=None, rows=4, k=FAKE, v=FAKE, sb=4096, sh=512, st=128):
    return ckv.lib.ckv_q8_read(R(cache or _q8()), None, rows, k, v, sb, sh, st, None)


def _dense(cache=None, q=FAKE, out=FAKE, ws=FAKE, n=1 << 40):
    return ckv.lib.ckv_dense_decode_q8(R(cache or _q8()), q, out, ws, n, None)


def _sparse(cache=None, graph=None, sel=None, q=FAKE, out=FAKE, k_new=None, ws=FAKE, n=1 << 40):
    return ckv.lib.ckv_sparse_decode_q8(R(cache or _q8()), q, R(graph or _graph()), R(sel or _sel()), out, None, k_new,
                                        None, ws, n, None)


CASES = [
    ("plan B 0", lambda: _plan(_table(B=0)), INVALID),
    ("plan B above", lambda: _plan(_table(B=8193)), UNSUPPORTED),
    ("plan block", lambda: _plan(_table(block=48)), UNSUPPORTED),
    ("plan block 8", lambda: _plan(_table(block=8)), UNSUPPORTED),
    ("plan n_blocks", lambda: _plan(_table(n_blocks=0)), INVALID),
    ("plan max_blocks", lambda: _plan(_table(max_blocks=0)), INVALID),
    ("plan slots past 31 bits", lambda: _plan(_table(n_blocks=1 << 25)), UNSUPPORTED),
    ("plan positions past 31 bits", lambda: _plan(_table(max_blocks=1 << 25)), UNSUPPORTED),
    ("plan null table", lambda: _plan(_table(table=None)), INVALID),
    ("plan null len", lambda: _plan(_table(len=None)), INVALID),
    ("plan null dev_err", lambda: _plan(_table(dev_err=None)), INVALID),
    ("plan null free list", lambda: _plan(_table(free_list=None)), INVALID),
    ("plan null n_free", lambda: _plan(_table(n_free=None)), INVALID),
    ("plan null add", lambda: _plan(add=None), INVALID),
    ("plan rows < 0", lambda: _plan(plan=_pl(n_rows=-1)), INVALID),
    ("plan null start", lambda: _plan(plan=_pl(start=None)), INVALID),
    ("plan null slot", lambda: _plan(plan=_pl(slot=None)), INVALID),
    ("plan null granted", lambda: _plan(plan=_pl(granted=None)), INVALID),
    ("append format", lambda: _append(_q8(format=2)), UNSUPPORTED),
    ("append dtype", lambda: _append(_q8(dtype=2)), UNSUPPORTED),
    ("append d", lambda: _append(_q8(d=96)), UNSUPPORTED),
    ("append ratio", lambda: _append(_q8(Hq=48)), UNSUPPORTED),
    ("append Hq % Hkv", lambda: _append(_q8(Hq=30)), INVALID),
    ("append pool past 31 bits", lambda: _append(_q8(_table(n_blocks=1 << 22))), UNSUPPORTED),
    ("append units", lambda: _append(_q8(_table(B=8192))), UNSUPPORTED),
    ("append null pool", lambda: _append(_q8(v=None)), INVALID),
    ("append null scale", lambda: _append(_q8(k_scale=None)), INVALID),
    ("append misaligned pool", lambda: _append(_q8(k=FAKE + 8)), MISALIGNED),
    ("append null rows", lambda: _append(k=None), INVALID),
    ("append misaligned rows", lambda: _append(v=FAKE + 2), MISALIGNED),
    ("append misaligned stride", lambda: _append(st=1025), MISALIGNED),
    ("append negative stride", lambda: _append(sh=-128), INVALID),
    ("append T_rows < 0", lambda: _append(T_rows=-1), INVALID),
    ("read R < 0", lambda: _read(rows=-1), INVALID),
    ("read null", lambda: _read(v=None), INVALID),
    ("read misaligned", lambda: _read(k=FAKE + 8), MISALIGNED),
    ("read R above", lambda: _read(rows=(1 << 30) + 1), UNSUPPORTED),
    ("read overlapping rows", lambda: _read(st=64), INVALID),
    ("dense null q", lambda: _dense(q=None), INVALID),
    ("dense misaligned q", lambda: _dense(q=FAKE + 8), MISALIGNED),
    ("dense misaligned out", lambda: _dense(out=FAKE + 4), MISALIGNED),
    ("dense null ws", lambda: _dense(ws=None), WORKSPACE),
    ("dense small ws", lambda: _dense(n=4096), WORKSPACE),
    ("dense misaligned ws", lambda: _dense(ws=FAKE + 128), WORKSPACE),
    ("dense too many tiles", lambda: _dense(_q8(_table(B=512, max_blocks=1 << 20))), UNSUPPORTED),
    ("sparse T_cap", lambda: _sparse(graph=_graph(T_cap=8192), sel=_sel()), CAPACITY),
    ("sparse T_cap 0", lambda: _sparse(graph=_graph(T_cap=0, S=0), sel=_sel()), INVALID),
    ("sparse mode", lambda: _sparse(graph=_graph(mode=3)), INVALID),
    ("sparse null sel", lambda: _sparse(sel=_sel(sel_tok=None)), INVALID),
    ("sparse misaligned k_new", lambda: _sparse(k_new=FAKE + 2), MISALIGNED),
    ("sparse small ws", lambda: _sparse(n=1 << 20), WORKSPACE),
]


@pytest.mark.parametrize("name,call,status", CASES, ids=[c[0] for c in CASES])
def test_refusals(name, call, status):
    got = call()
    assert got not in (OK, CUDA)
    assert got == status, ckv.ckv_last_error()
    assert ckv.ckv_last_error()


@pytest.mark.parametrize("fn", ["ckv_plan_blocks", "ckv_quant_append", "ckv_q8_read", "ckv_dense_decode_q8",
                                "ckv_sparse_decode_q8"])
def test_null_descriptors(fn):
    f = getattr(ckv.lib, fn)
    args = [None if t is not ctypes.c_int32 and t is not ctypes.c_int64 and t is not ctypes.c_size_t else 0
            for t in f.argtypes]
    assert f(*args) == INVALID


def test_nothing_to_do_is_ok_without_a_launch():
    assert _append(plan=_pl(n_rows=0, slot=None)) == OK
    assert _read(rows=0) == OK


def test_workspace_size():
    out = ctypes.c_size_t(0)
    assert ckv.lib.ckv_q8_workspace_size(R(_q8()), None, None, R(out)) == OK
    dense = out.value
    assert dense > 256
    assert ckv.lib.ckv_q8_workspace_size(R(_q8()), R(_graph()), R(_sel()), R(out)) == OK
    assert out.value >= dense
    assert ckv.lib.ckv_q8_workspace_size(R(_q8(d=80)), None, None, R(out)) == UNSUPPORTED
    assert ckv.lib.ckv_q8_workspace_size(R(_q8()), None, None, None) == INVALID


# ---------------------------------------------------------------------------
# the binding
# ---------------------------------------------------------------------------

def _cpu_cache(**kw):
    a = dict(B=2, Hkv=2, Hq=4, d=64, n_blocks=8, block=16, max_blocks=4, device="cpu")
    a.update(kw)
    return ckv.new_q8_cache(**a)


def test_binding_builds_descriptors():
    c = _cpu_cache(fmt="e4m3", dtype=torch.float32)
    assert (c.desc.format, c.desc.dtype, c.desc.blocks.B, c.desc.blocks.max_blocks) == (1, 0, 2, 4)
    assert c.k.dtype == torch.float8_e4m3fn and c.k.shape == (8, 2, 16, 64)
    assert c.blocks.free_list[int(c.blocks.n_free) - 1] == 0 and (c.table == -1).all()
    assert c.desc.blocks.dev_err == c.dev_err.data_ptr()


@pytest.mark.parametrize("bad", [
    lambda c: ckv.q8_cache(c.k.view(torch.uint8), c.v, c.k_scale, c.v_scale, c.table, c.len, 4),
    lambda c: ckv.q8_cache(c.k, c.v[:4], c.k_scale, c.v_scale, c.table, c.len, 4),
    lambda c: ckv.q8_cache(c.k, c.v, c.k_scale.double(), c.v_scale, c.table, c.len, 4),
    lambda c: ckv.q8_cache(c.k, c.v, c.k_scale, c.v_scale, c.table.long(), c.len, 4),
    lambda c: ckv.q8_cache(c.k, c.v, c.k_scale, c.v_scale, c.table, c.len[:1], 4),
    lambda c: ckv.q8_cache(c.k.transpose(2, 3), c.v, c.k_scale, c.v_scale, c.table, c.len, 4),
    lambda c: ckv.q8_cache(c.k, c.v, c.k_scale, c.v_scale, c.table, c.len, 4, torch.float16),
    lambda c: ckv.new_q8_cache(2, 2, 4, 64, 8, fmt="int4", device="cpu"),
    lambda c: ckv.Plan(torch.zeros(2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)),
    lambda c: ckv.ckv_plan_blocks(c, torch.zeros(3, dtype=torch.int32), ckv.new_plan(c, 4)),
    lambda c: ckv.ckv_plan_blocks(c, torch.zeros(2, dtype=torch.int64), ckv.new_plan(c, 4)),
    lambda c: ckv.ckv_plan_blocks(c, torch.zeros(2, dtype=torch.int32), ckv.new_plan(_cpu_cache(B=3), 4)),
    lambda c: ckv.ckv_plan_blocks(c, torch.zeros(2, dtype=torch.int32), ckv.new_plan(c, 4)),  # not on a GPU
    lambda c: ckv.ckv_quant_append(c, ckv.new_plan(c, 3), torch.zeros(3, 2, 64), torch.zeros(3, 2, 64)),  # dtype
    lambda c: ckv.ckv_quant_append(c, ckv.new_plan(c, 3), *[torch.zeros(4, 2, 64, dtype=torch.bfloat16)] * 2),
    lambda c: ckv.ckv_quant_append(c, ckv.new_plan(c, 3), *[torch.zeros(3, 64, dtype=torch.bfloat16)] * 2),
    lambda c: ckv.ckv_quant_append(c, ckv.new_plan(c, 3), torch.zeros(3, 2, 64, dtype=torch.bfloat16),
                                   torch.zeros(2, 3, 64, dtype=torch.bfloat16).transpose(0, 1)),
    lambda c: ckv.ckv_quant_append(c, ckv.new_plan(c, 3), *[torch.zeros(2, 0, 2, 64, dtype=torch.bfloat16)] * 2),
    lambda c: ckv.ckv_q8_read(c, *[torch.zeros(2, 2, 5, 32, dtype=torch.bfloat16)] * 2),
    lambda c: ckv.ckv_q8_read(c, *[torch.zeros(2, 2, 5, 64, dtype=torch.bfloat16)] * 2, first=torch.zeros(2)),
    lambda c: ckv.ckv_dense_decode_q8(c, torch.zeros(2, 4, 64), torch.zeros(2, 4, 64), torch.zeros(9, dtype=torch.uint8)),
    lambda c: ckv.ckv_dense_decode_q8(c, torch.zeros(2, 4, 64, dtype=torch.bfloat16), torch.zeros(2, 4, 128)[:, :, ::2],
                                      torch.zeros(9, dtype=torch.uint8)),
])
def test_binding_refuses(bad):
    with pytest.raises(ValueError):
        bad(_cpu_cache())
