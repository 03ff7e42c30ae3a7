"""The computing operators' C ABI and binding without a GPU: exports, sizes,
and refusals before any HIP call (addresses are never dereferenced)."""
import ctypes
import os
import re

import pytest
import torch

import combine_get_dispatch_06_amd as cgd

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000


def _vp(v):
    return None if v is None else ctypes.c_void_p(v)


def test_header_declares_the_operators_and_the_library_has_them():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "cgd_experts.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(cgd_[a-z_0-9]+)\s*\(", text)))
    assert names == sorted([
        "cgd_route", "cgd_route_backward", "cgd_linear", "cgd_linear_workspace_bytes", "cgd_grouped_linear",
        "cgd_grouped_linear_workspace_bytes", "cgd_linear_backward", "cgd_linear_backward_workspace_bytes",
        "cgd_grouped_linear_backward", "cgd_grouped_linear_backward_workspace_bytes"])
    lib = cgd.load()
    for n in names:
        assert hasattr(lib, n), n


def _route(**kw):
    a = dict(logits=FAKE, lt=1, T=16, E=64, K=8, mode=0, bias=None, G=1, KG=1, top=1, ren=1, scale=1.0, idx=FAKE, w=FAKE)
    a.update(kw)
    return cgd.load().cgd_route(_vp(a["logits"]), a["lt"], a["T"], a["E"], a["K"], a["mode"], _vp(a["bias"]), a["G"],
                                a["KG"], a["top"], a["ren"], a["scale"], _vp(a["idx"]), _vp(a["w"]), None)


@pytest.mark.parametrize("kw", [dict(T=-1), dict(T=1 << 31), dict(E=0), dict(E=513), dict(K=0), dict(K=17), dict(K=9, E=8),
                                dict(lt=2), dict(mode=2), dict(G=0), dict(G=3), dict(E=256, G=128, KG=128), dict(KG=0),
                                dict(G=4, KG=5), dict(G=8, KG=1, K=9, E=64), dict(top=0), dict(top=3),
                                dict(logits=None), dict(idx=None), dict(w=None), dict(logits=FAKE + 2),
                                dict(idx=FAKE + 4), dict(w=FAKE + 2), dict(bias=FAKE + 2)])
def test_route_refuses(kw):
    assert _route(**kw) == -1
    assert cgd.load().cgd_last_error()


@pytest.mark.parametrize("kw", [dict(T=-1), dict(E=513), dict(K=0), dict(lt=3), dict(mode=-1), dict(g=None), dict(l=None),
                                dict(idx=None), dict(out=None), dict(out=FAKE + 1), dict(idx=FAKE + 4)])
def test_route_backward_refuses(kw):
    a = dict(g=FAKE, l=FAKE, lt=1, idx=FAKE, T=16, E=64, K=8, mode=0, out=FAKE)
    a.update(kw)
    rc = cgd.load().cgd_route_backward(_vp(a["g"]), _vp(a["l"]), a["lt"], _vp(a["idx"]), a["T"], a["E"], a["K"],
                                       a["mode"], 1, 1.0, _vp(a["out"]), None)
    assert rc == -1


def _linear(grouped=False, **kw):
    a = dict(x=FAKE, xt=0, xs=None, st=0, sb=0, fmt=0, w=FAKE, ws=None, T=4096, G=4, off=FAKE, cap=0, cnt=None, I=4096,
             O=4096, b=None, act=0, res=None, out=FAKE, ot=0, pre=None, wk=None, wb=0)
    a.update(kw)
    lib = cgd.load()
    head = (_vp(a["x"]), a["xt"], _vp(a["xs"]), a["st"], a["sb"], a["fmt"], _vp(a["w"]), _vp(a["ws"]), a["T"])
    if grouped:
        return lib.cgd_grouped_linear(*head, a["G"], _vp(a["off"]), a["cap"], _vp(a["cnt"]), a["I"], a["O"], _vp(a["b"]),
                                      a["act"], _vp(a["out"]), _vp(a["pre"]), _vp(a["wk"]), a["wb"], None)
    return lib.cgd_linear(*head, a["I"], a["O"], _vp(a["b"]), a["act"], _vp(a["res"]), _vp(a["out"]), a["ot"],
                          _vp(a["pre"]), _vp(a["wk"]), a["wb"], None)


COMMON = [dict(T=-1), dict(T=1 << 31), dict(xt=1), dict(xt=3), dict(I=0), dict(I=12), dict(I=(1 << 20) + 8), dict(O=0),
          dict(O=(1 << 19) + 1), dict(act=-1), dict(act=5), dict(x=None), dict(w=None), dict(out=None),
          dict(x=FAKE + 2), dict(w=FAKE + 8), dict(out=FAKE + 4), dict(pre=FAKE + 2), dict(b=FAKE + 1),
          dict(xt=2, I=4096 + 8), dict(xt=2), dict(xt=2, ws=FAKE), dict(xt=2, xs=FAKE, ws=FAKE, fmt=3),
          dict(xt=2, xs=FAKE, ws=FAKE, st=-1), dict(xt=2, xs=FAKE, ws=FAKE, st=1 << 21),
          dict(xt=2, xs=FAKE + 2, ws=FAKE), dict(xt=2, xs=FAKE, ws=FAKE, act=4, O=100), dict(O=1 << 19, T=(1 << 31) - 1)]


@pytest.mark.parametrize("kw", COMMON + [dict(ot=2), dict(ot=1, xt=2, xs=FAKE, ws=FAKE), dict(res=FAKE + 2)])
def test_linear_refuses(kw):
    assert _linear(**kw) == -1
    assert cgd.load().cgd_last_error()


@pytest.mark.parametrize("kw", COMMON + [dict(G=0), dict(G=513), dict(off=FAKE + 2), dict(cnt=FAKE + 1),
                                         dict(off=None, cap=1000), dict(off=None, cap=-1)])
def test_grouped_linear_refuses(kw):
    assert _linear(grouped=True, **kw) == -1


def test_split_products_need_their_workspace():
    lib = cgd.load()
    need = lib.cgd_linear_workspace_bytes(128, 7168, 256, 0, 0)
    assert need > 0 and _linear(T=128, I=7168, O=256) == -3
    assert _linear(T=128, I=7168, O=256, wk=FAKE, wb=need - 1) == -3
    assert _linear(T=128, I=7168, O=256, wk=FAKE + 64, wb=need) == -3
    assert lib.cgd_linear_workspace_bytes(4096, 4096, 4096, 0, 0) == 0
    assert lib.cgd_linear_workspace_bytes(128, 7167, 256, 0, 0) == 0
    assert lib.cgd_grouped_linear_workspace_bytes(1024, 600, 0, 4096, 4096, 0, 0) == 0
    assert lib.cgd_linear_backward_workspace_bytes(100, 64, 64, 0, 0) == 0          # d is grad_out itself
    assert lib.cgd_linear_backward_workspace_bytes(100, 64, 60, 0, 0) >= 100 * 64 * 2  # rows are padded to 16 bytes
    assert lib.cgd_linear_backward_workspace_bytes(100, 64, 64, 4, 0) >= 100 * 128 * 2
    assert lib.cgd_grouped_linear_backward_workspace_bytes(100, 4, 64, 64, 0, 1) > 0


@pytest.mark.parametrize("kw", [dict(T=-1), dict(I=4), dict(O=0), dict(act=7), dict(g=None), dict(x=None), dict(w=None),
                                dict(act=1), dict(g=FAKE + 2), dict(gx=FAKE + 2), dict(gw=FAKE + 8), dict(gb=FAKE + 1)])
@pytest.mark.parametrize("grouped", [False, True])
def test_backward_refuses(grouped, kw):
    a = dict(g=FAKE, x=FAKE, w=FAKE, T=128, I=64, O=64, pre=None, act=0, gx=FAKE, gw=FAKE, gb=None)
    a.update(kw)
    lib = cgd.load()
    tail = (a["I"], a["O"], _vp(a["pre"]), a["act"], _vp(a["gx"]), _vp(a["gw"]), _vp(a["gb"]), None, 0, None)
    head = (_vp(a["g"]), _vp(a["x"]), _vp(a["w"]), a["T"])
    rc = lib.cgd_grouped_linear_backward(*head, 4, _vp(FAKE), 0, None, *tail) if grouped else \
        lib.cgd_linear_backward(*head, *tail)
    assert rc == -1


def test_backward_needs_its_workspace():
    lib = cgd.load()
    rc = lib.cgd_linear_backward(_vp(FAKE), _vp(FAKE), _vp(FAKE), 128, 64, 64, _vp(FAKE), 2, _vp(FAKE), _vp(FAKE), None,
                                 None, 0, None)
    assert rc == -3


def test_binding_refuses_host_tensors_and_bad_choices():
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(8, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        cgd.linear(x, w)
    with pytest.raises(ValueError, match="GPU"):
        cgd.grouped_linear(x, w[None], torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="GPU"):
        cgd.linear_backward(x, x, w)
    with pytest.raises(ValueError, match="GPU"):
        cgd.route(torch.zeros(4, 8), 2)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        cgd.route(torch.zeros(4, 8, dtype=torch.float16), 2)
    with pytest.raises(TypeError):
        cgd.linear((x,), w)
