"""The C ABI and binding of the norm, the adapters, dropout and combine's gradient
without a GPU: exports, sizes, and refusals before any HIP call (addresses are
never dereferenced); the generator that the dropout tests compare with, against
the published vectors."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import combine_get_dispatch_06_amd as cgd
from philox import kept, words

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000


def _vp(v):
    return None if v is None else ctypes.c_void_p(v)


def test_header_declares_the_operators_and_the_library_has_them():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "cgd_layer.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(cgd_[a-z_0-9]+)\s*\(", text)))
    assert names == sorted([
        "cgd_rms_norm", "cgd_rms_norm_backward", "cgd_rms_norm_backward_workspace_bytes", "cgd_adapter_linear",
        "cgd_adapter_linear_workspace_bytes", "cgd_adapter_linear_backward",
        "cgd_adapter_linear_backward_workspace_bytes", "cgd_dropout", "cgd_combine_backward"])
    lib = cgd.load()
    for n in names:
        assert hasattr(lib, n), n
    for n in ("rms_norm", "rms_norm_backward", "adapter_linear", "adapter_linear_backward", "dropout",
              "dropout_backward", "combine_backward"):
        assert n in cgd.__all__ and callable(getattr(cgd, n))


@pytest.mark.parametrize("kw", [dict(n=-1), dict(n=1 << 31), dict(H=0), dict(H=12), dict(H=32776), dict(wt=2), dict(eps=-1.0),
                                dict(eps=float("nan")), dict(eps=float("inf")), dict(x=None), dict(w=None), dict(y=None),
                                dict(q=FAKE), dict(sc=FAKE), dict(sum=FAKE), dict(x=FAKE + 8), dict(y=FAKE + 2),
                                dict(res=FAKE + 4), dict(w=FAKE + 8), dict(res=FAKE, sum=FAKE + 8),
                                dict(q=FAKE, sc=FAKE, H=72), dict(q=FAKE, sc=FAKE, fmt=3), dict(q=FAKE, sc=FAKE, fmt=-1),
                                dict(q=FAKE, sc=FAKE + 2), dict(q=FAKE + 8, sc=FAKE)])
def test_norm_refuses(kw):
    a = dict(x=FAKE, res=None, w=FAKE, wt=0, eps=1e-6, n=4, H=128, y=FAKE, q=None, sc=None, fmt=0, sum=None)
    a.update(kw)
    rc = cgd.load().cgd_rms_norm(_vp(a["x"]), _vp(a["res"]), _vp(a["w"]), a["wt"], a["eps"], a["n"], a["H"], _vp(a["y"]),
                                 _vp(a["q"]), _vp(a["sc"]), a["fmt"], _vp(a["sum"]), None)
    assert rc == -1 and cgd.load().cgd_last_error()


@pytest.mark.parametrize("kw,want", [(dict(n=-1), -1), (dict(H=20), -1), (dict(wt=3), -1), (dict(g=None), -1),
                                     (dict(x=None), -1), (dict(w=None), -1), (dict(g=FAKE + 2), -1), (dict(gs=FAKE + 8), -1),
                                     (dict(gx=FAKE + 4), -1), (dict(gw=FAKE + 1), -1), (dict(wt=1, gw=FAKE + 2), -1),
                                     (dict(wb=0), -3), (dict(wk=None), -3), (dict(wk=FAKE + 64), -3)])
def test_norm_backward_refuses(kw, want):
    lib = cgd.load()
    need = lib.cgd_rms_norm_backward_workspace_bytes(100, 128)
    assert need > 0 and lib.cgd_rms_norm_backward_workspace_bytes(100, 12) == 0
    a = dict(g=FAKE, x=FAKE, w=FAKE, wt=0, n=100, H=128, gs=None, gx=FAKE, gw=FAKE, wk=FAKE, wb=need)
    a.update(kw)
    rc = lib.cgd_rms_norm_backward(_vp(a["g"]), _vp(a["x"]), _vp(a["w"]), a["wt"], 1e-6, a["n"], a["H"], _vp(a["gs"]),
                                   _vp(a["gx"]), _vp(a["gw"]), _vp(a["wk"]), a["wb"], None)
    assert rc == want


SIZES = [(dict(T=-1), -1), (dict(T=(1 << 26) + 1), -1), (dict(J=0), -1), (dict(J=513), -1), (dict(R=0), -1), (dict(R=12), -1),
         (dict(R=264), -1), (dict(I=0), -1), (dict(I=36), -1), (dict(I=(1 << 20) + 8), -1), (dict(O=0), -1),
         (dict(O=(1 << 20) + 8), -1), (dict(a=None), -1), (dict(b=None), -1), (dict(idx=None), -1), (dict(x=FAKE + 8), -1),
         (dict(a=FAKE + 2), -1), (dict(b=FAKE + 4), -1), (dict(idx=FAKE + 4), -1), (dict(sc=FAKE + 2), -1), (dict(wb=0), -3),
         (dict(wk=None), -3), (dict(wk=FAKE + 128), -3)]


@pytest.mark.parametrize("kw,want", SIZES + [(dict(x=None), -1), (dict(out=None), -1), (dict(out=FAKE + 8), -1),
                                             (dict(res=FAKE + 2), -1), (dict(hid=FAKE + 4), -1)])
def test_adapters_refuse(kw, want):
    lib = cgd.load()
    need = lib.cgd_adapter_linear_workspace_bytes(100, 4, 16, 64, 60)
    assert need > 0 and lib.cgd_adapter_linear_workspace_bytes(0, 4, 16, 64, 60) == 0
    a = dict(x=FAKE, a=FAKE, b=FAKE, sc=None, idx=FAKE, T=100, J=4, R=16, I=64, O=60, res=None, out=FAKE, hid=None, wk=FAKE,
             wb=need)
    a.update(kw)
    rc = lib.cgd_adapter_linear(_vp(a["x"]), _vp(a["a"]), _vp(a["b"]), _vp(a["sc"]), _vp(a["idx"]), a["T"], a["J"], a["R"],
                                a["I"], a["O"], _vp(a["res"]), _vp(a["out"]), _vp(a["hid"]), _vp(a["wk"]), a["wb"], None)
    assert rc == want


@pytest.mark.parametrize("kw,want", SIZES + [(dict(O=60), -1), (dict(g=None), -1), (dict(g=FAKE + 2), -1), (dict(x=None), -1),
                                             (dict(hid=None), -1), (dict(hid=FAKE + 2), -1), (dict(gx=FAKE + 8), -1),
                                             (dict(ga=FAKE + 8), -1), (dict(gb=FAKE + 8), -1)])
def test_adapters_backward_refuse(kw, want):
    lib = cgd.load()
    a = dict(g=FAKE, x=FAKE, a=FAKE, b=FAKE, sc=None, idx=FAKE, hid=FAKE, T=100, J=4, R=16, I=64, O=64, gx=FAKE, ga=FAKE,
             gb=FAKE, wk=FAKE, wb=lib.cgd_adapter_linear_backward_workspace_bytes(100, 4, 16, 64, 64))
    a.update(kw)
    rc = lib.cgd_adapter_linear_backward(
        _vp(a["g"]), _vp(a["x"]), _vp(a["a"]), _vp(a["b"]), _vp(a["sc"]), _vp(a["idx"]), _vp(a["hid"]), a["T"], a["J"], a["R"],
        a["I"], a["O"], _vp(a["gx"]), _vp(a["ga"]), _vp(a["gb"]), _vp(a["wk"]), a["wb"], None)
    assert rc == want


@pytest.mark.parametrize("kw", [dict(n=-1), dict(p=-0.1), dict(p=1.1), dict(p=float("nan")), dict(x=None), dict(out=None),
                                dict(x=FAKE + 2), dict(res=FAKE + 8), dict(out=FAKE + 4), dict(state=FAKE + 4)])
def test_dropout_refuses(kw):
    a = dict(x=FAKE, res=None, n=100, p=0.5, state=None, out=FAKE)
    a.update(kw)
    rc = cgd.load().cgd_dropout(_vp(a["x"]), _vp(a["res"]), a["n"], a["p"], 1, 2, _vp(a["state"]), _vp(a["out"]), None)
    assert rc == -1


@pytest.mark.parametrize("kw", [dict(T=-1), dict(T=1 << 31), dict(K=0), dict(K=17), dict(H=0), dict(H=12), dict(cap=-1),
                                dict(cap=1 << 31), dict(g=None), dict(y=None), dict(dst=None), dict(w=None), dict(gy=None),
                                dict(gw=None), dict(g=FAKE + 8), dict(y=FAKE + 2), dict(gy=FAKE + 4), dict(dst=FAKE + 2),
                                dict(w=FAKE + 1), dict(gw=FAKE + 2)])
def test_combine_backward_refuses(kw):
    a = dict(g=FAKE, y=FAKE, cap=100, H=64, dst=FAKE, w=FAKE, T=10, K=8, gy=FAKE, gw=FAKE)
    a.update(kw)
    rc = cgd.load().cgd_combine_backward(_vp(a["g"]), _vp(a["y"]), a["cap"], a["H"], _vp(a["dst"]), _vp(a["w"]), a["T"], a["K"],
                                         _vp(a["gy"]), _vp(a["gw"]), None)
    assert rc == -1


def test_nothing_to_do_needs_no_pointers():
    lib = cgd.load()
    assert lib.cgd_rms_norm(None, None, _vp(FAKE), 0, 1e-6, 0, 128, None, None, None, 0, None, None) == 0
    assert lib.cgd_adapter_linear(None, _vp(FAKE), _vp(FAKE), None, None, 0, 4, 8, 64, 64, None, None, None, None, 0, None) == 0
    assert lib.cgd_dropout(None, None, 0, 0.5, 1, 2, None, None, None) == 0
    assert lib.cgd_combine_backward(None, None, 0, 64, None, None, 0, 8, None, None, None) == 0


def test_binding_refuses_host_tensors_and_types():
    x, w = torch.zeros(4, 128, dtype=torch.bfloat16), torch.zeros(128)
    i = torch.zeros(4, dtype=torch.int64)
    for call in (lambda: cgd.rms_norm(x, w), lambda: cgd.rms_norm_backward(x, x, w), lambda: cgd.dropout(x, 0.5, 1),
                 lambda: cgd.dropout_backward(x, 0.5, 1), lambda: cgd.adapter_linear(x, x[None], x[None], i),
                 lambda: cgd.adapter_linear_backward(x, x, x[None], x[None], i, x)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    h = cgd.DispatchHandle(i.int(), i.int(), i.int()[:, None], i.int(), 3, 1, 1, 4)
    with pytest.raises(ValueError, match="GPU"):
        cgd.combine_backward(x, x, h, torch.zeros(4, 1))
    with pytest.raises(TypeError, match="Handle"):
        cgd.combine_backward(x, x, i, torch.zeros(4, 1))
    with pytest.raises(TypeError):
        cgd.rms_norm([1.0], w)
    with pytest.raises(TypeError):
        cgd.dropout([1.0], 0.5, 1)


def test_generator_gives_the_published_words():
    """The known answers of Philox4x32-10 that its authors publish with it."""
    def one(ctr, key):
        w = words(np.array([ctr[0] | ctr[1] << 32], np.uint64), ctr[2] | ctr[3] << 32, key[0] | key[1] << 32)
        return ["%08x" % v for v in w[0]]
    f = 0xFFFFFFFF
    assert one((0, 0, 0, 0), (0, 0)) == ["6627e8d5", "e169c58d", "bc57ac4c", "9b00dbd8"]
    assert one((f, f, f, f), (f, f)) == ["408f276d", "41c83b0e", "a20bc7c6", "6d5451fd"]
    assert one((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0)) == \
        ["d16cfe09", "94fdcceb", "5001e420", "24126ea1"]


def test_oracle_mask_has_the_probability():
    n = 1 << 20
    for p in (0.0, 0.1, 0.5, 1.0):
        limit = round(p * 65536)
        share = 1 - kept(n, 77, 5, limit).mean()
        assert abs(share - limit / 65536) <= 5 * (0.25 / n) ** 0.5
