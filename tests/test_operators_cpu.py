"""Refusals of the group norm, the query attention and the gradient clipping,
without a GPU: bad arguments are rejected on the host (status code, message,
nothing launched).  Device pointers are fake addresses that are never
dereferenced."""
import ctypes
import math

import numpy as np
import pytest
import torch

import scale_deformable_attention_03_b200 as msda
from scale_deformable_attention_03_b200 import build as msda_build

OK, INVALID, UNSUPPORTED, WORKSPACE, CUDA = 0, 1, 2, 3, 4
FAKE = 0x7f0000000000  # a 256-byte aligned address, never dereferenced


@pytest.fixture(scope="module")
def L():
    msda_build.build()
    return msda.lib()


def _clip(L, tensors, max_norm=1.0, eps=1e-6, scale=1.0, ws=FAKE + (1 << 32), ws_bytes=None,
          total=FAKE + (1 << 33), count=None):
    t = (msda.Grad * max(1, len(tensors)))(*[msda.Grad(*x) for x in tensors])
    n = len(tensors) if count is None else count
    if ws_bytes is None:
        ws_bytes = L.msda_clip_grad_norm_workspace_size(n)
    return L.msda_clip_grad_norm(t if tensors else None, n, max_norm, eps, scale, ws, ws_bytes,
                                 total, None)


@pytest.mark.parametrize("kw,code,fragment", [
    (dict(count=-1), INVALID, "count"),
    (dict(max_norm=-1.0), INVALID, "max_norm"),
    (dict(max_norm=math.nan), INVALID, "max_norm"),
    (dict(eps=0.0), INVALID, "eps"),
    (dict(eps=math.inf), INVALID, "eps"),
    (dict(scale=0.0), INVALID, "grad_scale"),
    (dict(scale=math.inf), INVALID, "grad_scale"),
    (dict(total=None), INVALID, "total_norm"),
    (dict(total=FAKE + 2), INVALID, "total_norm"),
    (dict(ws=None), WORKSPACE, "workspace"),
    (dict(ws=FAKE + 8), WORKSPACE, "workspace"),
    (dict(ws_bytes=16), WORKSPACE, "workspace"),
])
def test_clip_rejects_bad_arguments(L, kw, code, fragment):
    assert _clip(L, [(FAKE, FAKE, 100, 0, 0)], **kw) == code
    assert fragment in L.msda_last_error().decode()


@pytest.mark.parametrize("tensors,fragment", [
    ([(0, 0, 5, 0, 0)], "grad is null"),
    ([(FAKE, FAKE, 5, 2, 0)], "grad dtype"),
    ([(FAKE, FAKE, 5, 0, 9)], "out dtype"),
    ([(FAKE, FAKE, -1, 0, 0)], "values"),
    ([(FAKE + 2, FAKE + 2, 5, 0, 0)], "aligned"),
    ([(FAKE, FAKE + 1001, 5, 0, 1)], "aligned"),
    ([(FAKE, FAKE, 5, 0, 1)], "in place"),
    ([(FAKE, FAKE, 5, 0, 0), (FAKE, FAKE, 5, 0, 0)], "overlap"),
    ([(FAKE, FAKE, 5, 0, 0), (FAKE + 16, FAKE + 16, 5, 0, 0)], "overlap"),
    ([(FAKE, FAKE + 4096, 5, 0, 0), (FAKE + 1024, FAKE + 4096, 5, 0, 0)], "overlap"),
    ([(FAKE, FAKE + 4, 5, 0, 0)], "overlap"),
    ([(FAKE + (1 << 33), 0, 5, 0, 0)], "overlap"),   # over total_norm
])
def test_clip_rejects_bad_tensors(L, tensors, fragment):
    assert _clip(L, tensors) == INVALID
    assert fragment in L.msda_last_error().decode()


def test_clip_workspace_grows_with_the_table(L):
    f = L.msda_clip_grad_norm_workspace_size
    assert f(0) == f(960) > 0 and f(961) == 2 * f(960)


def _tables(shapes=((3, 4), (2, 2)), starts=None):
    s = np.asarray(shapes, dtype=np.int64).reshape(-1, 2)
    st = (np.concatenate([[0], np.cumsum(s[:, 0] * s[:, 1])[:-1]]) if starts is None
          else np.asarray(starts)).astype(np.int64)
    p = ctypes.POINTER(ctypes.c_int64)
    return s, st, s.ctypes.data_as(p), st.ctypes.data_as(p)


NORM = dict(d=(2, 16, 32, 2, 4), shapes=((3, 4), (2, 2)), starts=None, x=FAKE, xt=0, gamma=None,
            beta=None, eps=1e-5, act=0, yt=0, y=FAKE + (1 << 30), ws=FAKE + (1 << 31), ws_bytes=None)


def _norm(L, **kw):
    a = dict(NORM, **kw)
    keep = _tables(a["shapes"], a["starts"])
    d = msda.NormDims(*a["d"])
    n = L.msda_group_norm_workspace_size(d) if a["ws_bytes"] is None else a["ws_bytes"]
    return L.msda_group_norm(a["x"], a["xt"], keep[2], keep[3], d, a["gamma"], a["beta"], a["eps"],
                             a["act"], a["yt"], a["y"], None, None, a["ws"], n, None)


def _norm_back(L, gx=FAKE + (1 << 30), gy=FAKE + (1 << 29), gxt=0, gyt=0, mean=FAKE, **kw):
    a = dict(NORM, **kw)
    keep = _tables(a["shapes"], a["starts"])
    d = msda.NormDims(*a["d"])
    n = L.msda_group_norm_backward_workspace_size(d) if a["ws_bytes"] is None else a["ws_bytes"]
    return L.msda_group_norm_backward(a["x"], a["xt"], keep[2], keep[3], d, a["gamma"], a["beta"],
                                      mean, FAKE, a["act"], gy, gyt, gxt, gx, None, None, a["ws"], n,
                                      None)


NORM_BAD = [
    (dict(d=(-1, 16, 32, 2, 4)), INVALID, "B (-1)"),
    (dict(d=(2, 0, 32, 2, 4)), INVALID, "Nv (0)"),
    (dict(d=(2, 16, 36, 2, 4)), UNSUPPORTED, "C = 36"),
    (dict(d=(2, 16, 2056, 2, 4)), UNSUPPORTED, "C = 2056"),
    (dict(d=(2, 16, 0, 2, 4)), UNSUPPORTED, "C = 0"),
    (dict(d=(2, 16, 32, 0, 4)), UNSUPPORTED, "L = 0"),
    (dict(d=(2, 16, 32, 9, 4)), UNSUPPORTED, "L = 9"),
    (dict(d=(2, 16, 32, 2, 0)), INVALID, "G = 0"),
    (dict(d=(2, 16, 32, 2, 3)), INVALID, "G = 3"),
    (dict(d=(2, 15, 32, 2, 4)), INVALID, "does not fit"),
    (dict(starts=(0, -1)), INVALID, "does not fit"),
    (dict(starts=(0, 11)), INVALID, "shares rows"),
    (dict(starts=(3, 0)), INVALID, "shares rows"),
    (dict(shapes=((3, 4), (0, 2)), starts=(0, 12)), INVALID, "shape"),
    (dict(d=(2 ** 30, 2 ** 20, 2048, 2, 4)), UNSUPPORTED, "too many rows"),
    (dict(x=0), INVALID, "x is null"),
    (dict(x=FAKE + 8), INVALID, "x must be 16-byte"),
    (dict(xt=5), INVALID, "x_dtype"),
    (dict(gamma=FAKE + 4), INVALID, "gamma"),
    (dict(beta=FAKE + 4), INVALID, "beta"),
    (dict(act=3), INVALID, "activation"),
    (dict(ws=None), WORKSPACE, "workspace"),
    (dict(ws=FAKE + 128), WORKSPACE, "workspace"),
    (dict(ws_bytes=64), WORKSPACE, "workspace"),
]


@pytest.mark.parametrize("kw,code,fragment", NORM_BAD + [
    (dict(yt=2), INVALID, "y_dtype"),
    (dict(y=None), INVALID, "y is null"),
    (dict(y=FAKE), INVALID, "overlaps"),
    (dict(y=FAKE + 2 * 16 * 32 * 4 - 16), INVALID, "overlaps"),
    (dict(eps=0.0), INVALID, "eps"),
    (dict(eps=math.nan), INVALID, "eps"),
])
def test_group_norm_rejects(L, kw, code, fragment):
    assert _norm(L, **kw) == code
    assert fragment in L.msda_last_error().decode()


@pytest.mark.parametrize("kw,code,fragment", NORM_BAD + [
    (dict(gxt=2), INVALID, "gx_dtype"),
    (dict(gyt=2), INVALID, "gy_dtype"),
    (dict(gx=None), INVALID, "grad_x is null"),
    (dict(gy=None), INVALID, "grad_y is null"),
    (dict(mean=None), INVALID, "mean is null"),
    (dict(gx=FAKE), INVALID, "overlaps"),
    (dict(gx=FAKE + (1 << 29)), INVALID, "overlaps"),
])
def test_group_norm_backward_rejects(L, kw, code, fragment):
    assert _norm_back(L, **kw) == code
    assert fragment in L.msda_last_error().decode()


def test_group_norm_of_no_items(L):
    assert _norm(L, d=(0, 16, 32, 2, 4), x=0, y=0, ws=0) == OK
    assert _norm_back(L, d=(0, 16, 32, 2, 4), x=0, gx=0, gy=0, mean=0, ws=0) == OK


def _attention(**kw):
    a = dict(q=FAKE, k=FAKE + (1 << 24), v=FAKE + (2 << 24), q_stride=64, k_stride=64, v_stride=128,
             q_points=None, k_points=None, tau=None, q_group=None, k_group=None, scale=0.2, B=2,
             Nq=10, Nk=300, H=2)
    a.update(kw)
    return msda.Attention(**a)


def _attend(L, p, out=FAKE + (3 << 24), lse=FAKE + (4 << 24)):
    return L.msda_query_attention(p, out, lse, None)


def _attend_back(L, p, lse=FAKE + (4 << 24), go=FAKE + (5 << 24), gq=FAKE + (6 << 24),
                 gk=FAKE + (7 << 24), gv=FAKE + (8 << 24), gt=FAKE + (9 << 24),
                 ws=FAKE + (1 << 30), n=1 << 30):
    return L.msda_query_attention_backward(p, lse, go, gq, gk, gv, gt, ws, n, None)


ATTENTION_BAD = [
    (dict(B=-1), INVALID, "B (-1)"),
    (dict(Nq=-1), INVALID, "Nq (-1)"),
    (dict(Nk=-2), INVALID, "Nk (-2)"),
    (dict(H=0), INVALID, "H (0)"),
    (dict(H=2 ** 21, q_stride=2 ** 27), UNSUPPORTED, "H ="),
    (dict(B=2 ** 30, Nq=2 ** 20), UNSUPPORTED, "too many rows"),
    (dict(Nk=2 ** 31 - 1), UNSUPPORTED, "too many rows"),
    (dict(scale=math.inf), INVALID, "scale"),
    (dict(q=None), INVALID, "q is null"),
    (dict(k=None), INVALID, "k is null"),
    (dict(v=FAKE + 8), INVALID, "v must be 16-byte"),
    (dict(q_stride=56), INVALID, "q_stride"),
    (dict(k_stride=68), INVALID, "k_stride"),
    (dict(v_stride=-64), INVALID, "v_stride"),
    (dict(tau=FAKE), INVALID, "go together"),
    (dict(q_points=FAKE, k_points=FAKE), INVALID, "go together"),
    (dict(q_points=FAKE + 4, k_points=FAKE, tau=FAKE), INVALID, "8-byte"),
    (dict(q_points=FAKE, k_points=FAKE, tau=FAKE + 2), INVALID, "4-byte"),
    (dict(q_group=FAKE), INVALID, "go together"),
    (dict(q_group=FAKE, k_group=FAKE + 1), INVALID, "4-byte"),
]


@pytest.mark.parametrize("kw,code,fragment", ATTENTION_BAD)
def test_attention_rejects_bad_inputs(L, kw, code, fragment):
    for call in (_attend, _attend_back):
        assert call(L, _attention(**kw)) == code
        assert fragment in L.msda_last_error().decode()
    assert L.msda_query_attention(None, FAKE, FAKE, None) == INVALID


@pytest.mark.parametrize("kw,code", [
    (dict(out=None), INVALID), (dict(out=FAKE + 8), INVALID), (dict(lse=FAKE + 2), INVALID),
    (dict(out=FAKE), INVALID), (dict(out=FAKE + (2 << 24) + 64), INVALID)])
def test_attention_rejects_bad_outputs(L, kw, code):
    assert _attend(L, _attention(), **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(lse=None), INVALID), (dict(go=None), INVALID), (dict(gq=None), INVALID),
    (dict(gk=None), INVALID), (dict(gv=FAKE + 8), INVALID), (dict(gt=None), INVALID),
    (dict(gk=FAKE), INVALID), (dict(ws=None), WORKSPACE), (dict(ws=FAKE + 16), WORKSPACE),
    (dict(n=8), WORKSPACE)])
def test_attention_backward_rejects_bad_outputs(L, kw, code):
    p = _attention(q_points=FAKE, k_points=FAKE, tau=FAKE)
    assert _attend_back(L, p, **kw) == code


def test_attention_backward_rejects_grad_tau_without_tau(L):
    assert _attend_back(L, _attention()) == INVALID
    assert "grad_tau without tau" in L.msda_last_error().decode()


def test_layouts_are_compared_by_format_not_by_stride():
    """Of a 1 x 1 kernel's weight in channels-last memory the strides differ, the order does not."""
    w = torch.empty(8, 6, 1, 1)
    last = torch.empty_like(w, memory_format=torch.channels_last)
    odd = torch.empty_strided((8, 6, 1, 1), (6, 1, 6, 6))
    wide = torch.empty(8, 6, 3, 3)
    wide_last = wide.to(memory_format=torch.channels_last)
    same = msda._same_dense_layout
    assert same(w, last) and same(w, odd) and same(odd, last) and same(wide_last, wide_last)
    assert not same(wide, wide_last) and not same(wide[:, ::2], wide[:, ::2])


def test_attention_of_nothing(L):
    for kw in (dict(B=0), dict(Nq=0)):
        assert _attend(L, _attention(**kw, q=None), out=None, lse=None) == OK
    assert _attend_back(L, _attention(B=0, q=None, k=None, v=None), lse=None, go=None, gq=None,
                        gk=None, gv=None, ws=None, n=0) == OK
