"""Refusals of the group norm, the query attention and the gradient clipping,
without a GPU: bad arguments are rejected on the host (status code, message,
nothing launched).  Device pointers are fake addresses that are never
dereferenced."""
import ctypes
import math

import numpy as np
import pytest

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
