"""The C entry points with the arguments that may be NULL, against the same calls with them:
the other outputs keep their bits, and nothing is written in the place of the missing ones."""
import ctypes

import numpy as np
import pytest
import torch

import scale_deformable_attention_03_b200 as msda
from tests import test_gpu_group_norm as norm
from tests import test_gpu_query_attention as attention

pytestmark = pytest.mark.gpu

LEVELS = {"small": [(7, 11), (3, 5)], "large": [(60, 70), (30, 35)]}


def _tables(levels):
    s = np.array(levels, np.int64)
    st = np.concatenate([[0], np.cumsum(s[:, 0] * s[:, 1])[:-1]]).astype(np.int64)
    return s, st


def _stream():
    return torch.cuda.current_stream().cuda_stream


@pytest.mark.parametrize("which", LEVELS)
@pytest.mark.parametrize("missing", ["mean", "rstd", "both"])
def test_norm_without_its_statistics(which, missing):
    x, shapes, starts, gamma, beta = norm.problem(LEVELS[which], 0, 64, 8, 2, torch.float32, 3)
    y, mean, rstd = msda.msda_group_norm(x, shapes, starts, 8, gamma, beta, activation="relu")
    s, st = _tables(LEVELS[which])
    d = msda.NormDims(2, x.shape[1], 64, 2, 8)
    L = msda.lib()
    n = L.msda_group_norm_workspace_size(d)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    y2, m2, r2 = torch.empty_like(y), torch.full_like(mean, 5.0), torch.full_like(rstd, 5.0)
    keep_m, keep_r = missing == "rstd", missing == "mean"
    assert L.msda_group_norm(x.data_ptr(), 0, s.ctypes.data, st.ctypes.data, d, gamma.data_ptr(), beta.data_ptr(),
                             1e-5, 1, 0, y2.data_ptr(), m2.data_ptr() if keep_m else None,
                             r2.data_ptr() if keep_r else None, ws.data_ptr(), n, _stream()) == 0
    assert torch.equal(y, y2)
    assert torch.equal(m2, mean if keep_m else torch.full_like(mean, 5.0))
    assert torch.equal(r2, rstd if keep_r else torch.full_like(rstd, 5.0))


@pytest.mark.parametrize("which", LEVELS)
@pytest.mark.parametrize("want", [(False, False), (True, False), (False, True)])
def test_norm_gradient_without_the_parameters(which, want):
    x, shapes, starts, gamma, beta = norm.problem(LEVELS[which], 0, 64, 8, 2, torch.float32, 4)
    _, mean, rstd = msda.msda_group_norm(x, shapes, starts, 8, gamma, beta)
    dy = torch.randn(x.shape, device="cuda")
    first = msda.msda_group_norm_backward(x, shapes, starts, 8, mean, rstd, dy, gamma, beta)
    s, st = _tables(LEVELS[which])
    d = msda.NormDims(2, x.shape[1], 64, 2, 8)
    L = msda.lib()
    n = L.msda_group_norm_backward_workspace_size(d)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    gx, gg, gb = torch.empty_like(x), torch.full_like(gamma, 5.0), torch.full_like(beta, 5.0)
    assert L.msda_group_norm_backward(
        x.data_ptr(), 0, s.ctypes.data, st.ctypes.data, d, gamma.data_ptr(), beta.data_ptr(), mean.data_ptr(),
        rstd.data_ptr(), 0, dy.data_ptr(), 0, 0, gx.data_ptr(), gg.data_ptr() if want[0] else None,
        gb.data_ptr() if want[1] else None, ws.data_ptr(), n, _stream()) == 0
    assert torch.equal(gx, first[0])
    assert torch.equal(gg, first[1] if want[0] else torch.full_like(gg, 5.0))
    assert torch.equal(gb, first[2] if want[1] else torch.full_like(gb, 5.0))


@pytest.mark.parametrize("size", [(1, 17, 1000, 8), (2, 70, 60, 2), (4, 2400, 75, 8)])
@pytest.mark.parametrize("far", [False, True])
def test_attention_without_lse(size, far):
    a = attention.problem(*size, True, "shared", 5, joint=False)
    if far:
        a["k_points"] = a["k_points"] + 3000
    out, _ = msda.msda_query_attention(**a)
    B, Nq, Nk, H = size
    p = msda.Attention(*(a[n].data_ptr() for n in "qkv"), 32 * H, 32 * H, 32 * H,
                       *(a[n].data_ptr() for n in ("q_points", "k_points", "tau", "q_group", "k_group")),
                       32 ** -0.5, B, Nq, Nk, H)
    again = torch.empty_like(out)
    assert msda.lib().msda_query_attention(ctypes.byref(p), again.data_ptr(), None, _stream()) == 0
    assert torch.equal(out, again)


def test_clipping_without_an_output_counts_the_tensor():
    g = [torch.randn(n, device="cuda") for n in (1000, 20_001, 7)]
    out = [torch.full_like(t, 5.0) for t in g]
    total = torch.empty(1, device="cuda")
    t = (msda.Grad * 3)(*[msda.Grad(a.data_ptr(), None if i == 1 else o.data_ptr(), a.numel(), 0, 0)
                          for i, (a, o) in enumerate(zip(g, out))])
    L = msda.lib()
    n = L.msda_clip_grad_norm_workspace_size(3)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    assert L.msda_clip_grad_norm(t, 3, 1.0, 1e-6, 1.0, ws.data_ptr(), n, total.data_ptr(), _stream()) == 0
    want = [torch.empty_like(a) for a in g]
    all_of_them = msda.msda_clip_grad_norm(g, 1.0, out=want)
    assert torch.equal(total, all_of_them)
    assert torch.equal(out[0], want[0]) and torch.equal(out[2], want[2]) and bool((out[1] == 5).all())
