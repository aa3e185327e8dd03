"""msda_clip_grad_norm without a GPU: what a refused call leaves undone, and the layouts that
pass.  Device pointers are fake addresses that are never dereferenced."""
import ctypes

import pytest
import torch

import scale_deformable_attention_03_b200 as msda
from scale_deformable_attention_03_b200 import build as msda_build

UNSUPPORTED = 2
FAKE = 0x7f0000000000


@pytest.fixture(scope="module")
def L():
    msda_build.build()
    return msda.lib()


@pytest.mark.parametrize("count,at", [(1, 0), (64, 63), (65, 64), (960, 3), (961, 960), (2000, 1500)])
def test_too_many_values_are_refused_before_anything_is_launched(L, count, at):
    """A launch would fail here (no GPU, code 4) before the part of the list with the large tensor."""
    if torch.cuda.is_available():
        pytest.skip("would launch on fake addresses")
    t = (msda.Grad * count)()
    for i in range(count):
        t[i] = msda.Grad(FAKE + 4096 * i, None, 7, 0, 0)
    t[at] = msda.Grad(1 << 50, None, 1 << 44, 0, 0)
    n = L.msda_clip_grad_norm_workspace_size(count)
    code = L.msda_clip_grad_norm(t, count, 1.0, 1e-6, 1.0, 1 << 56, n, 1 << 57, None)
    assert code == UNSUPPORTED and "too many values" in L.msda_last_error().decode()


def test_layouts_without_gaps_in_the_same_order():
    same = msda._same_dense_layout
    w = torch.empty(6, 5, 4, 3)
    for order in ((0, 1, 2, 3), (3, 2, 1, 0), (1, 3, 0, 2), (2, 0, 3, 1)):
        t = w.permute(order)
        assert same(t, t) and same(t, torch.empty_like(t)) and same(t, t.clone())
    assert not same(w.permute(1, 0, 2, 3), torch.empty(5, 6, 4, 3))
    for hole in (w[:, :4], w[..., ::2], w[::2], torch.empty(5, 1).expand(5, 7), torch.empty(7).expand(5, 7)):
        assert not same(hole, hole)
    assert same(w[2:4], w[2:4]) and same(torch.empty(1).expand(1, 1), torch.empty(1, 1))
    square = torch.empty(5, 5)
    assert same(square.t(), square.t()) and not same(square, square.t())
    assert same(torch.empty(()), torch.empty(()))
    assert same(torch.empty(5, 0), torch.empty(5, 0)) and same(torch.empty(0, 5).t(), torch.empty(0, 5).t())


@pytest.mark.parametrize("grads", [[None], [torch.ones(3), None], [3.0], [torch.ones(3)]])
def test_what_is_no_cuda_tensor_is_refused(grads):
    with pytest.raises(msda.MsdaError, match="msda_clip_grad_norm"):
        msda.msda_clip_grad_norm(grads, 1.0)
    with pytest.raises(msda.MsdaError, match="msda_clip_grad_norm"):
        msda.msda_clip_grad_norm([], 1.0, total_norm=grads[-1])
