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
