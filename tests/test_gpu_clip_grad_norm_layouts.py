"""msda_clip_grad_norm on gradients whose dimensions lie in another order (those of a transposed
weight, of a channels-last map with a permuted view), in place and into outputs alike.

Tolerances as for contiguous tensors: total to 2^-23, an output to the two roundings of its
product (2^-23) and half a step of its type."""
import pytest
import torch

import scale_deformable_attention_03_b200 as msda
from tests import test_gpu_clip_grad_norm as clip

pytestmark = pytest.mark.gpu

VIEWS = {
    "transposed": lambda: torch.randn(70, 130, device="cuda").t(),
    "batched transpose": lambda: torch.randn(3, 40, 50, device="cuda").transpose(1, 2),
    "permuted map": lambda: torch.randn(2, 5, 7, 11, device="cuda").permute(3, 0, 2, 1),
    "channels last": lambda: torch.randn(4, 6, 3, 3, device="cuda").to(memory_format=torch.channels_last),
    "slice of the outer dimension": lambda: torch.randn(9, 33, device="cuda")[2:7],
}


@pytest.mark.parametrize("view", VIEWS)
@pytest.mark.parametrize("into", [None, torch.float32, torch.bfloat16])
def test_any_order_without_gaps(view, into):
    grads = [VIEWS[view](), torch.randn(77, device="cuda"), VIEWS[view]().bfloat16()]
    total, want = clip.expected(grads, 1.0, 1e-6, 1.0)
    outs = None if into is None else [torch.full_like(g, 9.0, dtype=into) for g in grads]
    assert outs is None or all(o.stride() == g.stride() for o, g in zip(outs, grads))
    got = msda.msda_clip_grad_norm(grads, 1.0, out=outs)
    assert abs(float(got) - total) <= total * 2.0 ** -23
    for o, w in zip(grads if outs is None else outs, want):
        clip.check(o, w, o.dtype)


def test_another_order_in_the_output_is_refused():
    g = torch.randn(8, 8, device="cuda")
    keep = g.clone()
    for out in (torch.empty(8, 8, device="cuda").t(), torch.empty(8, 16, device="cuda")[:, ::2]):
        with pytest.raises(msda.MsdaError):
            msda.msda_clip_grad_norm([g], 1.0, out=[out])
    with pytest.raises(msda.MsdaError):
        msda.msda_clip_grad_norm([torch.randn(8, 16, device="cuda")[:, :8]], 1.0)
    assert torch.equal(g, keep)
