"""msda_clip_grad_norm against the formula in 64 bits.

Tolerances: total is one rounding of a double sum (2^-24 relative, plus the
double sum's own 2^-40 or so); an output is g times a factor rounded once to
fp32, rounded once to its type: 2^-24 + half a step of the type (fp32 2^-24,
bf16 2^-8), and half of the type's smallest subnormal below its normal range."""
import math

import numpy as np
import pytest
import torch

import scale_deformable_attention_03_b200 as msda

pytestmark = pytest.mark.gpu

HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def make(sizes, dtype, seed, spread=1.0, offset=0):
    """Views of one buffer, `offset` values into it and one value apart."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    flat = torch.randn(sum(sizes) + len(sizes) + offset, generator=g, device="cuda").to(dtype)
    out, at = [], offset
    for i, n in enumerate(sizes):
        v = flat[at:at + n]
        v.mul_(spread ** (i % 3))
        out.append(v)
        at += n + 1
    return flat, out


def expected(grads, max_norm, eps, scale):
    total = scale * math.sqrt(sum(float((g.double() ** 2).sum()) for g in grads))
    f = scale * (1.0 if math.isinf(max_norm) else min(1.0, max_norm / (total + eps)))
    return total, [g.double() * f for g in grads]


def check(got, want, dtype, what=""):
    tol = want.abs() * (HALF_STEP[dtype] + 2.0 ** -23) + 2.0 ** -134
    assert bool(((got.double() - want).abs() <= tol).all()), what


@pytest.mark.parametrize("src", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dst", [torch.float32, torch.bfloat16, None])
@pytest.mark.parametrize("sizes,offset", [
    ([1], 0), ([1], 1), ([8191, 8192, 8193], 0), ([3, 0, 5, 70001, 0, 2], 3),
    ([257] * 70, 1), ([40000, 1, 1, 16384 + 4], 2), ([5] * 2000, 0)])
@pytest.mark.parametrize("scale,max_norm", [(1.0, 3.0), (0.5, 1e9), (1.0, math.inf), (2.0, 0.0)])
def test_norm_and_outputs(src, dst, sizes, offset, scale, max_norm):
    flat, grads = make(sizes, src, 7, spread=30.0, offset=offset)
    before = flat.clone()
    total, want = expected(grads, max_norm, 1e-6, scale)
    if dst is None:
        got_norm = msda.msda_clip_grad_norm(grads, max_norm, grad_scale=scale)
        outs, outflat = grads, flat
    else:
        outflat, outs = make(sizes, dst, 8, offset=(offset * 5) % 7)
        outflat.fill_(12345.0)
        got_norm = msda.msda_clip_grad_norm(grads, max_norm, grad_scale=scale, out=outs)
        assert torch.equal(flat, before)   # the gradients stay
    torch.cuda.synchronize()
    assert abs(float(got_norm) - total) <= total * 2.0 ** -23
    for g, w in zip(outs, want):
        check(g, w, g.dtype)
    # the values between the tensors are left as they were
    gaps = torch.ones(outflat.numel(), dtype=torch.bool, device="cuda")
    for o in outs:
        at = (o.data_ptr() - outflat.data_ptr()) // outflat.element_size() if o.numel() else 0
        gaps[at:at + o.numel()] = False
    ref = before if dst is None else torch.full_like(outflat, 12345.0)
    assert torch.equal(outflat[gaps], ref[gaps])


def test_huge_and_tiny_values_do_not_leave_the_range():
    for v in (1e30, 1e-30):
        g = torch.full((1000,), v, device="cuda")
        n = msda.msda_clip_grad_norm([g], v)
        torch.cuda.synchronize()
        want = float(np.float32(v)) * math.sqrt(1000)
        assert abs(float(n) - want) <= want * 2.0 ** -23
        if v > 1:
            check(g, torch.full((1000,), v / math.sqrt(1000), device="cuda").double(), g.dtype)


@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_non_finite_values(bad):
    g = [torch.ones(100, device="cuda"), torch.ones(9000, device="cuda")]
    g[1][8999] = bad
    n = float(msda.msda_clip_grad_norm(g, 1.0))
    if math.isnan(bad):
        assert math.isnan(n) and all(bool(torch.isnan(t).all()) for t in g)
    else:
        assert n == math.inf and bool((g[0] == 0).all()) and bool((g[1][:8999] == 0).all())
        assert math.isnan(float(g[1][8999]))


def test_same_bits_on_every_run_and_under_capture():
    _, grads = make([100003, 7, 65536], torch.float32, 3)
    outs = [torch.empty_like(g) for g in grads]
    total = torch.empty(1, device="cuda")
    ws = torch.empty(msda.lib().msda_clip_grad_norm_workspace_size(3), dtype=torch.uint8,
                     device="cuda")
    msda.msda_clip_grad_norm(grads, 1.0, out=outs, total_norm=total, workspace=ws)
    first = [o.clone() for o in outs] + [total.clone()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        msda.msda_clip_grad_norm(grads, 1.0, out=outs, total_norm=total, workspace=ws)
    for o in outs:
        o.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, outs + [total]))
    for g in grads:
        g.mul_(3.0)          # the replay reads the new values
    graph.replay()
    torch.cuda.synchronize()
    want_total, want = expected(grads, 1.0, 1e-6, 1.0)
    assert abs(float(total) - want_total) <= want_total * 2.0 ** -23
    for o, w in zip(outs, want):
        check(o, w, o.dtype)


def test_other_stream_and_channels_last():
    s = torch.cuda.Stream()
    w = torch.randn(8, 16, 3, 3, device="cuda").contiguous(memory_format=torch.channels_last)
    ref = w.double().clone()
    s.wait_stream(torch.cuda.current_stream())
    n = msda.msda_clip_grad_norm([w], 1.0, stream=s)
    s.synchronize()
    total = float(ref.norm())
    assert abs(float(n) - total) <= total * 2.0 ** -23
    check(w, ref / (total + 1e-6), w.dtype)


def test_an_empty_list_has_the_norm_zero():
    total = torch.full((1,), 7.0, device="cuda")
    msda.msda_clip_grad_norm([], 1.0, total_norm=total)
    assert float(total) == 0.0
    assert float(msda.msda_clip_grad_norm([torch.empty(0, device="cuda")], 1.0)) == 0.0


def test_refusals():
    g = torch.randn(64, device="cuda")
    keep = g.clone()
    for call in (lambda: msda.msda_clip_grad_norm([g, g], 1.0),
                 lambda: msda.msda_clip_grad_norm([g, g[32:]], 1.0),
                 lambda: msda.msda_clip_grad_norm([g[:32]], 1.0, out=[g[1:33]]),
                 lambda: msda.msda_clip_grad_norm([g], -1.0),
                 lambda: msda.msda_clip_grad_norm([g], math.nan),
                 lambda: msda.msda_clip_grad_norm([g], 1.0, eps=0.0),
                 lambda: msda.msda_clip_grad_norm([g], 1.0, grad_scale=0.0),
                 lambda: msda.msda_clip_grad_norm([g.half()], 1.0),
                 lambda: msda.msda_clip_grad_norm([g.cpu()], 1.0),
                 lambda: msda.msda_clip_grad_norm([g[::2]], 1.0),
                 lambda: msda.msda_clip_grad_norm([g], 1.0, out=[g.bfloat16()[:63]]),
                 lambda: msda.msda_clip_grad_norm([g], 1.0, total_norm=g[:1]),
                 lambda: msda.msda_clip_grad_norm([], 1.0)):
        with pytest.raises(msda.MsdaError):
            call()
    torch.cuda.synchronize()
    assert torch.equal(g, keep)
