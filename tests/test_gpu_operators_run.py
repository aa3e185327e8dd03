"""The group norm, the query attention and the gradient clipping together with
the entry points they stand beside, as a training step uses them: normalised
maps are the value of the spatial cross-attention, one projection makes the
object queries' q, k and v, the gradients come back through both and are
clipped together.  Each result is held to 64 bits on its actual inputs (the
tolerances of the operators' own tests), and the captured step to the bits of
the eager one."""
import numpy as np
import pytest
import torch

import scale_deformable_attention_03_b200 as msda
from tests import test_gpu_clip_grad_norm as clip
from tests import test_gpu_group_norm as norm
from tests import test_gpu_query_attention as attention

pytestmark = pytest.mark.gpu

LEVELS = [(8, 10), (4, 5)]
NCAM, H, C, G, N, NQ, P, R = 2, 8, 256, 32, 77, 50, 4, 2


class Step:
    def __init__(self, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        rand = lambda *s: torch.rand(*s, generator=g, device="cuda")  # noqa: E731
        nv = sum(h * w for h, w in LEVELS)
        self.shapes = np.array(LEVELS, np.int64)
        self.starts = np.array([0, LEVELS[0][0] * LEVELS[0][1]], np.int64)
        self.features = rnd(1, NCAM, nv, C) * 2 + rnd(C)
        self.gamma, self.beta = 1 + 0.1 * rnd(2, C), 0.1 * rnd(2, C)
        self.ref, self.mask = rand(NCAM, 1, NQ, R, 2), (rand(NCAM, 1, NQ, R) < 0.5).to(torch.uint8)
        self.off, self.logits = rnd(1, NQ, H, 2, P, 2), rnd(1, NQ, H, 2, P)
        self.objects, self.w = rnd(N, C).bfloat16(), (rnd(3 * C, C) / 16).bfloat16()
        self.points, self.tau = rand(1, N, 2), 10 * rand(1, N, H)
        self.group = torch.where(torch.arange(N) < 40, 0, 1 + torch.arange(N) // 7).int()[None].cuda()
        self.g_sca, self.g_att = rnd(1, NQ, C), rnd(1, N, C).bfloat16()

    def qkv(self):
        y = self.proj.view(1, N, 3, H, 32)
        return y[:, :, 0], y[:, :, 1], y[:, :, 2]

    def attention_inputs(self):
        return dict(zip("qkv", self.qkv()), q_points=self.points, k_points=self.points, tau=self.tau,
                    q_group=self.group, k_group=self.group)

    def run(self):
        self.value, self.mean, self.rstd = msda.msda_group_norm(
            self.features, self.shapes, self.starts, G, self.gamma, self.beta, activation="relu")
        sca = (self.value.view(1, NCAM, -1, H, 32), self.shapes, self.starts, self.ref, self.mask,
               self.off, self.logits)
        self.sca = msda.sca_forward(*sca)
        self.proj = msda.msda_linear(self.objects, self.w, out_dtype=torch.bfloat16)
        a = self.attention_inputs()
        self.att, self.lse = msda.msda_query_attention(**a)
        g_value, _, _ = msda.sca_backward(*sca, self.g_sca, deterministic=True)
        self.g_value = g_value.view(1, NCAM, -1, C)
        self.g_norm = msda.msda_group_norm_backward(
            self.features, self.shapes, self.starts, G, self.mean, self.rstd, self.g_value, self.gamma,
            self.beta, activation="relu")
        self.g_heads = msda.msda_query_attention_backward(**a, lse=self.lse, grad_out=self.g_att)
        self.grads = list(self.g_norm) + list(self.g_heads)
        self.clipped = [torch.empty(t.shape, device="cuda") for t in self.grads]
        self.total = msda.msda_clip_grad_norm(self.grads, 1.0, out=self.clipped)
        return [self.value, self.mean, self.rstd, self.sca, self.att, self.lse, *self.grads,
                *self.clipped, self.total]


def test_a_training_step():
    s = Step(1)
    s.run()
    torch.cuda.synchronize()
    x = s.features.view(NCAM, -1, C)
    y, mean, rstd, core = norm.forward64(x, s.shapes, s.starts, G, s.gamma, s.beta, 1e-5, "relu")
    assert bool(((s.value.view_as(y).double() - y).abs() <= 2.0 ** -14 * core + 2.0 ** -24 * y.abs()).all())
    wx, wg, wb, size, sg, sb = norm.backward64(
        x, s.shapes, s.starts, G, s.mean.view_as(mean), s.rstd.view_as(rstd), s.g_value.view(NCAM, -1, C),
        s.gamma, s.beta, "relu")
    tol = 2.0 ** -18 + 2.0 ** -20
    assert bool(((s.g_norm[0].view_as(wx).double() - wx).abs() <= tol * size + 2.0 ** -24 * wx.abs()).all())
    assert bool(((s.g_norm[1].double() - wg).abs() <= 2.0 ** -18 * sg + 2.0 ** -24 * wg.abs()).all())
    assert bool(((s.g_norm[2].double() - wb).abs() <= 2.0 ** -18 * sb + 2.0 ** -24 * wb.abs()).all())
    attention.check_forward(s.attention_inputs(), s.att, s.lse)
    attention.check_backward(s.attention_inputs(), s.g_att, s.g_heads)
    total, want = clip.expected(s.grads, 1.0, 1e-6, 1.0)
    assert total > 1.0 and abs(float(s.total) - total) <= total * 2.0 ** -23
    for o, w in zip(s.clipped, want):
        clip.check(o, w, o.dtype)


def test_the_captured_step_gives_the_same_bits():
    s = Step(2)
    first = [t.clone() for t in s.run()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = s.run()
    for t in out:
        t.zero_()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, out))


def test_two_steps_at_once():
    steps = [Step(3), Step(4)]
    alone = [[t.clone() for t in s.run()] for s in steps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(5):
        got = []
        for s, st in zip(steps, streams):
            with torch.cuda.stream(st):
                got.append(s.run())
    torch.cuda.synchronize()
    for a, b in zip(alone, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_nothing_is_written_around_the_outputs():
    g = torch.Generator(device="cuda").manual_seed(6)

    def framed(shape, dtype):
        n = int(np.prod(shape))
        flat = torch.full((n + 128,), 3.0, device="cuda", dtype=dtype)
        return flat, flat[64:64 + n].view(shape)

    frames = []
    new = lambda shape, dtype=torch.float32: (frames.append(framed(shape, dtype)), frames[-1][1])[1]  # noqa: E731
    x = torch.randn(2, 53, 40, generator=g, device="cuda")
    shapes, starts = np.array([[5, 7], [3, 4]]), np.array([2, 40])
    y, mean, rstd = msda.msda_group_norm(x, shapes, starts, 5, out=new((2, 53, 40), torch.bfloat16),
                                         mean=new((2, 2, 5)), rstd=new((2, 2, 5)))
    msda.msda_group_norm_backward(x, shapes, starts, 5, mean, rstd, x,
                                  out=(new((2, 53, 40)), new((2, 40)), new((2, 40))))
    a = attention.problem(2, 67, 131, 3, True, "shared", 9)
    _, lse = msda.msda_query_attention(**a, out=new((2, 67, 96), torch.bfloat16), lse=new((2, 3, 67)))
    do = torch.randn(2, 67, 96, generator=g, device="cuda").bfloat16()
    msda.msda_query_attention_backward(
        **a, lse=lse, grad_out=do,
        out=(new((2, 67, 3, 32), torch.bfloat16), new((2, 131, 3, 32), torch.bfloat16),
             new((2, 131, 3, 32), torch.bfloat16), new((2, 67, 3))))
    msda.msda_clip_grad_norm([x], 0.5, out=[new((2, 53, 40))], total_norm=new((1,)))
    torch.cuda.synchronize()
    for flat, t in frames:
        n = t.numel()
        assert bool((flat[:64] == 3).all()) and bool((flat[64 + n:] == 3).all())
