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


def test_norm_of_many_small_items():
    """More spans than CTAs: every run crosses many levels and items."""
    levels, B = [(1, 1), (1, 2), (2, 1)], 3001
    x, shapes, starts, gamma, beta = norm.problem(levels, 1, 16, 2, B, torch.float32, 8)
    y, mean, rstd = msda.msda_group_norm(x, shapes, starts, 2, gamma, beta, activation="silu")
    want, _, _, core = norm.forward64(x, shapes, starts, 2, gamma, beta, 1e-5, "silu")
    assert bool(((y.double() - want).abs() <= 2.0 ** -14 * core + 2.0 ** -24 * want.abs()).all())
    dy = torch.randn(x.shape, device="cuda")
    gx, gg, gb = msda.msda_group_norm_backward(x, shapes, starts, 2, mean, rstd, dy, gamma, beta, "silu")
    wx, wg, wb, size, sg, sb = norm.backward64(x, shapes, starts, 2, mean, rstd, dy, gamma, beta, "silu")
    assert bool(((gx.double() - wx).abs() <= (2.0 ** -18 + 2.0 ** -20) * size + 2.0 ** -24 * wx.abs()).all())
    assert bool(((gg.double() - wg).abs() <= 2.0 ** -18 * sg + 2.0 ** -24 * wg.abs()).all())
    assert bool(((gb.double() - wb).abs() <= 2.0 ** -18 * sb + 2.0 ** -24 * wb.abs()).all())


def test_offsets_past_32_bits():
    """Elements behind the 2^31st of each operator's tensors."""
    # the norm: five items of 2^20 rows of 512, the last one checked.  Its sums are longer than
    # the small problems': at most 2^20 / 296 * 5 rows a run, four of them side by side, are 4500
    # additions in fp32; their roundings are of random sign, 6 sqrt(4500) u (1 + D^2) < 2^-11 of
    # the variance, half of it in r, and 2^-12 of a spread in the mean
    x = torch.randn(5, 1 << 20, 512, device="cuda", dtype=torch.bfloat16)
    shapes, starts = np.array([[1024, 1024]]), np.array([0])
    y, mean, rstd = msda.msda_group_norm(x, shapes, starts, 8)
    e = x[4].double().view(-1, 8, 64)
    mu = e.mean((0, 2), keepdim=True)
    r = 1 / torch.sqrt(((e - mu) ** 2).mean((0, 2), keepdim=True) + 1e-5)
    want = ((e - mu) * r).view(-1, 512)
    tol = 2.0 ** -11 * (1 + want.abs()) + 2.0 ** -8 * want.abs()
    assert bool(((y[4].double() - want).abs() <= tol).all())
    del e, want, tol
    gx, _, gb = msda.msda_group_norm_backward(x, shapes, starts, 8, mean, rstd, y)
    assert bool(torch.isfinite(gx[4]).all()) and bool((gx[4, -1] != x[4, -1]).any())
    del x, y, gx
    torch.cuda.empty_cache()
    # the attention: keys and values as slices of rows of 2^18 values
    wide = torch.zeros(1, 9000, 1 << 13, 32, device="cuda", dtype=torch.bfloat16)
    wide[:, :, -4:] = torch.randn(1, 9000, 4, 32, device="cuda").bfloat16()
    a = dict(q=torch.randn(1, 33, 2, 32, device="cuda").bfloat16(), k=wide[:, :, -2:],
             v=wide[:, :, -4:-2])
    out, lse = msda.msda_query_attention(**a)
    small = {**a, "k": a["k"].contiguous(), "v": a["v"].contiguous()}
    assert all(torch.equal(s, t) for s, t in zip((out, lse), msda.msda_query_attention(**small)))
    do = torch.randn(1, 33, 64, device="cuda").bfloat16()
    assert all(s is None or torch.equal(s, t) for s, t in zip(
        msda.msda_query_attention_backward(**a, lse=lse, grad_out=do),
        msda.msda_query_attention_backward(**small, lse=lse, grad_out=do)))
    attention.check_forward(small, out, lse)
    del wide, a
    torch.cuda.empty_cache()
    # the clipping: one tensor, in place
    n = (1 << 31) + 12345
    g = torch.full((n,), 0.5, device="cuda", dtype=torch.bfloat16)
    total = msda.msda_clip_grad_norm([g], 1.0)
    want = 0.5 * n ** 0.5
    assert abs(float(total) - want) <= want * 2.0 ** -23
    f = torch.tensor(0.5 / (want + 1e-6)).bfloat16()
    assert bool((g[-20000:] == f.cuda()).all()) and bool((g[:20000] == f.cuda()).all())


def test_the_first_call_of_a_process_is_captured():
    """No call before the capture: nothing that a first call sets up needs a stream."""
    import subprocess
    import sys
    code = """
import numpy as np, torch
import scale_deformable_attention_03_b200 as msda
x = torch.randn(2, 700, 256, device="cuda")
q = torch.randn(1, 700, 8, 32, device="cuda").bfloat16()
p, tau = torch.rand(1, 700, 2, device="cuda"), torch.rand(1, 700, 8, device="cuda")
do = torch.randn(1, 700, 256, device="cuda").bfloat16()
def step():
    y, m, r = msda.msda_group_norm(x, np.array([[20, 35]]), np.array([0]), 32)
    g = msda.msda_group_norm_backward(x, np.array([[20, 35]]), np.array([0]), 32, m, r, y)
    o, l = msda.msda_query_attention(q, q, q, p, p, tau)
    h = msda.msda_query_attention_backward(q, q, q, l, do, p, p, tau)
    n = msda.msda_clip_grad_norm(list(g), 1.0)
    return [y, m, r, *g, o, l, *h, n]
s = torch.cuda.Stream()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph, stream=s):
    out = step()
graph.replay()
torch.cuda.synchronize()
first = [t.clone() for t in out]
assert all(torch.equal(a, b) for a, b in zip(first, step()))
print("captured first")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stderr[-2000:]
