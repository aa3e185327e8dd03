"""msda_group_norm and its backward against the formulas in 64 bits.

Tolerances, from the roundings (u = 2^-24; h the half step of the output's
type, fp32 2^-24 and bf16 2^-8).
Variance: within a chunk and channel the sums are fp32, relative to the chunk's
first row: 8 additions in a thread and at most 32 over the slots, 40 u of
sum d^2 = M2 + n D^2 at worst, D the first row's distance from the channel's
mean; beyond the chunk they are double.  With D at most 5 spreads (normal
inputs of this size) that is 40 * 26 u < 2^-13.9 of the variance, half of it
for r: 2^-14.9.  Forward: z - beta has r's error and three more roundings,
together under 2^-14.5 |z - beta|; z itself is rounded once, silu's own error is
below 2^-19 |z| (sigmoid: an exponential good to 2^-20, a division and two
roundings) and its slope below 1.1, so 2^-14 (|z - beta| + |z| / 16) covers both.
The mean comes from the same sums: 40 u of the mean distance from the chunk's
first row, at most 1 + D = 6 spreads, moves z by 240 u |gamma| < 2^-16 |gamma|
whatever x is (near z = beta nothing else covers it).
Backward (mean and rstd are given): sums of n terms in fp32 over a chunk, 40 u,
and the terms' own roundings (about 6 u, silu's slope 2^-19): 2^-18 of the sum
of magnitudes; grad_x adds about ten roundings of |r| (|t| + mean|t| + |xh|
mean|t xh|), under 2^-20 of it; then h."""
import numpy as np
import pytest
import torch

import scale_deformable_attention_03_b200 as msda

pytestmark = pytest.mark.gpu

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
F32, BF16 = torch.float32, torch.bfloat16

# levels, gap rows after each, C, G
SHAPES = [
    ([(1, 1)], 0, 8, 1),
    ([(1, 1), (2, 3)], 1, 8, 8),
    ([(7, 11), (3, 5), (1, 2)], 2, 96, 12),
    ([(20, 25), (10, 13)], 0, 256, 32),
    ([(9, 15)], 3, 64, 64),
    ([(5, 7), (33, 9)], 0, 512, 1),
    ([(6, 5)], 0, 2048, 32),
    ([(11, 13)], 0, 1000, 8),
    ([(4, 5)] * 8, 1, 40, 5),
    ([(64, 1), (65, 1), (63, 1)], 0, 256, 2),
]


def problem(levels, gap, C, G, B, xt, seed, loc=0.0, spread=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    rows = [h * w + gap for h, w in levels]
    starts = np.concatenate([[0], np.cumsum(rows)[:-1]]).astype(np.int64)
    x = (rnd(B, sum(rows), C) * spread + loc + rnd(C)).to(xt)
    return x, np.array(levels, np.int64), starts, 1 + 0.3 * rnd(len(levels), C), 0.3 * rnd(len(levels), C)


def act64(z, act):
    return torch.relu(z) if act == "relu" else z * torch.sigmoid(z) if act == "silu" else z


def forward64(x, levels, starts, G, gamma, beta, eps, act):
    B, Nv, C = x.shape
    y = torch.zeros(B, Nv, C, device="cuda", dtype=torch.float64)
    core = torch.zeros_like(y)      # |z - beta|, for the tolerance
    mean = torch.zeros(B, len(levels), G, device="cuda", dtype=torch.float64)
    rstd = torch.zeros_like(mean)
    for l, ((h, w), st) in enumerate(zip(levels, starts)):
        e = x[:, st:st + h * w].double().reshape(B, h * w, G, C // G)
        mu = e.mean((1, 3), keepdim=True)
        r = 1 / torch.sqrt(((e - mu) ** 2).mean((1, 3), keepdim=True) + eps)
        z0 = ((e - mu) * r).reshape(B, h * w, C)
        z0 = z0 * gamma[l].double() if gamma is not None else z0
        z = z0 + beta[l].double() if beta is not None else z0
        y[:, st:st + h * w] = act64(z, act)
        core[:, st:st + h * w] = z0.abs() + z.abs() / 16 + (gamma[l].abs() if gamma is not None else 1) / 4
        mean[:, l], rstd[:, l] = mu[:, 0, :, 0], r[:, 0, :, 0]
    return y, mean, rstd, core


@pytest.mark.parametrize("levels,gap,C,G", SHAPES)
@pytest.mark.parametrize("xt,yt", [(F32, F32), (F32, BF16), (BF16, BF16), (BF16, F32)])
@pytest.mark.parametrize("act", ["none", "relu", "silu"])
def test_forward(levels, gap, C, G, xt, yt, act):
    x, shapes, starts, gamma, beta = problem(levels, gap, C, G, 3, xt, C + G)
    y = torch.full(x.shape, 77.0, device="cuda", dtype=yt)
    got, mean, rstd = msda.msda_group_norm(x, shapes, starts, G, gamma, beta, activation=act, out=y)
    assert got is y
    want, m, r, core = forward64(x, shapes, starts, G, gamma, beta, 1e-5, act)
    assert bool(((rstd.double() - r).abs() <= 2.0 ** -14.5 * r).all())
    assert bool(((mean.double() - m).abs() <= 2.0 ** -22 * (m.abs() + 1 / r)).all())
    tol = 2.0 ** -14 * core + HALF[yt] * want.abs() + 2.0 ** -126
    assert bool(((y.double() - want).abs() <= tol).all())


@pytest.mark.parametrize("loc", [0.0, 1000.0, -30000.0])
def test_a_mean_far_from_zero_costs_no_precision(loc):
    levels = [(31, 17)]
    x, shapes, starts, gamma, beta = problem(levels, 0, 64, 8, 2, F32, 5, loc=loc)
    y, _, _ = msda.msda_group_norm(x, shapes, starts, 8, gamma, beta)
    want, _, _, core = forward64(x, shapes, starts, 8, gamma, beta, 1e-5, "none")
    assert bool(((y.double() - want).abs() <= 2.0 ** -14 * core + 2.0 ** -23 * want.abs()).all())


def test_without_gamma_and_beta_and_leading_dimensions():
    x, shapes, starts, _, _ = problem([(5, 6)], 0, 32, 4, 6, F32, 1)
    y, mean, rstd = msda.msda_group_norm(x.reshape(2, 3, 30, 32), shapes, starts, 4)
    assert y.shape == (2, 3, 30, 32) and mean.shape == rstd.shape == (2, 3, 1, 4)
    want, _, _, core = forward64(x, shapes, starts, 4, None, None, 1e-5, "none")
    assert bool(((y.reshape(6, 30, 32).double() - want).abs() <= 2.0 ** -14 * core).all())
    gx, gg, gb = msda.msda_group_norm_backward(x.reshape(2, 3, 30, 32), shapes, starts, 4, mean,
                                               rstd, y)
    assert gx.shape == y.shape and gg.shape == gb.shape == (1, 32)


def test_unordered_levels_and_constant_rows():
    # level 1 lies before level 0; a constant map has the spread 0: y = beta
    shapes, starts = np.array([[2, 3], [3, 3]]), np.array([10, 0])
    x = torch.full((1, 17, 16), 2.5, device="cuda")
    beta = torch.arange(32, device="cuda", dtype=F32).reshape(2, 16)
    y, mean, rstd = msda.msda_group_norm(x, shapes, starts, 2, None, beta)
    want = torch.zeros(1, 17, 16, device="cuda")
    want[:, 10:16], want[:, 0:9] = beta[0], beta[1]
    assert torch.equal(y, want) and bool((mean == 2.5).all())
    assert bool(((rstd - 1e-5 ** -0.5).abs() <= 2.0 ** -23 * 1e-5 ** -0.5 + 1e-5).all())


def test_a_nan_stays_in_its_group():
    x, shapes, starts, gamma, beta = problem([(4, 4), (2, 2)], 0, 16, 2, 2, F32, 3)
    x[1, 3, 9] = float("nan")
    y, _, _ = msda.msda_group_norm(x, shapes, starts, 2, gamma, beta)
    bad = torch.isnan(y)
    assert bool(bad[1, :16, 8:].all()) and int(bad.sum()) == 16 * 8


def backward64(x, levels, starts, G, mean, rstd, dy, gamma, beta, act):
    B, Nv, C = x.shape
    L = len(levels)
    dx, size = torch.zeros(2, B, Nv, C, device="cuda", dtype=torch.float64)
    par = torch.zeros(4, L, C, device="cuda", dtype=torch.float64)   # d_gamma, d_beta, their magnitudes
    for l, ((h, w), st) in enumerate(zip(levels, starts)):
        n = h * w
        e = x[:, st:st + n].double().reshape(B, n, G, C // G)
        mu, r = (t[:, l].double()[:, None, :, None] for t in (mean, rstd))
        hat = ((e - mu) * r).reshape(B, n, C)
        ga = gamma[l].double() if gamma is not None else torch.ones(C, device="cuda").double()
        z = hat * ga + (beta[l].double() if beta is not None else 0)
        d = dy[:, st:st + n].double()
        dz = d * (z > 0) if act == "relu" else d
        if act == "silu":
            sg = torch.sigmoid(z)
            dz = d * sg * (1 + z * (1 - sg))
        slope = 2 * d.abs() if act == "silu" else dz.abs()   # what the slope's own rounding moves
        par[0, l], par[1, l] = (dz * hat).sum((0, 1)), dz.sum((0, 1))
        par[2, l], par[3, l] = (slope * hat.abs()).sum((0, 1)), slope.sum((0, 1))
        g4 = lambda t: t.reshape(B, n, G, C // G)  # noqa: E731
        t, ta, hh = g4(dz * ga), g4(slope * ga.abs()), g4(hat)
        dx[:, st:st + n] = (r * (t - t.mean((1, 3), keepdim=True)
                                 - hh * (t * hh).mean((1, 3), keepdim=True))).reshape(B, n, C)
        size[:, st:st + n] = (r * (ta + ta.mean((1, 3), keepdim=True)
                                   + hh.abs() * (ta * hh.abs()).mean((1, 3), keepdim=True))).reshape(B, n, C)
    return dx, par[0], par[1], size, par[2], par[3]


@pytest.mark.parametrize("levels,gap,C,G", SHAPES)
@pytest.mark.parametrize("xt,dt,ot", [(F32, F32, F32), (F32, BF16, F32), (BF16, F32, BF16),
                                      (BF16, BF16, BF16), (F32, F32, BF16), (F32, BF16, BF16),
                                      (BF16, F32, F32), (BF16, BF16, F32)])
@pytest.mark.parametrize("act", ["none", "relu", "silu"])
def test_backward(levels, gap, C, G, xt, dt, ot, act):
    x, shapes, starts, gamma, beta = problem(levels, gap, C, G, 2, xt, C * 3 + G)
    y, mean, rstd = msda.msda_group_norm(x, shapes, starts, G, gamma, beta, activation=act)
    gen = torch.Generator(device="cuda").manual_seed(9)
    dy = torch.randn(x.shape, generator=gen, device="cuda").to(dt)
    used = torch.zeros(x.shape[1], dtype=torch.bool, device="cuda")
    for (h, w), st in zip(levels, starts):
        used[st:st + h * w] = True
    dy[:, ~used] = float("nan")     # rows of no level are not read
    dx = torch.full(x.shape, 55.0, device="cuda", dtype=ot)
    gg, gb = torch.full((2, len(levels), C), 55.0, device="cuda")
    msda.msda_group_norm_backward(x, shapes, starts, G, mean, rstd, dy, gamma, beta,
                                  activation=act, out=(dx, gg, gb))
    wx, wg, wb, size, sg, sb = backward64(x, shapes, starts, G, mean, rstd, dy, gamma, beta, act)
    assert bool(((gg.double() - wg).abs() <= 2.0 ** -18 * sg + 2.0 ** -24 * wg.abs()).all())
    assert bool(((gb.double() - wb).abs() <= 2.0 ** -18 * sb + 2.0 ** -24 * wb.abs()).all())
    tol = (2.0 ** -18 + 2.0 ** -20) * size + HALF[ot] * wx.abs() + 2.0 ** -126
    assert bool(((dx.double() - wx).abs() <= tol).all())


@pytest.mark.parametrize("act", ["none", "silu"])
def test_gradient_against_differences(act):
    """Central differences of the forward in 64 bits along random directions."""
    levels, G = [(5, 4), (2, 3)], 4
    x, shapes, starts, gamma, beta = problem(levels, 1, 24, G, 2, F32, 21)
    y, mean, rstd = msda.msda_group_norm(x, shapes, starts, G, gamma, beta, activation=act)
    gen = torch.Generator(device="cuda").manual_seed(2)
    dy = torch.randn(x.shape, generator=gen, device="cuda")
    dx, gg, gb = msda.msda_group_norm_backward(x, shapes, starts, G, mean, rstd, dy, gamma, beta,
                                               activation=act)
    f = lambda a, b, c: float((forward64(a, shapes, starts, G, b, c, 1e-5, act)[0] * dy).sum())  # noqa: E731
    h = 1e-5
    for k, (t, g) in enumerate(((x, dx), (gamma, gg), (beta, gb))):
        for _ in range(4):
            u = torch.randn(t.shape, generator=gen, device="cuda").double()
            args = [x.double(), gamma.double(), beta.double()]
            up, down = list(args), list(args)
            up[k], down[k] = args[k] + h * u, args[k] - h * u
            diff = (f(*up) - f(*down)) / (2 * h)
            # the difference is off by h^2 times a third derivative (about 1e-8 here), the
            # gradient by 2^-17 of the magnitudes that it adds
            assert abs(diff - float((g.double() * u).sum())) <= 2.0 ** -17 * float((g.double().abs() * u.abs()).sum()) * 4 + 1e-6


def test_relu_border_is_exact():
    # every z of the second half of the channels is exactly 0 or within an fp32 rounding of it
    C, G = 16, 2
    x = torch.randn(1, 64, C, device="cuda")
    shapes, starts = np.array([[8, 8]]), np.array([0])
    _, mean, rstd = msda.msda_group_norm(x, shapes, starts, G)
    gamma = torch.ones(1, C, device="cuda")
    beta = -((x[0, 5] - mean[0, 0].repeat_interleave(8)) * rstd[0, 0].repeat_interleave(8))[None].contiguous()
    dy = torch.ones_like(x)
    _, _, gb = msda.msda_group_norm_backward(x, shapes, starts, G, mean, rstd, dy, gamma, beta,
                                             activation="relu")
    z = ((x.double() - mean.double()[0, 0].repeat_interleave(8)) * rstd.double()[0, 0].repeat_interleave(8)
         + beta.double())
    assert torch.equal(gb[0], (z > 0).sum((0, 1)).float())


def test_same_bits_streams_and_capture():
    x, shapes, starts, gamma, beta = problem([(40, 50), (20, 25)], 0, 256, 32, 3, BF16, 4)
    dy = torch.randn(x.shape, device="cuda")
    lib = msda.lib()
    d = msda.NormDims(3, x.shape[1], 256, 2, 32)
    ws = torch.empty(lib.msda_group_norm_workspace_size(d), dtype=torch.uint8, device="cuda")
    wb = torch.empty(lib.msda_group_norm_backward_workspace_size(d), dtype=torch.uint8, device="cuda")
    y, mean, rstd = msda.msda_group_norm(x, shapes, starts, 32, gamma, beta, activation="silu")
    grads = msda.msda_group_norm_backward(x, shapes, starts, 32, mean, rstd, dy, gamma, beta, "silu")
    first = [t.clone() for t in (y, mean, rstd) + grads]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    again = msda.msda_group_norm(x, shapes, starts, 32, gamma, beta, activation="silu", stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        msda.msda_group_norm(x, shapes, starts, 32, gamma, beta, activation="silu", out=y, mean=mean,
                             rstd=rstd, workspace=ws)
        msda.msda_group_norm_backward(x, shapes, starts, 32, mean, rstd, dy, gamma, beta, "silu",
                                      out=grads, workspace=wb)
    for t in (y, mean, rstd) + grads:
        t.zero_()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, (y, mean, rstd) + grads))


def test_empty_batch():
    x = torch.empty(0, 6, 16, device="cuda")
    shapes, starts = np.array([[2, 3]]), np.array([0])
    y, mean, rstd = msda.msda_group_norm(x, shapes, starts, 4)
    gx, gg, gb = msda.msda_group_norm_backward(x, shapes, starts, 4, mean, rstd, y)
    assert y.shape == gx.shape == (0, 6, 16) and bool((gg == 0).all()) and bool((gb == 0).all())


def test_refusals():
    x = torch.randn(2, 12, 16, device="cuda")
    ok, st = np.array([[3, 4]]), np.array([0])
    f = msda.msda_group_norm
    mean = torch.zeros(2, 1, 4, device="cuda")
    for call in (lambda: f(x.half(), ok, st, 4), lambda: f(x.cpu(), ok, st, 4),
                 lambda: f(x.transpose(1, 2), ok, st, 4), lambda: f(x, ok, st, 5),
                 lambda: f(x, ok, st, 0), lambda: f(x, ok, st, 4, eps=0.0),
                 lambda: f(x, ok, st, 4, activation="tanh"), lambda: f(x, ok, st, 4, out=x),
                 lambda: f(x, np.array([[3, 5]]), st, 4),
                 lambda: f(x, np.array([[2, 3], [2, 3]]), np.array([0, 5]), 4),
                 lambda: f(x, ok, np.array([0, 1]), 4),
                 lambda: f(x, ok, st, 4, gamma=torch.ones(1, 8, device="cuda")),
                 lambda: f(x, ok, st, 4, gamma=torch.ones(1, 16, device="cuda").bfloat16()),
                 lambda: f(x, ok, st, 4, out_dtype=torch.float16),
                 lambda: f(torch.randn(2, 12, 12, device="cuda"), ok, st, 4),
                 lambda: f(torch.randn(2, 12, 4096, device="cuda"), ok, st, 4),
                 lambda: f(x, ok, st, 4, workspace=torch.empty(16, dtype=torch.uint8, device="cuda")),
                 lambda: msda.msda_group_norm_backward(x, ok, st, 4, mean, mean, x[:1]),
                 lambda: msda.msda_group_norm_backward(x, ok, st, 4, mean[:1], mean, x),
                 lambda: msda.msda_group_norm_backward(
                     x, ok, st, 4, mean, mean, x, out=(x, mean, mean))):
        with pytest.raises(msda.MsdaError):
            call()
