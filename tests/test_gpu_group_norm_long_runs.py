"""The group norm where a thread adds up many rows: a first row far from the
others, a blank corner under a large mean, gradients without a sign of their own.

Bounds, for any data (u = 2^-24; N values of a group with the mean m, X_i = x_i - m,
M = sum X^2, s = sqrt(M / N)).  A thread adds eight rows of a channel in fp32, relative to
the first of the eight, whose X is B; everything beyond is double.
  The eight rows' sum of d = x - x_first: each d is rounded (u), seven additions: off by
  8 u sum |d|; their sum of d^2: 10 u sum d^2.
  Mean: sum over all blocks of 8 u sum |d| <= 8 u sum (|X| + |B|) <= 8 u N s (1 + sqrt(8)),
  since the 8 B^2 of a block are at most eight times its own sum of X^2: 31 u s.
  M: the sums' errors enter as 2 B times that of d, 16 u |B| sum |d| <= 16 u (|B| sum |X| +
  8 B^2) <= 16 u (12 B^2 + sum X^2 / 2) <= 200 u sum X^2, and as 10 u sum d^2 <= 20 u
  (sum X^2 + 8 B^2) <= 180 u sum X^2.  Together 380 u M, half of it for r: 190 u.
  r itself and mean are rounded once more (u).  z - beta: 190 u and three roundings of
  itself, and the mean's 31 u |gamma| (s r <= 1): 2^-16 |z - beta| + 2^-19 |gamma|.
Gradients: blocks of eight terms in fp32, each term off by 6 u of itself, then double, and
one rounding of a run's sum and of the result: 16 u = 2^-20 of the sum of magnitudes;
grad_x adds ten roundings of r (|t| + mean |t| + |xh| mean |t xh|): 2^-19 of it in all."""
import numpy as np
import pytest
import torch

import scale_deformable_attention_03_b200 as msda

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
HALF = {F32: 2.0 ** -24, BF16: 2.0 ** -8}
CAMERA = [(116, 200), (58, 100)]

# items, levels, C, G; rows of a channel that one thread adds up
LONG = [
    (6, CAMERA, 256, 32),          # 73
    (4, [(512, 480)], 512, 8),     # 830
    (1, [(1000, 237)], 2048, 32),  # 800
    (3, [(40, 41)], 40, 5),        # 4, of 51 threads side by side
]


def far_first_row(B, levels, C, far, dtype, seed, blank):
    """Features of spread 1 around 0 whose first row of each level is `far` (a spike), or
    around `far` with a first row of zeros (a blank corner)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows = [h * w for h, w in levels]
    starts = np.concatenate([[0], np.cumsum(rows)[:-1]]).astype(np.int64)
    x = torch.randn(B, sum(rows), C, generator=g, device="cuda")
    if blank:
        x += far
    for st in starts:
        x[:, int(st)] = 0.0 if blank else far
    gamma = 1 + 0.3 * torch.randn(len(levels), C, generator=g, device="cuda")
    beta = 0.3 * torch.randn(len(levels), C, generator=g, device="cuda")
    return x.to(dtype), np.array(levels, np.int64), starts, gamma, beta


def levels64(x, levels, starts, G):
    """Per item and level: the rows, their values in 64 bits [rows, G, C / G], mean and r [G]."""
    for b in range(x.shape[0]):
        for l, ((h, w), st) in enumerate(zip(levels, starts)):
            at = slice(int(st), int(st) + h * w)
            e = x[b, at].double().view(h * w, G, -1)
            mu = e.mean((0, 2), keepdim=True)
            r = 1 / torch.sqrt(((e - mu) ** 2).mean((0, 2), keepdim=True) + 1e-5)
            yield b, l, at, e, mu, r


@pytest.mark.parametrize("B,levels,C,G", LONG)
@pytest.mark.parametrize("far", [30.0, 300.0, 3000.0, -1e6])
@pytest.mark.parametrize("blank", [False, True])
@pytest.mark.parametrize("xt,yt", [(F32, F32), (BF16, BF16)])
def test_a_first_row_far_from_the_others(B, levels, C, G, far, blank, xt, yt):
    x, shapes, starts, gamma, beta = far_first_row(B, levels, C, far, xt, 3, blank)
    y, mean, rstd = msda.msda_group_norm(x, shapes, starts, G, gamma, beta, out_dtype=yt)
    for b, l, at, e, mu, r in levels64(x, levels, starts, G):
        r0, m0 = r[0, :, 0], mu[0, :, 0]
        assert bool(((rstd[b, l].double() - r0).abs() <= 2.0 ** -16 * r0).all()), (b, l)
        assert bool(((mean[b, l].double() - m0).abs() <= 2.0 ** -19 / r0 + 2.0 ** -24 * m0.abs()).all()), (b, l)
        z = ((e - mu) * r).view(-1, C) * gamma[l].double()
        want = z + beta[l].double()
        tol = 2.0 ** -16 * z.abs() + 2.0 ** -19 * gamma[l].double().abs() + (HALF[yt] + 2.0 ** -24) * want.abs()
        assert bool(((y[b, at].double() - want).abs() <= tol).all()), (b, l)


@pytest.mark.parametrize("B,levels,C,G", LONG)
@pytest.mark.parametrize("dy", [0.1, -0.7, None])
def test_gradients_of_one_sign(B, levels, C, G, dy):
    """A loss that is a mean gives every row the same gradient: roundings do not cancel."""
    x, shapes, starts, gamma, beta = far_first_row(B, levels, C, 2.0, F32, 4, False)
    gen = torch.Generator(device="cuda").manual_seed(5)
    g = torch.full_like(x, dy) if dy else torch.rand(x.shape, generator=gen, device="cuda")
    _, mean, rstd = msda.msda_group_norm(x, shapes, starts, G, gamma, beta)
    gx, gg, gb = msda.msda_group_norm_backward(x, shapes, starts, G, mean, rstd, g, gamma, beta)
    sums = torch.zeros(4, len(levels), C, device="cuda", dtype=torch.float64)
    for b, l, at, e, _, _ in levels64(x, levels, starts, G):
        mu, r = (t[b, l].double()[None, :, None] for t in (mean, rstd))
        hat = (e - mu) * r
        d = g[b, at].double().view_as(e)
        for k, t in enumerate((d * hat, d, (d * hat).abs(), d.abs())):
            sums[k, l] += t.sum(0).view(-1)
        t = d * gamma[l].double().view(1, G, -1)
        avg = lambda v: v.mean((0, 2), keepdim=True)  # noqa: E731
        want = r * (t - avg(t) - hat * avg(t * hat))
        size = r * (t.abs() + avg(t.abs()) + hat.abs() * avg((t * hat).abs()))
        assert bool(((gx[b, at].double().view_as(e) - want).abs() <= 2.0 ** -19 * size + 2.0 ** -24 * want.abs()).all()), (b, l)
    assert bool(((gg.double() - sums[0]).abs() <= 2.0 ** -20 * sums[2] + 2.0 ** -24 * sums[0].abs()).all())
    assert bool(((gb.double() - sums[1]).abs() <= 2.0 ** -20 * sums[3] + 2.0 ** -24 * sums[1].abs()).all())


def test_gradient_behind_the_2_31st_element():
    """The last of five items of 2^20 rows of 512 against the formula, and the parameters'
    gradients over all of them."""
    gen = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn(5, 1 << 20, 512, generator=gen, device="cuda", dtype=BF16)
    g = torch.randn(5, 1 << 20, 512, generator=gen, device="cuda", dtype=BF16)
    shapes, starts, G = np.array([[1024, 1024]]), np.array([0]), 8
    _, mean, rstd = msda.msda_group_norm(x, shapes, starts, G)
    gx, gg, gb = msda.msda_group_norm_backward(x, shapes, starts, G, mean, rstd, g)
    sums = torch.zeros(4, 512, device="cuda", dtype=torch.float64)
    for b in range(5):
        hat = (x[b].double().view(-1, G, 64) - mean[b, 0].double()[:, None]) * rstd[b, 0].double()[:, None]
        d = g[b].double().view_as(hat)
        for k, t in enumerate((d * hat, d, (d * hat).abs(), d.abs())):
            sums[k] += t.sum(0).view(-1)
        if b in (0, 4):
            avg = lambda v: v.mean((0, 2), keepdim=True)  # noqa: E731
            r = rstd[b, 0].double()[:, None]
            want = r * (d - avg(d) - hat * avg(d * hat))
            size = r * (d.abs() + avg(d.abs()) + hat.abs() * avg((d * hat).abs()))
            off = (gx[b].double().view_as(hat) - want).abs()
            assert bool((off <= 2.0 ** -19 * size + HALF[BF16] * want.abs()).all()), b
            del want, size, off
        del hat, d
    assert bool(((gg[0].double() - sums[0]).abs() <= 2.0 ** -20 * sums[2] + 2.0 ** -24 * sums[0].abs()).all())
    assert bool(((gb[0].double() - sums[1]).abs() <= 2.0 ** -20 * sums[3] + 2.0 ** -24 * sums[1].abs()).all())
