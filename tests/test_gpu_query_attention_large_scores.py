"""msda_query_attention and its backward where scores are far from zero: a tau that cuts
off all keys but the nearest, a bias of thousands, products of thousands.

A cut-off: queries lie a quarter from their nearest key on a line of keys one apart, so
with tau T the nearest key's score is -T / 4 and the next one's -3 T / 4.  The fp32 scores
are off by 2^-20 of themselves at most, so from T = 1e8 on every other weight is exactly 0
and the nearest one's 1 (the score is its row's own reference, whatever its rounding):
out is that key's v, bit for bit, and lse is -T / 4 to 2^-20 of itself and the products
(under 32 |q| |k| scale = 200).  In the gradient p is 1 and D = dp up to the order of their
32 products (40 u a, a = sum |do v|), so ds is at most 80 u a = 2^-17 a, which is all that
grad_q, grad_k and grad_tau are made of, and grad_v_j is the sum of its queries' grad_out
in fp32, rounded once.  The backward knows the row's reference from lse only; scores and lse
are formed the same way in both, so their difference is exactly 0 at the nearest key as long
as the logarithm of the sum of weights is 0, which it is here."""
import math

import pytest
import torch

import scale_deformable_attention_03_b200 as msda
from tests import test_gpu_query_attention as attention

pytestmark = pytest.mark.gpu

# split keys, one tile, more tiles than the visibility is looked up for at once, two heads per CTA
SIZES = [(1, 300, 200, 2), (2, 5, 700, 2), (1, 40, 9, 3), (1, 70, 20_000, 1), (4, 2400, 75, 8)]


def line(B, Nq, Nk, H, tau, groups, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    a = dict(q=rnd(B, Nq, H, 32).bfloat16(), k=rnd(B, Nk, H, 32).bfloat16(), v=rnd(B, Nk, H, 32).bfloat16())
    near = torch.stack([torch.randperm(Nq, generator=g, device="cuda") % Nk for _ in range(B)])
    a["q_points"], a["k_points"] = torch.zeros(B, Nq, 2, device="cuda"), torch.zeros(B, Nk, 2, device="cuda")
    a["q_points"][..., 0] = near + 0.25
    a["k_points"][..., 0] = torch.arange(Nk, device="cuda")
    a["tau"] = torch.full((B, Nq, H), tau, device="cuda")
    if groups:   # everybody's keys, and a padding query that sees none
        a["q_group"] = torch.ones(B, Nq, dtype=torch.int32, device="cuda")
        a["k_group"] = torch.zeros(B, Nk, dtype=torch.int32, device="cuda")
        a["q_group"][:, -1] = -1
    return a, near


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("tau", [1e8, 3e9, 1e10, 7.7e12, 1e20, 1e30])
@pytest.mark.parametrize("groups", [False, True])
def test_a_tau_that_cuts_off_all_but_the_nearest(size, tau, groups):
    B, Nq, Nk, H = size
    a, near = line(*size, tau, groups, sum(size))
    on = torch.ones(B, Nq, dtype=torch.bool, device="cuda")
    if groups:
        on[:, -1] = False
    out, lse = msda.msda_query_attention(**a)
    want = torch.gather(a["v"], 1, near[:, :, None, None].expand(B, Nq, H, 32)) * on[..., None, None]
    assert torch.equal(out.view(B, Nq, H, 32), want)
    off = (lse.double() + tau / 4).abs()
    assert bool((off.permute(0, 2, 1)[on] <= 2.0 ** -20 * tau / 4 + 200).all())
    assert bool((lse.permute(0, 2, 1)[~on] == -math.inf).all())
    do = torch.randn(B, Nq, H * 32, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).bfloat16()
    gq, gk, gv, gt = msda.msda_query_attention_backward(**a, lse=lse, grad_out=do)
    d = do.double().view(B, Nq, H, 32) * on[..., None, None]
    at = near[:, :, None, None].expand(B, Nq, H, 32)
    ds = 2.0 ** -17 * (d * want.double()).abs().sum(-1, keepdim=True)
    sums = torch.zeros(3, B, Nk, H, 32, device="cuda", dtype=torch.float64)
    sums[0].scatter_add_(1, at, d)
    sums[1].scatter_add_(1, at, d.abs())
    sums[2].scatter_add_(1, at, ds * a["q"].double().abs())
    near_k = torch.gather(a["k"], 1, at).double().abs()
    assert bool((gq.double().abs() <= ds * near_k).all())
    assert bool((gk.double().abs() <= sums[2]).all())
    assert bool((gt.double().abs() <= ds[..., 0]).all())
    assert bool(((gv.double() - sums[0]).abs() <= 2.0 ** -16 * sums[1] + 2.0 ** -8 * sums[0].abs()).all())


@pytest.mark.parametrize("size", SIZES + [(1, 900, 900, 8)])
@pytest.mark.parametrize("tau", [1e8, 1e10, 1e30])
@pytest.mark.parametrize("groups", [False, True])
def test_a_cut_off_with_the_own_key_at_distance_zero(size, tau, groups):
    """The score of the own key is near zero, those of all others are far: with split keys only
    some CTAs of a cluster end far.  Every other weight is 0, the own one 1 up to e = 40 u S +
    2^-19 = 2^-16 (S = scale sum |q k| < 100), twice that and a rounding to bf16 in out."""
    B, Nq, Nk, H = size
    a, near = line(*size, tau, groups, 80 + sum(size))
    a["q_points"][..., 0] = near
    on = torch.ones(B, Nq, 1, 1, device="cuda", dtype=torch.float64)
    if groups:
        on[:, -1] = 0
    out, lse = msda.msda_query_attention(**a)
    at = near[:, :, None, None].expand(B, Nq, H, 32)
    k, v = (torch.gather(a[n].double(), 1, at) for n in ("k", "v"))
    want = v * on
    assert bool(((out.double().view(B, Nq, H, 32) - want).abs() <= (2.0 ** -7 + 2.0 ** -15) * want.abs()).all())
    score = 32 ** -0.5 * (a["q"].double() * k).sum(-1)
    off = (lse.permute(0, 2, 1).double() - score).abs()[on[..., 0, 0] > 0]
    assert bool((off <= 2.0 ** -16).all())
    do = torch.randn(B, Nq, H * 32, device="cuda", generator=torch.Generator(device="cuda").manual_seed(6)).bfloat16()
    gq, gk, gv, gt = msda.msda_query_attention_backward(**a, lse=lse, grad_out=do)
    d = do.double().view(B, Nq, H, 32) * on
    ds = 2.0 ** -14 * (d * v).abs().sum(-1, keepdim=True)   # p (dp - p dp), each p off by 2^-16
    sums = torch.zeros(3, B, Nk, H, 32, device="cuda", dtype=torch.float64)
    sums[0].scatter_add_(1, at, d)
    sums[1].scatter_add_(1, at, d.abs())
    sums[2].scatter_add_(1, at, ds * a["q"].double().abs())
    assert bool((gq.double().abs() <= ds * k.abs()).all())
    assert bool((gk.double().abs() <= sums[2]).all())
    assert bool((gt == 0).all())   # the only pair with a weight has the distance 0
    assert bool(((gv.double() - sums[0]).abs() <= (2.0 ** -8 + 2.0 ** -14) * sums[1] + 2.0 ** -8 * sums[0].abs()).all())


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("tau", [3e7, 1e10, 1e20])
@pytest.mark.parametrize("groups", [False, True])
def test_two_keys_at_the_same_distance(size, tau, groups):
    """Half-way between two keys, with q = 0: the weights are a half each, although lse has no
    room for the logarithm of 2.  Tolerances: a half is exact, also in bf16; D and dp as above,
    so ds is off by 2^-17 a, a = sum over both of |do v|, beside what bf16 leaves over (h |ds|)."""
    B, Nq, Nk, H = size
    a, near = line(*size, tau, groups, 70 + sum(size))
    near = near % (Nk - 1)
    a["q_points"][..., 0] = near + 0.5
    a["q"].zero_()
    on = torch.ones(B, Nq, 1, 1, device="cuda", dtype=torch.float64)
    if groups:
        on[:, -1] = 0
    out, lse = msda.msda_query_attention(**a)
    at = [(near + i)[:, :, None, None].expand(B, Nq, H, 32) for i in (0, 1)]
    k, v = ([torch.gather(a[n].double(), 1, i) for i in at] for n in ("k", "v"))
    want = (v[0] + v[1]) / 2 * on
    got = out.double().view(B, Nq, H, 32)
    assert bool(((got - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -22 * (v[0].abs() + v[1].abs())).all())
    do = torch.randn(B, Nq, H * 32, device="cuda", generator=torch.Generator(device="cuda").manual_seed(5)).bfloat16()
    gq, gk, gv, gt = msda.msda_query_attention_backward(**a, lse=lse, grad_out=do)
    d = do.double().view(B, Nq, H, 32) * on
    dp = [(d * t).sum(-1, keepdim=True) for t in v]
    ds = (dp[0] - dp[1]) / 4                     # of the first; the second's is its negative
    off = 2.0 ** -17 * sum((d * t).abs().sum(-1, keepdim=True) for t in v)
    scale = 32 ** -0.5
    want = scale * ds * (k[0] - k[1])
    tol = scale * (off + 2.0 ** -8 * ds.abs()) * (k[0].abs() + k[1].abs()) + 2.0 ** -8 * want.abs()
    assert bool(((gq.double() - want).abs() <= tol).all())
    assert bool((gk == 0).all())
    assert bool((gt.double().abs() <= off[..., 0] + 2.0 ** -20 * ds.abs()[..., 0]).all())
    sums = torch.zeros(2, B, Nk, H, 32, device="cuda", dtype=torch.float64)
    for i in at:
        sums[0].scatter_add_(1, i, d / 2)
        sums[1].scatter_add_(1, i, d.abs() / 2)
    assert bool(((gv.double() - sums[0]).abs() <= 2.0 ** -16 * sums[1] + 2.0 ** -8 * sums[0].abs()).all())


@pytest.mark.parametrize("size", [(1, 300, 301, 8), (2, 1, 4097, 2), (1, 70, 129, 1), (4, 2400, 75, 8)])
@pytest.mark.parametrize("groups", [None, "shared"])
@pytest.mark.parametrize("shift", [300.0, 3000.0, 30000.0])
def test_a_bias_of_thousands(size, groups, shift):
    """All keys far away from the queries: every score is near -tau shift, the differences
    are what the weights are made of.  Tolerances: the general ones, on these magnitudes."""
    a = attention.problem(*size, True, groups, 50 + sum(size))
    a["k_points"][..., 0] += shift
    a["tau"] = a["tau"] + 2
    out, lse = msda.msda_query_attention(**a)
    attention.check_forward(a, out, lse)
    B, Nq, Nk, H = size
    do = torch.randn(B, Nq, H * 32, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2)).bfloat16()
    grads = msda.msda_query_attention_backward(**a, lse=lse, grad_out=do)
    assert all(bool(torch.isfinite(t).all()) for t in grads)
    attention.check_backward(a, do, grads)


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("size", [(2, 100, 32, 2), (1, 33, 300, 1)])
@pytest.mark.parametrize("big", [2.0 ** 14, 2.0 ** 30, 2.0 ** 60])
def test_products_that_leave_one_key(size, bias, big):
    """q_i . k_j scale is `big` for one key and 0 for the others."""
    B, Nq, Nk, H = size
    a = attention.problem(*size, bias, None, 9, joint=False)
    if bias:
        a["tau"] = a["tau"].abs()
    a["q"].zero_()
    a["k"].zero_()
    for i in range(Nq):
        a["q"][:, i, :, i % 32] = big
    for j in range(32):
        a["k"][:, (j * 7) % Nk, :, j] = 1.0
    near = torch.tensor([(i % 32) * 7 % Nk for i in range(Nq)], device="cuda").expand(B, Nq)
    out, lse = msda.msda_query_attention(**a, scale=1.0)
    at = near[:, :, None, None].expand(B, Nq, H, 32)
    assert torch.equal(out.view(B, Nq, H, 32), torch.gather(a["v"], 1, at))
    assert bool(((lse.double() - big).abs() <= 2.0 ** -22 * big + 30).all())
    do = torch.randn(B, Nq, H * 32, device="cuda").bfloat16()
    gq, gk, gv, gt = msda.msda_query_attention_backward(**a, lse=lse, grad_out=do, scale=1.0)
    # p = 1 up to lse's own rounding (2^-24 of 2^14 at most where the bias gives the score more
    # digits than it holds; beyond that it holds the score itself)
    d = do.double().view(B, Nq, H, 32)
    sums = torch.zeros(2, B, Nk, H, 32, device="cuda", dtype=torch.float64)
    sums[0].scatter_add_(1, at, d)
    sums[1].scatter_add_(1, at, d.abs())
    assert bool(((gv.double() - sums[0]).abs() <= (2.0 ** -8 + 2.0 ** -8) * sums[1]).all())
    assert all(bool(torch.isfinite(t).all()) for t in (gq, gk, gv) + ((gt,) if bias else ()))


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("size", [(2, 100, 32, 2), (1, 33, 3000, 1), (4, 2400, 75, 8)])
@pytest.mark.parametrize("scale,one", [(1e-6, 2.0 ** 40), (1e6, 1.0), (1e6, 2.0 ** 70)])
def test_the_smallest_and_largest_scale(size, bias, scale, one):
    """q_i . k_j is `one` for one key and 0 for the others; with a bias the score is a million
    times larger than that at most.  One weight is 1, the others are 0 (1e6 apart)."""
    B, Nq, Nk, H = size
    a = attention.problem(*size, bias, None, 11, joint=False)
    a["q"].zero_()
    a["k"].zero_()
    i = torch.arange(Nq, device="cuda")
    a["q"][:, i, :, i % 32] = one
    j = torch.arange(32, device="cuda")
    a["k"][:, (j * 7) % Nk, :, j] = 1.0
    near = ((i % 32) * 7 % Nk).expand(B, Nq)
    out, lse = msda.msda_query_attention(**a, scale=scale)
    at = near[:, :, None, None].expand(B, Nq, H, 32)
    v = torch.gather(a["v"], 1, at)
    assert torch.equal(out.view(B, Nq, H, 32), v)
    want = one * scale
    if bias:
        b = torch.arange(B, device="cuda")[:, None]
        d = (a["q_points"].double() - a["k_points"].double()[b, near]).norm(dim=-1)
        want = want - a["tau"].double() * d[..., None]
    assert bool(((lse.permute(0, 2, 1).double() - want).abs() <= 2.0 ** -21 * one * scale).all())
    do = torch.randn(B, Nq, H * 32, device="cuda", generator=torch.Generator(device="cuda").manual_seed(7)).bfloat16()
    gq, gk, gv, gt = msda.msda_query_attention_backward(**a, lse=lse, grad_out=do, scale=scale)
    d = do.double().view(B, Nq, H, 32)
    ds = 2.0 ** -17 * (d * v.double()).abs().sum(-1, keepdim=True)
    sums = torch.zeros(2, B, Nk, H, 32, device="cuda", dtype=torch.float64)
    sums[0].scatter_add_(1, at, d)
    sums[1].scatter_add_(1, at, d.abs())
    assert bool(((gv.double() - sums[0]).abs() <= 2.0 ** -16 * sums[1] + 2.0 ** -8 * sums[0].abs()).all())
    assert bool((gq.double().abs() <= scale * ds * 1.01).all())
    assert gt is None or bool((gt.double().abs() <= 2 * ds[..., 0]).all())


@pytest.mark.parametrize("Nk", [90, 900])
def test_a_nan_in_a_live_query_is_not_hidden(Nk):
    a = attention.problem(1, 20, Nk, 2, True, None, 3, joint=False)
    a["q"][0, 7, 0, 5] = float("nan")
    out, lse = msda.msda_query_attention(**a)
    assert bool(torch.isnan(out[0, 7, :32]).all()) and bool(torch.isnan(lse[0, 0, 7]))
    keep = torch.ones(20, dtype=torch.bool, device="cuda")
    keep[7] = False
    assert bool(torch.isfinite(out[0, keep]).all()) and bool(torch.isfinite(lse[0, :, keep]).all())


@pytest.mark.parametrize("size", [(2, 150, 260, 2), (1, 70, 1500, 2), (4, 2400, 75, 8)])
@pytest.mark.parametrize("holds", [float("nan"), 1e4, -1e30])
def test_what_padding_holds_moves_no_bit(size, holds):
    B, Nq, Nk, H = size
    a = attention.problem(*size, True, "shared", 60 + sum(size), joint=False)
    do = torch.randn(B, Nq, H * 32, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3)).bfloat16()
    results = []
    for value in (0.0, holds):
        for name, t in dict(a, do=do).items():
            if t.is_floating_point():
                pad = (a["k_group"] if name in ("k", "v", "k_points") else a["q_group"]) < 0
                t[pad] = value
        out, lse = msda.msda_query_attention(**a)
        results.append((out, lse) + msda.msda_query_attention_backward(**a, lse=lse, grad_out=do))
    assert all(torch.equal(x, y) for x, y in zip(*results))
