"""msda_query_attention and its backward against the formulas in 64 bits.

Tolerances, from the roundings, on each problem's own magnitudes (u = 2^-24,
h = 2^-8 the half step of bf16).  A score sums 32 products in fp32 and takes
four more roundings: it is off by 40 u S, S_ij = scale sum |q k| + |tau| dist,
and so is lse (plus 2^-23 of itself and 2^-20 for the base-2 exponentials and
the logarithm).  A weight p is then off by e = 40 u (max S + |lse|) + 2^-19 of
itself (twice that with the sum it is divided by).
  out: 2 e + h (the weights' rounding) of sum p |v|, plus h |out|.
  grad_v: e + h of sum_i p |do|, plus h |grad_v|.
  ds = p (dp - D): dp is off by 40 u a, a = sum |do v|; D by sum p (2 e a); so
  ds by 2 e A, A = p (a + sum p a); the products round it to bf16 (h |ds|) and
  add up in fp32 (2^-16 of the magnitudes, for up to 2^8 tiles one after the
  other); grad_q and grad_k round once more (h).
Where there are few rows, weights and ds are kept to 2^-16 instead of h: bf16 of
them and bf16 of what that leaves over."""
import math

import pytest
import torch

import scale_deformable_attention_03_b200 as msda

pytestmark = pytest.mark.gpu

U, HALF = 2.0 ** -24, 2.0 ** -8

SIZES = [(1, 1, 1, 1), (2, 1, 130, 2), (1, 65, 63, 3), (2, 128, 64, 4), (1, 300, 301, 8),
         (1, 200, 1, 2), (1, 17, 1000, 8), (3, 70, 129, 1), (1, 3, 5000, 2)]
#: two heads per CTA (the grid is large enough)
LARGE = (4, 2400, 75, 8)


def problem(B, Nq, Nk, H, bias, groups, seed, joint=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    rand = lambda *s: torch.rand(*s, generator=g, device="cuda")  # noqa: E731
    if joint:   # keys and values side by side in a wider row
        kv = rnd(B, Nk, 2, H, 32).bfloat16()
        k, v = kv[:, :, 0], kv[:, :, 1]
    else:
        k, v = rnd(B, Nk, H, 32).bfloat16(), rnd(B, Nk, H, 32).bfloat16()
    a = dict(q=rnd(B, Nq, H, 32).bfloat16(), k=k, v=v)
    if bias:
        a.update(q_points=rand(B, Nq, 2), k_points=rand(B, Nk, 2), tau=15 * rand(B, Nq, H) - 1)
    if groups:
        qg = torch.randint(0, 5, (B, Nq), generator=g, device="cuda", dtype=torch.int32)
        kg = torch.sort(torch.randint(-1, 7, (B, Nk), generator=g, device="cuda", dtype=torch.int32),
                        dim=1).values.contiguous()
        if groups == "no shared":
            kg[kg == 0] = 1
        qg[:, Nq // 2:Nq // 2 + 3] = -1 if Nq > 3 else 9
        qg[:, -1] = 9        # a group that no key has: sees group 0 only, or nothing
        a.update(q_group=qg, k_group=kg)
        # padding holds anything
        a["q"][qg < 0] = float("nan")
        a["k"][kg < 0] = float("nan")
        a["v"][kg < 0] = float("inf")
        if bias:
            a["q_points"][qg < 0] = float("inf")
            a["k_points"][kg < 0] = float("nan")
            a["tau"][qg < 0] = float("nan")
    return a


def clean(a):
    """The inputs in 64 bits, with zeros where padding holds anything."""
    c = {n: t.double() if t.is_floating_point() else t for n, t in a.items()}
    for n, t in c.items():
        if t.is_floating_point():
            c[n] = torch.nan_to_num(t, 0.0, 0.0, 0.0)
    return c


def heads64(a, b, h):
    """Scores, visibility, distances and magnitudes of one head."""
    c = {n: t[0] for n, t in clean({n: t[b:b + 1] for n, t in a.items()}).items()}
    scale = 32 ** -0.5
    q, k = c["q"][:, h], c["k"][:, h]
    s, S = scale * q @ k.T, scale * q.abs() @ k.abs().T
    dist = None
    if "tau" in c:
        dist = torch.cdist(c["q_points"], c["k_points"], compute_mode="donot_use_mm_for_euclid_dist")
        s = s - c["tau"][:, h, None] * dist
        S = S + c["tau"][:, h, None].abs() * dist
    sees = torch.ones(s.shape, dtype=torch.bool, device="cuda")
    if "q_group" in c:
        qg, kg = c["q_group"][:, None], c["k_group"][None]
        sees = (qg >= 0) & (kg >= 0) & ((kg == 0) | (kg == qg))
    s = s.masked_fill(~sees, -math.inf)
    S = torch.where(sees, S, 0.0)
    lse = torch.logsumexp(s, 1) if s.shape[1] else torch.full((s.shape[0],), -math.inf, device="cuda").double()
    p = torch.exp(s - torch.where(lse.isinf(), 0.0, lse)[:, None])
    top = S.amax(1) if s.shape[1] else torch.zeros_like(lse)
    e = 40 * U * (top + torch.where(lse.isinf(), 0.0, lse).abs()) + 2.0 ** -19
    return q, k, c["v"][:, h], p, lse, dist, S, e


def check_forward(a, out, lse, heads=None, weight=HALF):
    B, Nq, H, _ = a["q"].shape
    for b in range(B):
        for h in heads or range(H):
            q, k, v, p, want_lse, _, S, e = heads64(a, b, h)
            want = p @ v
            got = out[b, :, 32 * h:32 * h + 32].double()
            tol = (2 * e[:, None] + weight) * (p @ v.abs()) + HALF * want.abs() + 2.0 ** -126
            assert bool(((got - want).abs() <= tol).all()), (b, h)
            empty = want_lse.isinf()
            assert torch.equal(lse[b, h].isinf(), empty)
            assert bool((got[empty] == 0).all()) and bool((lse[b, h][empty] < 0).all())
            off = (lse[b, h].double() - want_lse).abs()[~empty]
            assert bool((off <= (e + 2.0 ** -23 * want_lse.abs())[~empty]).all()), (b, h)


def check_backward(a, do, grads, heads=None, weight=HALF):
    gq, gk, gv, gt = grads
    B, Nq, H, _ = a["q"].shape
    scale = 32 ** -0.5
    for b in range(B):
        for h in heads or range(H):
            q, k, v, p, lse, dist, S, e = heads64(a, b, h)
            d = torch.nan_to_num(do[b, :, 32 * h:32 * h + 32].double(), 0.0, 0.0, 0.0)
            dp, ab = d @ v.T, d.abs() @ v.abs().T
            D = (p * dp).sum(1, keepdim=True)
            ds = p * (dp - D)
            A = 2 * e[:, None] * p * (ab + (p * ab).sum(1, keepdim=True))
            near = lambda got, want, tol: bool(((got.double() - want).abs() <= tol + 2.0 ** -126).all())  # noqa: E731
            w = weight * ds.abs() + A + 2.0 ** -16 * ds.abs()
            assert near(gv[b, :, h], p.T @ d, ((e[:, None] + weight + 2.0 ** -16) * p).T @ d.abs()
                        + HALF * (p.T @ d).abs()), ("v", b, h)
            assert near(gq[b, :, h], scale * ds @ k, scale * w @ k.abs() + HALF * (scale * ds @ k).abs()), ("q", b, h)
            assert near(gk[b, :, h], scale * ds.T @ q, scale * w.T @ q.abs() + HALF * (scale * ds.T @ q).abs()), ("k", b, h)
            if dist is not None:
                assert near(gt[b, :, h], -(ds * dist).sum(1),
                            ((A + 2.0 ** -16 * ds.abs()) * dist).sum(1)), ("tau", b, h)


MODES = [(False, None), (True, None), (False, "shared"), (True, "shared"), (True, "no shared")]


@pytest.mark.parametrize("size", SIZES + [LARGE])
@pytest.mark.parametrize("bias,groups", MODES)
def test_forward(size, bias, groups):
    a = problem(*size, bias, groups, sum(size))
    B, Nq, Nk, H = size
    flat = torch.full((B * Nq * H * 32 + 64,), 9.0, device="cuda", dtype=torch.bfloat16)
    out = flat[32:-32].view(B, Nq, H * 32)
    got, lse = msda.msda_query_attention(**a, out=out)
    check_forward(a, out, lse)
    assert bool((flat[:32] == 9).all()) and bool((flat[-32:] == 9).all())


@pytest.mark.parametrize("size", SIZES + [LARGE])
@pytest.mark.parametrize("bias,groups", MODES)
def test_backward(size, bias, groups):
    a = problem(*size, bias, groups, 1 + sum(size))
    B, Nq, Nk, H = size
    _, lse = msda.msda_query_attention(**a)
    do = torch.randn(B, Nq, H * 32, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3)).bfloat16()
    if groups:
        do[a["q_group"] < 0] = float("nan")
    grads = msda.msda_query_attention_backward(**a, lse=lse, grad_out=do)
    assert all(g is None or bool(torch.isfinite(g).all()) for g in grads)
    check_backward(a, do, grads)


@pytest.mark.parametrize("size", [(2, 1, 4097, 8), (1, 64, 300, 16), (3, 300, 17, 2), (1, 5, 5, 1)])
@pytest.mark.parametrize("bias,groups", [(False, None), (True, None), (False, "shared"), (True, "shared")])
def test_few_rows_keep_their_weights(size, bias, groups):
    """Up to 1024 rows the outputs are off by their own rounding and fp32's errors."""
    a = problem(*size, bias, groups, 30 + sum(size))
    B, Nq, Nk, H = size
    out, lse = msda.msda_query_attention(**a)
    if B * Nq * H <= 1024:
        check_forward(a, out, lse, weight=2.0 ** -16)
    do = torch.randn(B, Nq, H * 32, device="cuda", generator=torch.Generator(device="cuda").manual_seed(4)).bfloat16()
    grads = msda.msda_query_attention_backward(**a, lse=lse, grad_out=do)
    check_backward(a, do, grads, weight=2.0 ** -16)


def test_one_key_takes_all_the_weight():
    """ds is exactly 0 up to the weight's own error: nothing of the output's rounding enters."""
    a = problem(1, 40, 1, 2, True, None, 5)
    _, lse = msda.msda_query_attention(**a)
    do = torch.randn(1, 40, 64, device="cuda").bfloat16()
    check_backward(a, do, msda.msda_query_attention_backward(**a, lse=lse, grad_out=do))


@pytest.mark.parametrize("groups", [None, "shared"])
def test_long_sides(groups):
    """More tiles than the visibility is looked up for at once, on either side."""
    a = problem(1, 600, 140_001, 32, True, groups, 2)
    out, lse = msda.msda_query_attention(**a)
    check_forward(a, out, lse, heads=[0, 31])
    for Nq, Nk in ((70, 140_001), (140_001, 70)):
        a = problem(1, Nq, Nk, 1, True, groups, 4)
        _, lse = msda.msda_query_attention(**a)
        do = torch.randn(1, Nq, 32, device="cuda").bfloat16()
        grads = msda.msda_query_attention_backward(**a, lse=lse, grad_out=do)
        assert all(bool(torch.isfinite(g).all()) for g in grads)
        check_backward(a, do, grads)


def test_documents_are_independent():
    """A packed batch gives every document what it gets alone."""
    sizes = [1, 64, 33, 130, 200]
    n = sum(sizes)
    a = problem(1, n, n, 4, True, None, 12, joint=False)
    a["q_group"] = a["k_group"] = torch.repeat_interleave(
        torch.arange(1, 6, dtype=torch.int32), torch.tensor(sizes))[None].cuda()
    out, lse = msda.msda_query_attention(**a)
    check_forward(a, out, lse)
    at = 0
    for m in sizes:
        one = {k: t[:, at:at + m].contiguous() for k, t in a.items() if "group" not in k}
        o, _ = msda.msda_query_attention(**one)
        diff = (o.double() - out[:, at:at + m].double()).abs()
        # two evaluations of the same sums: each within h of the weights and h of the output
        assert bool((diff <= 4 * HALF * one["v"].abs().double().amax()).all())
        at += m


@pytest.mark.parametrize("step", [1, 10, 1000, 64_000_000])
@pytest.mark.parametrize("bias", [False, True])
def test_what_nobody_sees_reaches_nothing(bias, step):
    """Keys of groups that no query has and queries of groups that no key has hold NaN; the
    groups lie close together, far apart and 64 apart modulo the others."""
    B, Nq, Nk, H = 2, 150, 260, 2
    a = problem(B, Nq, Nk, H, bias, None, 21, joint=False)
    g = torch.Generator(device="cuda").manual_seed(22)
    qg = 1 + step * torch.randint(0, 24, (B, Nq), generator=g, device="cuda", dtype=torch.int32)
    kg = 1 + step * torch.randint(0, 32, (B, Nk), generator=g, device="cuda", dtype=torch.int32)
    qg[qg == 1 + 5 * step] = 1 + 6 * step   # a hole within the queries' groups,
    qg[qg == 1 + 7 * step] = 1
    kg[kg == 1 + 9 * step] = 1              # and one within the keys'
    a.update(q_group=qg, k_group=kg)
    sees = qg[:, :, None] == kg[:, None]
    q_off, k_off = ~sees.any(2), ~sees.any(1)
    assert bool(q_off.any()) and bool(k_off.any())
    a["q"][q_off], a["k"][k_off], a["v"][k_off] = float("nan"), float("nan"), float("inf")
    if bias:
        a["q_points"][q_off], a["k_points"][k_off] = float("nan"), float("inf")
        a["tau"][q_off] = float("nan")
    out, lse = msda.msda_query_attention(**a)
    check_forward(a, out, lse)
    do = torch.randn(B, Nq, H * 32, device="cuda").bfloat16()
    do[q_off] = float("nan")
    grads = msda.msda_query_attention_backward(**a, lse=lse, grad_out=do)
    assert all(t is None or bool(torch.isfinite(t).all()) for t in grads)
    assert bool((grads[0][q_off] == 0).all())
    assert bool((grads[1][k_off] == 0).all()) and bool((grads[2][k_off] == 0).all())
    check_backward(a, do, grads)


@pytest.mark.parametrize("bias,groups", [(False, None), (True, "shared")])
def test_gradient_against_differences(bias, groups):
    a = problem(1, 20, 30, 2, bias, groups, 8)
    _, lse = msda.msda_query_attention(**a)
    do = torch.randn(1, 20, 64, device="cuda").bfloat16()
    grads = msda.msda_query_attention_backward(**a, lse=lse, grad_out=do)
    c = clean(a)
    gen = torch.Generator(device="cuda").manual_seed(1)

    def f(x):
        total = 0.0
        for h in range(2):
            _, _, v, p, *_ = heads64(x, 0, h)
            total += float(((p @ v) * do[0, :, 32 * h:32 * h + 32].double()).sum())
        return total

    step = 1e-5
    for n, g in zip(("q", "k", "v", "tau"), grads):
        if g is None:
            continue
        for _ in range(4):
            u = torch.randn(g.shape, generator=gen, device="cuda").double()
            up, down = dict(c), dict(c)
            up[n], down[n] = c[n] + step * u, c[n] - step * u
            diff = (f(up) - f(down)) / (2 * step)
            # ds and the gradient are each rounded to bf16 once (2 h of the magnitudes; the
            # magnitudes under ds's rounding are at most 4 times the gradient's here), the
            # difference is off by step^2 times a third derivative
            assert abs(diff - float((g.double() * u).sum())) <= 8 * HALF * float((g.double() * u).abs().sum()) + 1e-5


def test_same_bits_streams_and_capture():
    a = problem(2, 333, 333, 8, True, "shared", 6)
    do = torch.randn(2, 333, 256, device="cuda").bfloat16()
    out, lse = msda.msda_query_attention(**a)
    grads = msda.msda_query_attention_backward(**a, lse=lse, grad_out=do)
    first = [t.clone() for t in (out, lse) + grads]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o2, l2 = msda.msda_query_attention(**a, stream=s)
    g2 = msda.msda_query_attention_backward(**a, lse=l2, grad_out=do, stream=s)
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(first, (o2, l2) + g2))
    p = msda.Attention(B=2, Nq=333, Nk=333, H=8)
    ws = torch.empty(msda.lib().msda_query_attention_backward_workspace_size(p), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        msda.msda_query_attention(**a, out=out, lse=lse)
        msda.msda_query_attention_backward(**a, lse=lse, grad_out=do, out=grads, workspace=ws)
    for t in (out, lse) + grads:
        t.zero_()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(first, (out, lse) + grads))


def test_no_keys_no_queries_no_items():
    a = problem(2, 5, 0, 2, False, None, 1, joint=False)
    out, lse = msda.msda_query_attention(**a)
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())
    gq, gk, gv, _ = msda.msda_query_attention_backward(**a, lse=lse, grad_out=out)
    assert bool((gq == 0).all()) and gk.shape == (2, 0, 2, 32)
    a = problem(2, 0, 7, 2, True, None, 1, joint=False)
    out, lse = msda.msda_query_attention(**a)
    gq, gk, gv, gt = msda.msda_query_attention_backward(**a, lse=lse, grad_out=out)
    assert out.shape == (2, 0, 64) and bool((gk == 0).all()) and bool((gv == 0).all())
    a = problem(0, 4, 7, 2, False, None, 1, joint=False)
    out, lse = msda.msda_query_attention(**a)
    assert out.shape == (0, 4, 64)


def test_refusals():
    a = problem(2, 6, 7, 2, True, "shared", 1, joint=False)
    f = msda.msda_query_attention
    half = lambda t: t.half()  # noqa: E731
    for change in (dict(q=half(a["q"])), dict(q=a["q"].float()), dict(k=a["k"][:, :5]),
                   dict(v=a["v"][:1]), dict(q=a["q"].cpu()), dict(tau=None), dict(q_points=None),
                   dict(q_group=None), dict(k_group=a["k_group"].long()),
                   dict(k=a["k"].transpose(1, 2)), dict(v=a["v"][:, :1].expand(2, 7, 2, 32)),
                   dict(tau=a["tau"].double()), dict(scale=math.nan),
                   dict(out=torch.empty(2, 6, 64, device="cuda")), dict(out=a["q"].view(2, 6, 64)),
                   dict(q=torch.zeros(2, 6, 2, 64, device="cuda").bfloat16()),
                   dict(q=torch.zeros(2, 6, 2, 36, device="cuda").bfloat16()[..., :32])):
        with pytest.raises(msda.MsdaError):
            f(**{**a, **change})
