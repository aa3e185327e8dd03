"""The operators around multi-scale deformable attention in a detection transformer's training and
serving step, as they are measured: the group norm (with its activation) that makes the packed
multi-level value rows, and its gradient; the attention among object queries whose scores fall with
the distance of their reference points, under group masks, and its gradient; the clipping of all
gradients by their global norm.

`run` computes them in plain torch operations, or (own = True) through this package's entry points.
"""
import math

import numpy as np
import torch

own = False

#: [H_l, W_l] of the four levels of the surround-camera and of the detection workloads.
CAMERA_LEVELS = "116x200,58x100,29x50,15x25"
IMAGE_LEVELS = "100x150,50x75,25x38,13x19"

HEAD = 32  # channels per head


def listed():
    return [
        # serving, the smallest map of one image: launch latency is all there is
        {"name": "norm one small level", "op": "norm", "B": 1, "levels": "15x25", "C": 256, "G": 32,
         "x": "f32", "y": "f32", "act": "none", "gap": 0},
        # the input projections of an image pyramid, two images, bf16 through and through
        {"name": "norm image pyramid", "op": "norm", "B": 2, "levels": IMAGE_LEVELS, "C": 256, "G": 32,
         "x": "bf16", "y": "bf16", "act": "silu", "gap": 0},
        # six cameras, fp32 features to the bf16 value that the attention reads
        {"name": "norm six cameras", "op": "norm", "B": 6, "levels": CAMERA_LEVELS, "C": 256, "G": 32,
         "x": "f32", "y": "bf16", "act": "relu", "gap": 0},
        # training on odd maps with a width that is no power of two, rows between the levels unused
        {"name": "norm gradient odd maps", "op": "norm_grad", "B": 3, "levels": "37x53,19x27,7x11", "C": 96,
         "G": 12, "x": "bf16", "y": "bf16", "act": "silu", "gap": 5},
        # training, six cameras in fp32: the gradient that comes from grad_value
        {"name": "norm gradient six cameras", "op": "norm_grad", "B": 6, "levels": CAMERA_LEVELS, "C": 256,
         "G": 32, "x": "f32", "y": "f32", "act": "relu", "gap": 0},
        # serving a stream: each query attends to a long memory of earlier objects
        {"name": "attention one query", "op": "attention", "B": 2, "Nq": 1, "Nk": 4097, "H": 8,
         "points": True, "shared": 0, "size": 0, "pad": 0},
        # serving: the object queries among themselves
        {"name": "attention 900 objects", "op": "attention", "B": 1, "Nq": 900, "Nk": 900, "H": 8,
         "points": True, "shared": 0, "size": 0, "pad": 0},
        # the cells of a 100 x 100 ground grid among themselves
        {"name": "attention 100x100 grid", "op": "attention", "B": 1, "Nq": 10000, "Nk": 10000, "H": 8,
         "points": True, "shared": 0, "size": 0, "pad": 0},
        # training with groups of noised objects beside the matched ones, and a padded tail
        {"name": "attention gradient groups", "op": "attention_grad", "B": 2, "Nq": 1100, "Nk": 1100, "H": 8,
         "points": True, "shared": 900, "size": 19, "pad": 10},
        # training on a long set of proposals
        {"name": "attention gradient 5000", "op": "attention_grad", "B": 1, "Nq": 5000, "Nk": 5000, "H": 8,
         "points": True, "shared": 0, "size": 0, "pad": 0},
        # one attention module's gradients, packed one after the other with odd lengths
        {"name": "clip one module", "op": "clip", "tensors": 23, "total": 300_007, "g": "bf16", "out": "f32",
         "scale": 0.0009765625},
        # all gradients of a detector with its backbone
        {"name": "clip whole model", "op": "clip", "tensors": 300, "total": 69_000_001, "g": "f32", "out": "f32",
         "scale": 1.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "attention", "attention_grad", "clip"])
    if op in ("norm", "norm_grad"):
        C = rng.choice([64, 96, 128, 160, 256, 320, 512])
        h, w = _log(rng, 1, 100), _log(rng, 1, 160)
        sizes = [(-(-h >> i), -(-w >> i)) for i in range(rng.randint(1, 5))]
        least = min(a * b for a, b in sizes)  # a group has 64 values or more: the gradient of a few is all cancellation
        return {"op": op, "B": rng.randint(1, 6), "levels": ",".join("%dx%d" % s for s in sizes), "C": C,
                "G": rng.choice([g for g in range(1, C + 1) if C % g == 0 and least * C // g >= 64] or [1]), "x": rng.choice(["f32", "bf16"]),
                "y": rng.choice(["f32", "bf16"]), "act": rng.choice(["none", "relu", "silu"]),
                "gap": rng.choice([0, 0, 1, 7])}
    if op in ("attention", "attention_grad"):
        B, H = rng.randint(1, 4), rng.choice([1, 2, 3, 4, 8, 12])
        points = rng.random() < 0.75
        if rng.random() < 0.5:
            Nq, Nk = _log(rng, 1, 3000), _log(rng, 16, 3000)
            return {"op": op, "B": B, "Nq": Nq, "Nk": Nk, "H": H, "points": points, "shared": 0, "size": 0, "pad": 0}
        n = _log(rng, 16, 3000)
        pad = rng.randint(0, n // 4)
        return {"op": op, "B": B, "Nq": n, "Nk": n, "H": H, "points": points,
                "shared": rng.choice([0, (n - pad) // 2, n - pad]), "size": rng.randint(8, max(8, n // 5)), "pad": pad}
    n = _log(rng, 1, 400)
    return {"op": "clip", "tensors": n, "total": max(n, _log(rng, 100, 40_000_000)), "g": rng.choice(["f32", "bf16"]),
            "out": rng.choice(["f32", "bf16"]), "scale": rng.choice([1.0, 0.0009765625])}


DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _shapes(case):
    """[(H_l, W_l)], the first row of each level, and the number of rows: `gap` unused rows after each level."""
    shapes = [tuple(int(n) for n in s.split("x")) for s in case["levels"].split(",")]
    rows = [h * w + case["gap"] for h, w in shapes]
    return shapes, [sum(rows[:l]) for l in range(len(rows))], sum(rows)


def _groups(case):
    """int32 [N]: `shared` tokens of group 0 that all see, then groups of `size` that see themselves and those, then padding."""
    n = case["Nq"]
    i = torch.arange(n)
    g = torch.where(i < case["shared"], 0, 1 + (i - case["shared"]) // max(1, case["size"]))
    return torch.where(i < n - case["pad"], g, -1).to(torch.int32)


def _lengths(case):
    """Lengths of the gradient tensors: most of the total in a few, the others short and odd."""
    n, total = case["tensors"], case["total"]
    weight = np.array([1.0 / (1 + (7 * i) % n) for i in range(n)])
    sizes = np.maximum(1, np.floor((total - n) * weight / weight.sum())).astype(np.int64)
    sizes[0] += total - sizes.sum()
    return sizes.tolist()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    rand = lambda *s: torch.rand(*s, generator=gen, device="cuda")  # noqa: E731
    s = {"case": dict(case)}
    if case["op"] in ("norm", "norm_grad"):
        shapes, starts, rows = _shapes(case)
        B, C, L, G = case["B"], case["C"], len(shapes), case["G"]
        s["shapes"], s["starts"] = np.array(shapes, np.int64), np.array(starts, np.int64)
        # features have a mean and a spread of their own in every channel
        s["x"] = (randn(B, rows, C) * (0.5 + rand(C)) + randn(C)).to(DTYPES[case["x"]])
        s["gamma"], s["beta"] = 1 + 0.2 * randn(L, C), 0.2 * randn(L, C)
        if case["op"] == "norm_grad":
            s["grad"] = randn(B, rows, C).to(DTYPES[case["y"]])
            mean, rstd = _stats(s["x"], shapes, starts, G)
            s["mean"], s["rstd"] = mean.float(), rstd.float()
    elif case["op"] in ("attention", "attention_grad"):
        B, Nq, Nk, H = case["B"], case["Nq"], case["Nk"], case["H"]
        # queries and keys come out of one projection, side by side in a row, the values out of another
        s["q"], s["k"] = randn(B, Nq, H, HEAD).bfloat16(), randn(B, Nk, H, HEAD).bfloat16()
        if Nq == Nk:
            both = torch.stack([s["q"], s["k"]], 2)
            s["q"], s["k"] = both[:, :, 0], both[:, :, 1]
        s["v"] = randn(B, Nk, H, HEAD).bfloat16()
        s["points"] = (rand(B, Nq, 2), rand(B, Nk, 2)) if case["points"] else (None, None)
        s["tau"] = 20 * rand(B, Nq, H) if case["points"] else None
        s["group"] = _groups(case).expand(B, Nq).contiguous().cuda() if case["size"] else None
        if case["op"] == "attention_grad":
            s["grad"] = randn(B, Nq, H * HEAD).bfloat16()
            s["lse"] = _scores(s)[1].float()
    else:
        lengths = _lengths(case)
        # gradients of one layer are alike in size, those of different layers are not
        level = torch.repeat_interleave(10 ** (2 * rand(len(lengths)) - 3), torch.tensor(lengths, device="cuda"),
                                        output_size=sum(lengths))
        flat = (randn(sum(lengths)) * level / case["scale"]).to(DTYPES[case["g"]])
        s["out"] = torch.empty(sum(lengths), device="cuda", dtype=DTYPES[case["out"]])
        s["grads"], s["outs"] = list(flat.split(lengths)), list(s["out"].split(lengths))
    return s


EPS = 1e-5
MAX_NORM = 35.0


def _stats(x, shapes, starts, G):
    """Mean and reciprocal spread [B, L, G] of every level, in 64 bits."""
    B, _, C = x.shape
    each = [x[:, st:st + h * w].double().reshape(B, h * w, G, C // G) for (h, w), st in zip(shapes, starts)]
    mean = torch.stack([e.mean((1, 3)) for e in each], 1)
    var = torch.stack([((e - e.mean((1, 3), keepdim=True)) ** 2).mean((1, 3)) for e in each], 1)
    return mean, (var + EPS) ** -0.5


def _norm_level(s, x, l, st, n):
    """Level l's rows, normalised and then scaled and shifted, from the 64-bit statistics rounded once."""
    c = s["case"]
    B, C, G = c["B"], c["C"], c["G"]
    e = x[:, st:st + n].float().reshape(B, n, G, C // G)
    mean, var = e.double().mean((1, 3)), ((e.double() - e.double().mean((1, 3), keepdim=True)) ** 2).mean((1, 3))
    rstd = (var + EPS) ** -0.5
    hat = ((e - mean[:, None, :, None]) * rstd[:, None, :, None]).float().reshape(B, n, C)
    return hat * s["gamma"][l] + s["beta"][l], mean.float(), rstd.float()


def _act(z, act):
    return torch.where(z > 0, z, torch.zeros_like(z)) if act == "relu" else z / (1 + torch.exp(-z)) if act == "silu" else z


def _plain_norm(s):
    c = s["case"]
    shapes, starts, rows = _shapes(c)
    y = torch.zeros(c["B"], rows, c["C"], device="cuda", dtype=DTYPES[c["y"]])
    got = [_norm_level(s, s["x"], l, starts[l], h * w) for l, (h, w) in enumerate(shapes)]
    at = torch.cat([torch.arange(st, st + h * w, device="cuda") for (h, w), st in zip(shapes, starts)])
    y[:, at] = torch.cat([_act(z, c["act"]).to(y.dtype) for z, _, _ in got], 1)
    return y, torch.stack([m for _, m, _ in got], 1), torch.stack([r for _, _, r in got], 1)


def _norm_grad_level(s, l, st, n):
    c = s["case"]
    B, C, G = c["B"], c["C"], c["G"]
    mean, rstd = s["mean"][:, l, None, :, None], s["rstd"][:, l, None, :, None]
    hat = ((s["x"][:, st:st + n].float().reshape(B, n, G, C // G) - mean) * rstd).reshape(B, n, C)
    z = hat * s["gamma"][l] + s["beta"][l]
    dz = s["grad"][:, st:st + n].float()
    if c["act"] == "relu":  # the side of the border in 64 bits: one value on the wrong side is all of a gradient off
        wide = (s["x"][:, st:st + n].double().reshape(B, n, G, C // G) - mean.double()) * rstd.double()
        border = wide.reshape(B, n, C) * s["gamma"][l].double() + s["beta"][l].double()
        dz = torch.where(border > 0, dz, torch.zeros_like(dz))
    if c["act"] == "silu":
        sig = 1 / (1 + torch.exp(-z))
        dz = dz * sig * (1 + z * (1 - sig))
    d_gamma, d_beta = (dz * hat).double().sum((0, 1)), dz.double().sum((0, 1))
    t = (dz * s["gamma"][l]).reshape(B, n, G, C // G)
    hat = hat.reshape(B, n, G, C // G)
    m1 = t.double().mean((1, 3), keepdim=True).float()
    m2 = (t * hat).double().mean((1, 3), keepdim=True).float()
    return ((t - m1 - hat * m2) * rstd).reshape(B, n, C), d_gamma.float(), d_beta.float()


def _plain_norm_grad(s):
    c = s["case"]
    shapes, starts, rows = _shapes(c)
    dx = torch.zeros(c["B"], rows, c["C"], device="cuda", dtype=DTYPES[c["x"]])
    got = [_norm_grad_level(s, l, starts[l], h * w) for l, (h, w) in enumerate(shapes)]
    at = torch.cat([torch.arange(st, st + h * w, device="cuda") for (h, w), st in zip(shapes, starts)])
    dx[:, at] = torch.cat([d.to(dx.dtype) for d, _, _ in got], 1)
    return dx, torch.stack([g for _, g, _ in got]), torch.stack([b for _, _, b in got])


def _scores(s):
    """Scores [B, H, Nq, Nk] in fp32, -inf where the key is not seen; their log-sum-exp [B, H, Nq]; the distances."""
    q, k = s["q"].float().permute(0, 2, 1, 3), s["k"].float().permute(0, 2, 3, 1)
    a = torch.matmul(q, k) * HEAD ** -0.5
    dist = None
    if s["tau"] is not None:
        a_pts, b_pts = s["points"]
        dist = ((a_pts[:, :, None] - b_pts[:, None]) ** 2).sum(-1).sqrt()[:, None]
        a = a - s["tau"].permute(0, 2, 1)[..., None] * dist
    if s["group"] is not None:
        g = s["group"]
        sees = ((g[:, :, None] == g[:, None]) | (g[:, None] == 0)) & (g[:, :, None] >= 0) & (g[:, None] >= 0)
        a = a.masked_fill(~sees[:, None], -math.inf)
    top = a.amax(-1, keepdim=True)
    top = torch.where(top > -math.inf, top, torch.zeros_like(top))
    return a, (torch.exp(a - top).sum(-1).log() + top[..., 0]), dist


def _merge(t, dtype):
    """[B, H, N, 32] -> [B, N, H, 32]"""
    return t.permute(0, 2, 1, 3).contiguous().to(dtype)


def _plain_attention(s):
    a, lse, _ = _scores(s)
    p = torch.exp(a - torch.where(lse > -math.inf, lse, torch.zeros_like(lse))[..., None])
    o = torch.matmul(p, s["v"].float().permute(0, 2, 1, 3))
    return _merge(o, torch.bfloat16).flatten(2), lse


def _plain_attention_grad(s):
    a, _, dist = _scores(s)
    lse = s["lse"]
    p = torch.exp(a - torch.where(lse > -math.inf, lse, torch.zeros_like(lse))[..., None])
    do = s["grad"].float().reshape(s["q"].shape).permute(0, 2, 1, 3)
    v = s["v"].float().permute(0, 2, 3, 1)
    dv = torch.matmul(p.transpose(2, 3), do)
    dp = torch.matmul(do, v)
    ds = p * (dp - (p * dp).sum(-1, keepdim=True))
    dq = torch.matmul(ds, s["k"].float().permute(0, 2, 1, 3)) * HEAD ** -0.5
    dk = torch.matmul(ds.transpose(2, 3), s["q"].float().permute(0, 2, 1, 3)) * HEAD ** -0.5
    dt = None if dist is None else -(ds * dist).sum(-1).permute(0, 2, 1).contiguous()
    return _merge(dq, torch.bfloat16), _merge(dk, torch.bfloat16), _merge(dv, torch.bfloat16), dt


def _plain_clip(s):
    c = s["case"]
    flat = torch.cat([g.float() for g in s["grads"]])
    norm = (flat.double() ** 2).sum().sqrt() * c["scale"]
    factor = torch.clamp(MAX_NORM / (norm + 1e-6), max=1.0) * c["scale"]
    s["out"].copy_(flat * factor.float())
    return s["out"], norm.float().reshape(1)


def run(state):
    s = state
    c = s["case"]
    if own:
        import scale_deformable_attention_03_b200 as msda

        if c["op"] == "norm":
            return msda.msda_group_norm(s["x"], s["shapes"], s["starts"], c["G"], s["gamma"], s["beta"], eps=EPS,
                                        activation=c["act"], out_dtype=DTYPES[c["y"]])
        if c["op"] == "norm_grad":
            return msda.msda_group_norm_backward(s["x"], s["shapes"], s["starts"], c["G"], s["mean"], s["rstd"],
                                                 s["grad"], s["gamma"], s["beta"], activation=c["act"],
                                                 out_dtype=DTYPES[c["x"]])
        if c["op"] == "attention":
            return msda.msda_query_attention(s["q"], s["k"], s["v"], q_points=s["points"][0], k_points=s["points"][1],
                                             tau=s["tau"], q_group=s["group"], k_group=s["group"])
        if c["op"] == "attention_grad":
            return msda.msda_query_attention_backward(s["q"], s["k"], s["v"], s["lse"], s["grad"],
                                                      q_points=s["points"][0], k_points=s["points"][1], tau=s["tau"],
                                                      q_group=s["group"], k_group=s["group"])
        norm = msda.msda_clip_grad_norm(s["grads"], MAX_NORM, grad_scale=c["scale"], out=s["outs"])
        return s["out"], norm
    return {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "attention": _plain_attention,
            "attention_grad": _plain_attention_grad, "clip": _plain_clip}[c["op"]](s)


def _pairs(case):
    """Pairs of a query and a key that it sees, in one head of one item."""
    if not case["size"]:
        return case["Nq"] * case["Nk"]
    n = case["Nq"] - case["pad"]
    shared = min(n, case["shared"])
    rest = n - shared
    whole, last = divmod(rest, case["size"])
    return n * shared + whole * case["size"] ** 2 + last ** 2


def work(case):
    size = {"f32": 4, "bf16": 2}
    if case["op"] in ("norm", "norm_grad"):
        shapes, _, rows = _shapes(case)
        used = case["B"] * sum(h * w for h, w in shapes) * case["C"]
        full = case["B"] * rows * case["C"]
        small = len(shapes) * (2 * case["B"] * case["G"] + 2 * case["C"]) * 4
        if case["op"] == "norm":
            return {"bytes": used * size[case["x"]] + full * size[case["y"]] + small, "flops": 8 * used}
        return {"bytes": used * (size[case["x"]] + size[case["y"]]) + full * size[case["x"]] + small
                + 2 * len(shapes) * case["C"] * 4, "flops": 20 * used}
    if case["op"] in ("attention", "attention_grad"):
        B, Nq, Nk, H = case["B"], case["Nq"], case["Nk"], case["H"]
        rows = 2 * B * H * HEAD
        small = B * (8 * (Nq + Nk) + 4 * Nq * H) * case["points"] + B * (4 * Nq + 4 * Nk) * (case["size"] > 0) + 4 * B * H * Nq
        pairs = B * H * _pairs(case)
        if case["op"] == "attention":
            return {"bytes": rows * (2 * Nq + 2 * Nk) + small, "flops": 4 * HEAD * pairs}
        return {"bytes": rows * (3 * Nq + 4 * Nk) + small + 4 * B * H * Nq * case["points"], "flops": 10 * HEAD * pairs}
    return {"bytes": case["total"] * (size[case["g"]] + size[case["out"]]), "flops": 4 * case["total"]}


def _exact_norm(s):
    """The norm level by level in 64 bits, each group's values in one row."""
    c = s["case"]
    shapes, starts, rows = _shapes(c)
    B, C, G = c["B"], c["C"], c["G"]
    out, means, rstds = torch.zeros(B, rows, C, device="cuda", dtype=torch.float64), [], []
    for l, (h, w) in enumerate(shapes):
        e = s["x"][:, starts[l]:starts[l] + h * w].double().transpose(1, 2).reshape(B, G, -1)
        m = e.sum(-1, keepdim=True) / e.shape[-1]
        r = 1 / torch.sqrt((e - m).pow(2).sum(-1, keepdim=True) / e.shape[-1] + EPS)
        z = ((e - m) * r).reshape(B, C, h * w).transpose(1, 2) * s["gamma"][l].double() + s["beta"][l].double()
        z = z.clamp(min=0) if c["act"] == "relu" else z * torch.sigmoid(z) if c["act"] == "silu" else z
        out[:, starts[l]:starts[l] + h * w] = z
        means.append(m[..., 0])
        rstds.append(r[..., 0])
    return out, torch.stack(means, 1), torch.stack(rstds, 1)


def _exact_norm_grad(s):
    """The gradient in 64 bits from the given statistics: autograd through the scale, the shift and the activation,
    then each group's gradient with its projections on the constant and on the normalised values taken off."""
    c = s["case"]
    shapes, starts, rows = _shapes(c)
    B, C, G = c["B"], c["C"], c["G"]
    dx = torch.zeros(B, rows, C, device="cuda", dtype=torch.float64)
    d_gamma, d_beta = torch.zeros(2, len(shapes), C, device="cuda", dtype=torch.float64)
    for l, (h, w) in enumerate(shapes):
        at = slice(starts[l], starts[l] + h * w)
        e = s["x"][:, at].double().transpose(1, 2).reshape(B, G, -1)
        r = s["rstd"][:, l, :, None].double()
        hat = ((e - s["mean"][:, l, :, None].double()) * r).requires_grad_()
        gamma, beta = s["gamma"][l].double().requires_grad_(), s["beta"][l].double().requires_grad_()
        z = hat.reshape(B, C, h * w) * gamma[:, None] + beta[:, None]
        y = torch.relu(z) if c["act"] == "relu" else z * torch.sigmoid(z) if c["act"] == "silu" else z
        t, d_gamma[l], d_beta[l] = torch.autograd.grad(y, (hat, gamma, beta), s["grad"][:, at].double().transpose(1, 2))
        hat = hat.detach()
        t = r * (t - t.sum(-1, keepdim=True) / t.shape[-1] - hat * (t * hat).sum(-1, keepdim=True) / t.shape[-1])
        dx[:, at] = t.reshape(B, C, h * w).transpose(1, 2)
    return dx, d_gamma, d_beta


def _exact_attention(s):
    """One head of one item at a time, in 64 bits; the gradients by autograd."""
    c = s["case"]
    B, Nq, Nk, H = c["B"], c["Nq"], c["Nk"], c["H"]
    grad = c["op"] == "attention_grad"
    out = torch.zeros(B, Nq, H * HEAD, device="cuda", dtype=torch.float64)
    lse = torch.zeros(B, H, Nq, device="cuda", dtype=torch.float64)
    full = {n: torch.zeros(s[n].shape, device="cuda", dtype=torch.float64) for n in ("q", "k", "v")}
    full["tau"] = torch.zeros(B, Nq, H, device="cuda", dtype=torch.float64)
    for b in range(B):
        dist = None
        if s["tau"] is not None:
            d = [s["points"][0][b, :, None, i].double() - s["points"][1][b, None, :, i].double() for i in (0, 1)]
            dist = torch.hypot(d[0], d[1])
        sees = torch.ones(Nq, Nk, device="cuda", dtype=torch.bool)
        if s["group"] is not None:
            g = s["group"][b]
            sees = torch.logical_and(g[:, None] >= 0, torch.logical_or(g[None] == 0, g[None] == g[:, None]))
        some = sees.any(1)
        for h in range(H):
            q, k, v = (s[n][b, :, h].double().requires_grad_(grad) for n in ("q", "k", "v"))
            tau = s["tau"][b, :, h].double().requires_grad_(grad) if dist is not None else None
            a = (q / math.sqrt(HEAD)) @ k.T
            if dist is not None:
                a = a - tau[:, None] * dist
            a = torch.where(sees, a, torch.full_like(a, -1e300))
            lse[b, h] = torch.where(some, torch.logsumexp(a.detach(), 1), torch.full((Nq,), -math.inf, device="cuda", dtype=torch.float64))
            o = torch.where(some[:, None], torch.softmax(a, 1) @ v, torch.zeros(1, device="cuda", dtype=torch.float64))
            out[b, :, h * HEAD:(h + 1) * HEAD] = o.detach()
            if grad:
                wrt = (q, k, v) + ((tau,) if tau is not None else ())
                got = torch.autograd.grad(o, wrt, s["grad"][b, :, h * HEAD:(h + 1) * HEAD].double())
                for n, t in zip(("q", "k", "v", "tau"), got):
                    full[n][b, :, h] = t
            del a, o
    if grad:
        return full["q"], full["k"], full["v"], full["tau"] if s["tau"] is not None else None
    return out, lse


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(s)
    if case["op"] == "norm_grad":
        return _exact_norm_grad(s)
    if case["op"] in ("attention", "attention_grad"):
        return _exact_attention(s)
    squares = torch.stack([g.double().pow(2).sum() for g in s["grads"]])
    norm = squares.sum().sqrt() * case["scale"]
    factor = min(1.0, MAX_NORM / (float(norm) + 1e-6)) * case["scale"]
    return torch.cat([g.double() for g in s["grads"]]) * factor, norm.reshape(1)
