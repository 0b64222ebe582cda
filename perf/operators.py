"""Group norm on channels-last activations and 8-bit integer products: the cases that are timed.

`run` computes an operator's plain form in elementary torch operations, or, where `own` is true, makes the library's
calls.  Five paths:

    norm         group norm with an activation, forward: y, mean, rstd
    norm_bwd     its backward pass: dx, dgamma, dbeta
    product      int8 rows times int8 channels, with a scale for each, bias and ReLU
    linear       rows quantised to int8, then the product
    norm_linear  group norm with an activation, quantised for each pixel, then the product (a 1x1 convolution)

A token of `product` and `linear` is a row; of `norm_linear` a pixel.
"""
import math

import torch

own = False

EPS = 1e-5
WORKSPACE = 64 << 20  # bytes that a program keeps for the library's calls
FLOOR = 2.0 ** -100   # the smallest magnitude that a row's scale is made from


def _norm(name, op, n, h, w, c, g, act, dtype, **more):
    return dict(name=name, op=op, n=n, h=h, w=w, c=c, g=g, act=act, dtype=dtype, **more)


def listed():
    return [
        # one image between two convolutions of a small feature map: latency counts
        _norm("norm one image", "norm", 1, 28, 28, 256, 32, "silu", "bf16"),
        # the input of the 3x3 workload layer, normalised and rectified
        _norm("norm 112x112", "norm", 32, 112, 112, 128, 32, "relu", "bf16"),
        # odd extents, fp32, wide groups, no activation
        _norm("norm odd fp32", "norm", 3, 57, 43, 144, 9, "none", "f32"),
        # a training step on the bottleneck's 256-channel activations
        _norm("backward 56x56", "norm_bwd", 64, 56, 56, 256, 32, "silu", "bf16"),
        # a small batch in fp32, odd extents
        _norm("backward odd fp32", "norm_bwd", 2, 29, 31, 128, 16, "silu", "f32"),
        # one token through a wide layer: the weights are read once
        dict(name="product one token", op="product", m=1, k=4096, n=16384, bias=True, relu=False, dtype="bf16"),
        # a few tokens, nothing a multiple of a tile
        dict(name="product ragged", op="product", m=37, k=1040, n=1001, bias=True, relu=True, dtype="f32"),
        # a large batch of tokens: bound by the matrix units
        dict(name="product large", op="product", m=8192, k=8192, n=8192, bias=False, relu=False, dtype="bf16"),
        # the bottleneck's 256 -> 64 convolution over 64 images of 56x56
        dict(name="linear 1x1 pixels", op="linear", m=200704, k=256, n=64, bias=True, relu=True, dtype="bf16"),
        # four tokens through a small layer: latency of two calls
        dict(name="linear few tokens", op="linear", m=4, k=2048, n=2048, bias=True, relu=False, dtype="bf16"),
        # a pre-activation block's projection over a batch
        _norm("norm + 1x1 batch", "norm_linear", 32, 56, 56, 256, 32, "silu", "bf16", k_out=256),
        # and over one image
        _norm("norm + 1x1 image", "norm_linear", 1, 28, 28, 128, 32, "silu", "bf16", k_out=256),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "product", "linear", "norm_linear"])
    while True:
        if op in ("product", "linear"):
            m, n = _log(rng, 1, 65536), _log(rng, 16, 16384)
            k = _log(rng, 64, 8192)
            if rng.random() < 0.8:  # most layers' widths are whole 16-byte chunks
                k = max(64, k // 16 * 16)
            if m * n * k > 8192 ** 3 or m * (2 * k + n) > 8 << 25:
                continue
            return dict(op=op, m=m, k=k, n=n, bias=rng.random() < 0.7, relu=rng.random() < 0.4,
                        dtype="f32" if op == "product" and rng.random() < 0.3 else "bf16")
        g = rng.choice([1, 2, 4, 8, 9, 16, 32])
        c = g * _log(rng, 1, 64)
        n, h, w = _log(rng, 1, 64), _log(rng, 7, 112), _log(rng, 7, 112)
        if op == "norm_linear":
            c = -(-c // (16 * g)) * 16 * g
        if not 16 <= c <= 1024 or n * h * w * c > 64 * 56 * 56 * 256:
            continue
        if op == "norm_linear":
            return _pure(_norm("", op, n, h, w, c, g, rng.choice(["relu", "silu"]), "bf16", k_out=_log(rng, 16, 1024)))
        # the derivative of relu jumps at 0, where two correct roundings may disagree: silu and none are drawn
        act = rng.choice(["none", "silu"] if op == "norm_bwd" else ["none", "relu", "silu"])
        return _pure(_norm("", op, n, h, w, c, g, act, "f32" if rng.random() < 0.3 else "bf16"))


def _pure(case):
    del case["name"]
    return case


def _type(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def _int8_rows(gen, rows, k):
    """Rows as a quantised layer holds them: int8 values and the scale of each row."""
    v = torch.randn(rows, k, generator=gen, device="cuda")
    v *= torch.rand(rows, 1, generator=gen, device="cuda") + 0.5
    a = v.abs().amax(1)
    return torch.round(v * (127.0 / a)[:, None]).to(torch.int8), a / 127.0


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    s = dict(case=case, workspace=torch.empty(WORKSPACE, dtype=torch.uint8, device="cuda"))
    t = _type(case)
    if "c" in case:
        n, h, w, c, g = (case[k] for k in ("n", "h", "w", "c", "g"))
        # a convolution's output: every channel has its own offset and spread
        x = rand(n, h, w, c)
        x *= torch.exp(0.3 * rand(c))
        x += rand(c)
        s["x"] = x.to(t)
        s["gamma"] = 1 + 0.2 * rand(c)
        s["beta"] = 0.2 * rand(c)
        s["mean"] = torch.empty(n, g, device="cuda")
        s["rstd"] = torch.empty(n, g, device="cuda")
        if case["op"] == "norm":
            s["y"] = torch.empty_like(s["x"])
        if case["op"] == "norm_bwd":
            s["dy"] = rand(n, h, w, c).to(t)
            v = s["x"].view(n, h * w, g, c // g)  # what the forward pass saved
            for i in range(n):
                u = v[i].double()
                mu = u.mean((0, 2))
                s["mean"][i] = mu
                s["rstd"][i] = ((u - mu[:, None]).square().mean((0, 2)) + EPS).rsqrt()
            s["dx"] = torch.empty_like(s["x"])
            s["dgamma"] = torch.empty(c, device="cuda")
            s["dbeta"] = torch.empty(c, device="cuda")
        m, k, out = n * h * w, c, case.get("k_out")
    else:
        m, k, out = case["m"], case["k"], case["n"]
        if case["op"] == "product":
            s["q"], s["q_scale"] = _int8_rows(gen, m, k)
        else:
            s["x"] = (rand(m, k) * (torch.rand(m, 1, generator=gen, device="cuda") + 0.5)).to(t)
    if out:
        s["w"], s["w_scale"] = _int8_rows(gen, out, k)
        s["w_scale"] /= math.sqrt(k)
        s["bias"] = 0.1 * rand(out) if case.get("bias", True) else None
        s["y"] = torch.empty(m, out, dtype=t, device="cuda")
        if case["op"] != "product":
            s["q"] = torch.empty(m, k, dtype=torch.int8, device="cuda")
            s["q_scale"] = torch.empty(m, device="cuda")
    return s


# ------------------------------------------------------------------ the plain forms


def _plain_norm(s):
    case = s["case"]
    n, p, c, g = case["n"], case["h"] * case["w"], case["c"], case["g"]
    x = s["x"].float().view(n, p, g, c // g)
    mean = x.mean((1, 3))
    d = x - mean[:, None, :, None]
    rstd = 1 / torch.sqrt(d.square().mean((1, 3)) + EPS)
    z = (d * rstd[:, None, :, None]).view(n, p, c) * s["gamma"] + s["beta"]
    if case["act"] == "relu":
        z = z.clamp_min(0)
    elif case["act"] == "silu":
        z = z / (1 + torch.exp(-z))
    return z, mean, rstd


def _plain_norm_bwd(s):
    case = s["case"]
    n, p, c, g = case["n"], case["h"] * case["w"], case["c"], case["g"]
    rstd = s["rstd"][:, None, :, None]
    xh = ((s["x"].float().view(n, p, g, c // g) - s["mean"][:, None, :, None]) * rstd).view(n, p, c)
    dz = s["dy"].float().view(n, p, c)
    if case["act"] == "silu":
        z = xh * s["gamma"] + s["beta"]
        e = 1 / (1 + torch.exp(-z))
        dz = dz * (e * (1 + z * (1 - e)))
    dbeta = dz.sum((0, 1))
    dgamma = (dz * xh).sum((0, 1))
    t = (dz * s["gamma"]).view(n, p, g, c // g)
    xh = xh.view(n, p, g, c // g)
    m = p * (c // g)
    s1 = t.sum((1, 3), keepdim=True) / m
    s2 = (t * xh).sum((1, 3), keepdim=True) / m
    dx = (t - s1 - xh * s2) * rstd
    return dx.view(s["x"].shape).to(s["x"].dtype), dgamma, dbeta


def _plain_quantize(v):
    a = v.abs().amax(1).clamp_min(FLOOR)
    return torch.round(v * (127.0 / a)[:, None]), a / 127.0


def _plain_product(s, q, q_scale):
    y = (q @ s["w"].float().t()) * (q_scale[:, None] * s["w_scale"])
    if s["bias"] is not None:
        y = y + s["bias"]
    if s["case"].get("relu"):
        y = y.clamp_min(0)
    return y.to(s["y"].dtype)


def _plain(s):
    op = s["case"]["op"]
    if op == "norm":
        y, mean, rstd = _plain_norm(s)
        return [y.view(s["x"].shape).to(s["x"].dtype), mean, rstd]
    if op == "norm_bwd":
        return list(_plain_norm_bwd(s))
    if op == "product":
        return [_plain_product(s, s["q"].float(), s["q_scale"])]
    v = s["x"].float() if op == "linear" else _plain_norm(s)[0].reshape(-1, s["case"]["c"])
    return [_plain_product(s, *_plain_quantize(v))]


# ------------------------------------------------------------------ the library's calls


def _own(s):
    import cnn_convolution_conv2d_amd as c2
    case = s["case"]
    op, ws = case["op"], s["workspace"]
    dt = c2.F32 if case["dtype"] == "f32" else c2.BF16
    if "c" in case:
        n, h, w, c, g = case["n"], case["h"], case["w"], case["c"], case["g"]
        act = {"none": c2.ACT_NONE, "relu": c2.ACT_RELU, "silu": c2.ACT_SILU}[case["act"]]
        if op == "norm":
            c2.conv2d_group_norm_nhwc(s["x"], s["gamma"], s["beta"], s["y"], s["mean"], s["rstd"], ws, WORKSPACE,
                                      n, c, h, w, g, c, c, EPS, dt, act)
            return [s["y"], s["mean"], s["rstd"]]
        if op == "norm_bwd":
            c2.conv2d_group_norm_bwd_nhwc(s["dy"], s["x"], s["gamma"], s["beta"], s["mean"], s["rstd"], s["dx"],
                                          s["dgamma"], s["dbeta"], ws, WORKSPACE, n, c, h, w, g, c, c, c, dt, act)
            return [s["dx"], s["dgamma"], s["dbeta"]]
        c2.conv2d_group_norm_quant_nhwc(s["x"], s["gamma"], s["beta"], s["q"], s["q_scale"], None, None, ws, WORKSPACE,
                                        n, c, h, w, g, c, c, EPS, dt, act)
    elif op == "linear":
        c2.conv2d_quantize_rows(s["x"], s["q"], s["q_scale"], case["m"], case["k"], case["k"], case["k"], dt)
    m, k = s["q"].shape
    out = s["w"].shape[0]
    epi = (c2.EPI_BIAS if s["bias"] is not None else 0) | (c2.EPI_RELU if case.get("relu") else 0)
    c2.conv2d_int8_matmul(s["q"], s["q_scale"], s["w"], s["w_scale"], s["bias"], s["y"], ws, WORKSPACE,
                          m, k, out, k, k, out, dt, epi)
    return [s["y"]]


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ work and exact values


def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    if "c" in case:
        n, c, g = case["n"], case["c"], case["g"]
        p = n * case["h"] * case["w"]
        if case["op"] == "norm":
            return {"bytes": 2 * p * c * size + 8 * c + 8 * n * g, "flops": 9 * p * c}
        if case["op"] == "norm_bwd":
            return {"bytes": 3 * p * c * size + 16 * c + 8 * n * g, "flops": 24 * p * c}
        out = case["k_out"]
        return {"bytes": p * (c * size + out * size) + out * (c + 8) + 8 * c, "flops": 2 * p * c * out + 12 * p * c}
    m, k, n = case["m"], case["k"], case["n"]
    x = m * k + 4 * m if case["op"] == "product" else m * k * size
    return {"bytes": x + n * (k + 4) + (4 * n if case["bias"] else 0) + m * n * size, "flops": 2 * m * k * n}


def exact(case, seed):
    """The same values from the definitions, in 64 bits, image by image (row block by row block)."""
    s = prepare(case, seed)
    op = case["op"]
    f64 = torch.float64
    act = case.get("act")

    def normalised(i):
        u = s["x"][i].to(f64).reshape(-1, case["g"], case["c"] // case["g"])
        mu = u.sum((0, 2)) / u[:, 0].numel()
        var = (u - mu[:, None]).pow(2).sum((0, 2)) / u[:, 0].numel()
        r = (var + EPS) ** -0.5
        return ((u - mu[:, None]) * r[:, None]).reshape(-1, case["c"]), mu, r

    def activated(z):
        return z * torch.sigmoid(z) if act == "silu" else torch.relu(z) if act == "relu" else z

    def affine(xh):
        return xh * s["gamma"].to(f64) + s["beta"].to(f64)

    def product(q, scale):
        y = torch.matmul(q, s["w"].to(f64).T) * scale[:, None] * s["w_scale"].to(f64)
        y = y if s["bias"] is None else y + s["bias"].to(f64)
        return torch.relu(y) if case.get("relu") else y

    def quantised(v):
        scale = torch.clamp(torch.linalg.vector_norm(v, float("inf"), dim=1), min=FLOOR) / 127
        return torch.round(v / scale[:, None]), scale

    if op == "norm":
        got = [normalised(i) for i in range(case["n"])]
        y = torch.stack([activated(affine(xh)) for xh, _, _ in got]).view(s["x"].shape)
        return [y, torch.stack([mu for _, mu, _ in got]), torch.stack([r for _, _, r in got])]
    if op == "norm_bwd":
        dxs, dgamma, dbeta = [], 0, 0
        gamma, cg = s["gamma"].to(f64), case["c"] // case["g"]
        for i in range(case["n"]):
            mu, r = (s[k][i].to(f64).repeat_interleave(cg) for k in ("mean", "rstd"))
            xh = (s["x"][i].to(f64).reshape(-1, case["c"]) - mu) * r
            dz = s["dy"][i].to(f64).reshape(-1, case["c"])
            if act == "silu":
                z = affine(xh)
                e = torch.sigmoid(z)
                dz = dz * e * (1 + z - z * e)
            dbeta = dbeta + dz.sum(0)
            dgamma = dgamma + (dz * xh).sum(0)
            per = lambda v: v.sum(0).view(-1, cg).mean(1).repeat_interleave(cg) / len(dz)  # noqa: E731
            dxs.append(r * (gamma * dz - per(gamma * dz) - xh * per(gamma * dz * xh)))
        return [torch.stack(dxs).view(s["x"].shape), dgamma, dbeta]
    if op == "product":
        return [product(s["q"].to(f64), s["q_scale"].to(f64))]
    if op == "linear":
        return [product(*quantised(s["x"].to(f64)))]
    rows = [product(*quantised(activated(affine(normalised(i)[0])))) for i in range(case["n"])]
    return [torch.cat(rows)]
