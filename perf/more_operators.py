"""Root-mean-square norm with a residual, matrix products with an epilogue and dropout on rows of channels-last data:
the cases that are timed.

`run` computes an operator's plain form in elementary torch operations, or, where `own` is true, makes the library's
calls.  Six paths:

    rms          h = x + residual and its root-mean-square norm: h, y, rstd
    rms_linear   the norm in 8 bits for each row, then the 8-bit integer product (a 1x1 convolution): h, y
    rms_bwd      gradients of `rms`: dx (of x and residual alike), dgamma
    matmul       act(x w^T + bias) + residual, and the values before the activation where they are kept
    matmul_bwd   its gradients: dx, dw, dbias
    dropout      residual + x with its elements dropped by a counter-based generator, or the gradient of it

A row is a token, or a pixel of a 1x1 convolution.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-5
FLOOR = 2.0 ** -100   # the smallest magnitude that a row's 8-bit scale is made from
LOW = 0xffffffff
PHILOX = (0xD2511F53, 0xCD9E8D57, 0x9E3779B9, 0xBB67AE85)   # the generator's multipliers and key steps


def listed():
    return [
        # the norm before a layer's first product while one token is generated: latency counts
        dict(name="rms one token", op="rms", m=1, c=4096, residual=True, dtype="bf16"),
        # the same over a prompt or a training batch
        dict(name="rms 16384 tokens", op="rms", m=16384, c=4096, residual=True, dtype="bf16"),
        # the bottleneck's 256 channels over 32 images of 56x56, served in 8 bits
        dict(name="rms + 1x1 batch", op="rms_linear", m=100352, c=256, n=256, residual=True, dtype="bf16"),
        # the training step of the second case, with a gradient that reaches h past the norm
        dict(name="rms backward", op="rms_bwd", m=16384, c=4096, dh=True, dtype="bf16"),
        # a small batch in fp32, nothing a multiple of a vector
        dict(name="rms backward odd fp32", op="rms_bwd", m=777, c=1001, dh=False, dtype="f32"),
        # one token through a wide layer: the weights are read once
        dict(name="matmul one token", op="matmul", m=1, k=4096, n=16384, bias=True, residual=False, keep=False,
             act="silu", dtype="bf16"),
        # a few rows in fp32, odd extents
        dict(name="matmul ragged fp32", op="matmul", m=203, k=1001, n=517, bias=True, residual=True, keep=False,
             act="relu", dtype="f32"),
        # a training batch: bound by the matrix units
        dict(name="matmul large", op="matmul", m=8192, k=8192, n=8192, bias=True, residual=True, keep=False,
             act="silu", dtype="bf16"),
        # the gradients of a wide layer over a training batch
        dict(name="matmul backward", op="matmul_bwd", m=8192, k=4096, n=4096, bias=True, act="silu", dtype="bf16"),
        # and of the bottleneck's 256 -> 64 convolution over 32 images of 56x56: few weights, many pixels
        dict(name="matmul backward 1x1", op="matmul_bwd", m=100352, k=256, n=64, bias=True, act="relu", dtype="bf16"),
        # a residual branch's end in a training step
        dict(name="dropout 16384 tokens", op="dropout", m=16384, c=4096, p=0.1, residual=True, dtype="bf16"),
        # the gradient of a small one in fp32, odd extents
        dict(name="dropout odd fp32", op="dropout", m=57, c=333, p=0.5, residual=False, dtype="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rms", "rms_linear", "rms_bwd", "matmul", "matmul_bwd", "dropout"])
    f32 = op != "rms_linear" and rng.random() < 0.3
    size, dtype = (4, "f32") if f32 else (2, "bf16")
    while True:
        m = _log(rng, 1, 131072)
        if op in ("matmul", "matmul_bwd"):
            k, n = _log(rng, 16, 8192), _log(rng, 16, 16384)
            if rng.random() < 0.7:  # most layers' widths are whole 16-byte pieces
                k, n = max(16, k // 8 * 8), max(16, n // 8 * 8)
            # fp32 products run at a tenth of the bf16 rate
            if m * n * k > (8192 ** 3 if op == "matmul" else 8192 * 4096 ** 2) // (16 if f32 else 1):
                continue
            if max(m * k, m * n, k * n) * size > 8192 * 8192 * 2:
                continue
            case = dict(op=op, m=m, k=k, n=n, bias=rng.random() < 0.7, act=rng.choice(["none", "relu", "silu", "gelu"]),
                        dtype=dtype)
            if op == "matmul":
                case.update(residual=rng.random() < 0.5, keep=rng.random() < 0.4)
            return case
        c = _log(rng, 16, 16384)
        if rng.random() < 0.6:
            c = c // 8 * 8
        if op == "rms_linear":
            n = _log(rng, 16, 2048)
            if m * c > 100352 * 256 or m * max(c, n) > 100352 * 1024 or m * c * n > 8192 ** 3 // 16:
                continue
            return dict(op=op, m=m, c=c, n=n, residual=rng.random() < 0.6, dtype=dtype)
        if m * c * size > 16384 * 4096 * 2:
            continue
        if op == "rms_bwd":
            return dict(op=op, m=m, c=c, dh=rng.random() < 0.6, dtype=dtype)
        case = dict(op=op, m=m, c=c, residual=rng.random() < 0.6, dtype=dtype)
        if op == "dropout":
            case.update(p=round(rng.uniform(0.0, 0.9), 3))
        return case


def _type(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def workspace_bytes(case):
    """Room for a call's workspace: dz and copies of the operands in the widest type, with rows of whole pieces, and the
    parts of split sums.  The library's size functions say how much of it a call needs."""
    m = case["m"]
    if "k" in case:
        k, n = case["k"] + 8, case["n"] + 8
        return 4 * (m * n + (m + n) * k) + (64 << 20)
    return {"rms_bwd": 64 << 20, "rms_linear": 128 << 20}.get(case["op"], 0)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    t, m, op = _type(case), case["m"], case["op"]
    empty = lambda *s, dtype=t: torch.empty(*s, dtype=dtype, device="cuda")  # noqa: E731
    s = dict(case=case)
    s["workspace"] = empty(workspace_bytes(case), dtype=torch.uint8)
    if op in ("matmul", "matmul_bwd"):
        k, n = case["k"], case["n"]
        s["x"], s["w"] = rand(m, k).to(t), (rand(n, k) / math.sqrt(k)).to(t)
        if op == "matmul":
            s["bias"] = 0.1 * rand(n) if case["bias"] else None
            s["residual"] = rand(m, n).to(t) if case["residual"] else None
            s["z"] = empty(m, n) if case["keep"] else None
            s["y"] = empty(m, n)
        else:
            s["dy"] = rand(m, n).to(t)
            s["z"] = None if case["act"] == "none" else (rand(m, n) + 0.1).to(t)   # what the forward pass kept
            s["dx"], s["dw"] = empty(m, k), empty(n, k)
            s["dbias"] = empty(n, dtype=torch.float32) if case["bias"] else None
        return s
    c = case["c"]
    # a branch's output, and the stream that it is added to: channels of different spread
    s["x"] = (rand(m, c) * torch.exp(0.5 * rand(c))).to(t)
    s["residual"] = (2 * rand(m, c)).to(t) if case.get("residual") else None
    if op == "dropout":
        s["rng"] = torch.randint(0, 1 << 62, (2,), generator=gen, device="cuda")   # seed and offset
        s["y"] = empty(m, c)
        return s
    s["gamma"] = 1 + 0.2 * rand(c)
    s["rstd"] = empty(m, dtype=torch.float32)
    if op == "rms_bwd":
        s["h"] = s.pop("x")
        s["rstd"] = (s["h"].double().square().mean(1) + EPS).rsqrt().float()
        s["dy"] = rand(m, c).to(t)
        s["dh"] = rand(m, c).to(t) if case["dh"] else None
        s["dx"], s["dgamma"] = empty(m, c), empty(c, dtype=torch.float32)
        return s
    s["h"] = empty(m, c) if case["residual"] else None   # without a residual h is x
    if op == "rms":
        s["y"] = empty(m, c)
        return s
    v = rand(case["n"], c)
    v *= torch.rand(case["n"], 1, generator=gen, device="cuda") + 0.5
    a = v.abs().amax(1)
    s["w"], s["w_scale"] = torch.round(v * (127.0 / a)[:, None]).to(torch.int8), a / (127.0 * math.sqrt(c))
    s["q"], s["q_scale"] = empty(m, c, dtype=torch.int8), empty(m, dtype=torch.float32)
    s["y"] = empty(m, case["n"])
    return s


# ------------------------------------------------------------------ the plain forms


def _plain_act(z, act):
    if act == "relu":
        return z.clamp_min(0)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return z


def _plain_slope(z, act):
    """The activation's derivative."""
    if act == "relu":
        return (z > 0).float()
    if act == "silu":
        e = 1 / (1 + torch.exp(-z))
        return e * (1 + z * (1 - e))
    return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))


def _plain_norm(s):
    """The sum before its rounding, its norm and 1 / rms."""
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    rstd = 1 / torch.sqrt(h.square().mean(1) + EPS)
    return h, h * rstd[:, None] * s["gamma"], rstd


def _plain_rms_bwd(s):
    h, rstd = s["h"].float(), s["rstd"][:, None]
    dy = s["dy"].float()
    xh = h * rstd
    g = dy * s["gamma"]
    dx = (g - xh * (g * xh).mean(1, keepdim=True)) * rstd
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return [dx.to(s["dx"].dtype), (dy * xh).sum(0)]


def _plain_keep(s):
    """Which elements stay: 10 rounds of the generator on the counter (column / 4, row, offset) under the key (seed);
    a 64-bit product that wraps still has the right low 64 bits."""
    case = s["case"]
    m, c = case["m"], case["c"]
    seed, offset = s["rng"][0], s["rng"][1]
    v = [torch.arange(-(-c // 4), device="cuda").expand(m, -1), torch.arange(m, device="cuda")[:, None].expand(-1, -(-c // 4)),
         offset & LOW, offset >> 32]
    key = [seed & LOW, seed >> 32]
    for _ in range(10):
        a, b = v[0] * PHILOX[0], v[2] * PHILOX[1]
        v = [(b >> 32) & LOW ^ v[1] ^ key[0], b & LOW, (a >> 32) & LOW ^ v[3] ^ key[1], a & LOW]
        key = [(key[0] + PHILOX[2]) & LOW, (key[1] + PHILOX[3]) & LOW]
    return (torch.stack(v, 2) >= _threshold(case)).view(m, -1)[:, :c]


def _threshold(case):
    return int(float(np.float32(case["p"])) * 2.0 ** 32)


def _scale(case):
    return 1.0 / (1.0 - float(np.float32(case["p"])))


def _plain(s):
    case = s["case"]
    op, t = case["op"], _type(case)
    if op == "rms":
        h, y, rstd = _plain_norm(s)
        return [None if s["h"] is None else h.to(t), y.to(t), rstd]
    if op == "rms_linear":
        h, v, _ = _plain_norm(s)
        a = v.abs().amax(1).clamp_min(FLOOR)
        q = torch.round(v * (127.0 / a)[:, None])
        y = (q @ s["w"].float().t()) * ((a / 127.0)[:, None] * s["w_scale"])
        return [None if s["h"] is None else h.to(t), y.to(t)]
    if op == "rms_bwd":
        return _plain_rms_bwd(s)
    if op == "matmul":
        z = s["x"].float() @ s["w"].float().t()
        if s["bias"] is not None:
            z = z + s["bias"]
        y = _plain_act(z, case["act"])
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return [y.to(t), None if s["z"] is None else z.to(t)]
    if op == "matmul_bwd":
        dz = s["dy"].float()
        if s["z"] is not None:
            dz = dz * _plain_slope(s["z"].float(), case["act"])
        return [(dz @ s["w"].float()).to(t), (dz.t() @ s["x"].float()).to(t), dz.sum(0) if s["dbias"] is not None else None]
    y = torch.where(_plain_keep(s), s["x"].float() * _scale(case), 0.0)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return [y.to(t)]


# ------------------------------------------------------------------ the library's calls


def _own(s):
    import cnn_convolution_conv2d_amd as c2
    case = s["case"]
    op, m = case["op"], case["m"]
    dt = c2.F32 if case["dtype"] == "f32" else c2.BF16
    if op in ("matmul", "matmul_bwd"):
        k, n, ws = case["k"], case["n"], s["workspace"]
        act = {"none": c2.ACT_NONE, "relu": c2.ACT_RELU, "silu": c2.ACT_SILU, "gelu": c2.ACT_GELU}[case["act"]]
        if op == "matmul":
            c2.conv2d_matmul(s["x"], s["w"], s["bias"], s["residual"], s["z"], s["y"], ws, ws.numel(), m, k, n, k, k, n,
                             n, n, dt, act)
            return [s["y"], s["z"]]
        c2.conv2d_matmul_bwd(s["dy"], s["z"], s["x"], s["w"], s["dx"], s["dw"], s["dbias"], ws, ws.numel(), m, k, n, n,
                             n, k, k, k, k, dt, act)
        return [s["dx"], s["dw"], s["dbias"]]
    c = case["c"]
    if op == "rms":
        c2.conv2d_rms_norm(s["x"], s["residual"], s["gamma"], s["h"], s["y"], s["rstd"], m, c, c, c, c, c, EPS, dt)
        return [s["h"], s["y"], s["rstd"]]
    if op == "rms_linear":
        ws = s["workspace"]
        c2.conv2d_rms_norm_quant(s["x"], s["residual"], s["gamma"], s["h"], s["q"], s["q_scale"], None, m, c, c, c, c, c,
                                 EPS, dt)
        c2.conv2d_int8_matmul(s["q"], s["q_scale"], s["w"], s["w_scale"], None, s["y"], ws, ws.numel(), m, c, case["n"],
                              c, c, case["n"], dt, c2.EPI_NONE)
        return [s["h"], s["y"]]
    if op == "rms_bwd":
        ws = s["workspace"]
        c2.conv2d_rms_norm_bwd(s["dy"], s["dh"], s["h"], s["gamma"], s["rstd"], s["dx"], s["dgamma"], ws, ws.numel(), m,
                               c, c, c, c, c, dt)
        return [s["dx"], s["dgamma"]]
    c2.conv2d_dropout(s["x"], s["residual"], s["y"], s["rng"], case["p"], m, c, c, c, c, dt)
    return [s["y"]]


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ work and exact values


def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    op, m = case["op"], case["m"]
    if op == "matmul":
        k, n = case["k"], case["n"]
        rows = m * n * (1 + case["residual"] + case["keep"])
        return {"bytes": (m * k + n * k + rows) * size + 4 * n * case["bias"], "flops": 2 * m * k * n}
    if op == "matmul_bwd":
        k, n = case["k"], case["n"]
        rows = m * n * (1 + (case["act"] != "none"))
        return {"bytes": (2 * m * k + 2 * n * k + rows) * size + 4 * n * case["bias"], "flops": 4 * m * k * n}
    c = case["c"]
    if op == "rms_linear":
        n = case["n"]
        return {"bytes": m * (c * (1 + 2 * case["residual"]) + n) * size + n * (c + 4) + 4 * c,
                "flops": 2 * m * c * n + 8 * m * c}
    if op == "rms":
        return {"bytes": m * c * (2 + 2 * case["residual"]) * size + 4 * c + 4 * m, "flops": 5 * m * c}
    if op == "rms_bwd":
        return {"bytes": m * c * (3 + case["dh"]) * size + 8 * c + 4 * m, "flops": 11 * m * c}
    return {"bytes": m * c * (2 + case["residual"]) * size, "flops": 3 * m * c}


def _exact_keep(case, rng):
    """The generator once more, on the host in unsigned 64-bit arithmetic."""
    m, c = case["m"], case["c"]
    u = np.uint64
    low, half = u(LOW), u(32)
    seed, offset = (u(int(v)) for v in rng.tolist())
    col, row = np.meshgrid(np.arange(-(-c // 4), dtype=u), np.arange(m, dtype=u))
    c0, c1, c2, c3 = col, row, np.full_like(col, offset & low), np.full_like(col, offset >> half)
    k0, k1 = int(seed & low), int(seed >> half)
    for _ in range(10):
        c0 *= u(PHILOX[0])
        c2 *= u(PHILOX[1])
        c0, c1, c2, c3 = (c2 >> half) ^ c1 ^ u(k0), c2 & low, (c0 >> half) ^ c3 ^ u(k1), c0 & low
        k0, k1 = (k0 + PHILOX[2]) & LOW, (k1 + PHILOX[3]) & LOW
    keep = np.empty((m, c0.shape[1], 4), dtype=bool)
    for i, word in enumerate((c0, c1, c2, c3)):
        np.greater_equal(word, u(_threshold(case)), out=keep[:, :, i])
    return torch.from_numpy(keep.reshape(m, -1)[:, :c]).cuda()


def exact(case, seed):
    """The same values from the definitions, in 64 bits."""
    s = prepare(case, seed)
    op, act, f64 = case["op"], case.get("act"), torch.float64
    up = lambda name: s[name].to(f64)  # noqa: E731
    if op == "dropout":
        y = up("x") * _scale(case) * _exact_keep(case, s["rng"])
        return [y if s["residual"] is None else up("residual") + y]
    if op == "rms_bwd":
        h, dy = up("h"), up("dy")
        r, c = up("rstd").unsqueeze(1), case["c"]
        inner = torch.einsum("mc,mc,c->m", dy, h, up("gamma")).unsqueeze(1)
        dx = r * dy * up("gamma") - h * r ** 3 * inner / c
        return [dx if s["dh"] is None else dx + up("dh"), torch.mv((dy * h).T, up("rstd"))]
    if op in ("rms", "rms_linear"):
        h = up("x") if s["residual"] is None else torch.add(up("x"), up("residual"))
        r = (torch.linalg.vector_norm(h, dim=1) ** 2 / case["c"] + EPS) ** -0.5
        y = torch.einsum("mc,m,c->mc", h, r, up("gamma"))
        h = None if s["residual"] is None else h
        if op == "rms":
            return [h, y, r]
        scale = torch.clamp(torch.linalg.vector_norm(y, float("inf"), dim=1), min=FLOOR) / 127
        return [h, torch.matmul(torch.round(y / scale[:, None]), up("w").T) * torch.outer(scale, up("w_scale"))]
    normal = torch.distributions.Normal(torch.zeros((), dtype=f64, device="cuda"), 1.0, validate_args=False)
    if op == "matmul":
        z = torch.matmul(up("x"), up("w").T)
        z = z if s["bias"] is None else z + up("bias")
        y = {"none": lambda: z, "relu": lambda: torch.relu(z), "silu": lambda: z * torch.sigmoid(z),
             "gelu": lambda: z * normal.cdf(z)}[act]()
        return [y if s["residual"] is None else y + up("residual"), None if s["z"] is None else z]
    dz = up("dy")
    if act != "none":
        z = up("z")
        e = torch.sigmoid(z)
        dz = dz * {"relu": lambda: torch.heaviside(z, torch.zeros_like(z)), "silu": lambda: e + z * e * (1 - e),
                   "gelu": lambda: normal.cdf(z) + z * torch.exp(normal.log_prob(z))}[act]()
    return [torch.matmul(dz, up("w")), torch.matmul(dz.T, up("x")), dz.sum(0) if s["dbias"] is not None else None]
