"""The operators that make and keep what muon_step reads, as they are timed.

Three groups, which a training or serving program calls around the optimizer:
  norm    layer norm / RMS norm forward and backward (the gradients of the
          AdamW vectors of a shape table)
  keep    activations kept as 8-bit rows (int8 and one power-of-two scale per
          token), restored, and used in the weight gradient of a linear layer
          (the gradient of a Muon matrix)
  linear  the linear layer on 8-bit rows: quantized activations times
          quantized weights, and the gradient of its input
`run` computes them in elementary torch operations where `own` is false and
calls the package where it is true.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5


# --------------------------------------------------------------------- cases

def listed():
    return [
        # one decoding step of four sequences: the norm of a 4096-wide stream
        {"name": "norm_tokens", "op": "norm_fwd", "kind": "rms", "rows": 4, "cols": 4096, "dtype": "bf16", "pad": 0},
        # a GPT-2-small training batch (8 sequences of 1024), layer norm
        {"name": "norm_fwd_768", "op": "norm_fwd", "kind": "layer", "rows": 8192, "cols": 768, "dtype": "bf16", "pad": 0},
        {"name": "norm_bwd_768", "op": "norm_bwd", "kind": "layer", "rows": 8192, "cols": 768, "dtype": "bf16", "pad": 0},
        # ragged rows of odd width in 32 bits, cut out of a wider tensor
        {"name": "norm_bwd_odd", "op": "norm_bwd", "kind": "layer", "rows": 2049, "cols": 1001, "dtype": "f32", "pad": 6},
        # a long batch of a 4096-wide model with RMS norms
        {"name": "norm_bwd_4096", "op": "norm_bwd", "kind": "rms", "rows": 16384, "cols": 4096, "dtype": "bf16", "pad": 0},
        # activations of that batch kept in 8 bits and restored for a backward pass
        {"name": "keep_4096", "op": "keep", "rows": 16384, "cols": 4096, "dtype": "bf16", "pad": 0},
        # weight gradient of the fused 768-wide QKV projection
        {"name": "wgrad_qkv", "op": "wgrad", "tokens": 8192, "out": 2304, "in": 768, "dtype": "bf16", "pad": 0},
        # weight gradient in 32 bits, every size odd or ragged
        {"name": "wgrad_odd", "op": "wgrad", "tokens": 1531, "out": 701, "in": 301, "dtype": "f32", "pad": 3},
        # weight gradient of a 4096 -> 14336 projection
        {"name": "wgrad_14336", "op": "wgrad", "tokens": 8192, "out": 14336, "in": 4096, "dtype": "bf16", "pad": 0},
        # one token through norm and projection: the serving step
        {"name": "linear_token", "op": "linear", "norm": True, "tokens": 1, "out": 14336, "in": 4096, "dtype": "bf16", "pad": 0},
        # a prompt, or a training batch, through the same projection
        {"name": "linear_prompt", "op": "linear", "norm": False, "tokens": 8192, "out": 14336, "in": 4096, "dtype": "bf16", "pad": 0},
        # gradient of the input of that projection
        {"name": "igrad_14336", "op": "igrad", "tokens": 8192, "out": 14336, "in": 4096, "dtype": "bf16", "pad": 0},
    ]


def _size(rng, lo, hi):
    """Log-uniform over [lo, hi]; half of the draws are multiples of 64 where that fits."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if n >= 64 and rng.random() < 0.5:
        n -= n % 64
    return max(lo, min(hi, n))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "keep", "wgrad", "linear", "linear", "igrad"])
    dtype = "bf16" if rng.random() < 0.7 else "f32"
    pad = 0 if rng.random() < 0.6 else rng.randint(1, 40)
    if op in ("norm_fwd", "norm_bwd", "keep"):
        cols = _size(rng, 16, 14336)
        rows = _size(rng, 1, max(1, min(32768, 16384 * 4096 // (cols * (1 if dtype == "bf16" else 2)))))
        c = {"op": op, "rows": rows, "cols": cols, "dtype": dtype, "pad": pad}
        if op != "keep":
            c["kind"] = rng.choice(["layer", "rms"])
        return c
    most = 8192 * 14336 * 4096 // (1 if dtype == "bf16" else 3)
    out, inn = _size(rng, 64, 14336), _size(rng, 64, 14336)
    tokens = _size(rng, 1, max(1, min(16384, most // (out * inn))))
    c = {"op": op, "tokens": tokens, "out": out, "in": inn, "dtype": dtype, "pad": pad}
    if op == "linear":
        # a norm's last bits decide which way a value between two of the 8-bit
        # rows' steps goes: that shows in 32-bit outputs, not in 16-bit ones
        c["norm"] = dtype == "bf16" and rng.random() < 0.5
    return c


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op in ("norm_fwd", "norm_bwd", "keep"):
        r, c = case["rows"], case["cols"]
        vec = 2 if case.get("kind") == "layer" else 1
        if op == "norm_fwd":  # x, y, gamma (beta), the two statistics (one)
            return {"bytes": 2 * r * c * es + vec * c * es + vec * r * 4, "flops": 8 * r * c}
        if op == "norm_bwd":  # dy, x, dx, gamma, the vector gradients, the statistics
            return {"bytes": 3 * r * c * es + (1 + vec) * c * es + vec * r * 4, "flops": 14 * r * c}
        # x and the restored copy, the 8-bit rows and scales written and read
        return {"bytes": 2 * r * c * es + 2 * (r * c + 4 * r), "flops": 4 * r * c}
    t, n, k = case["tokens"], case["out"], case["in"]
    if op == "wgrad":
        b = t * n * es + t * k + 4 * t + n * k * es
    elif op == "igrad":
        b = t * n * es + n * k + 4 * n + t * k * es
    else:
        b = t * k * es + n * k + 4 * n + n * es + t * n * es + (2 * k * es if case["norm"] else 0)
    return {"bytes": b, "flops": 2 * t * n * k}


# -------------------------------------------------------------------- inputs

def _rows_of(g, rows, cols, pad, dtype, scale=1.0, outliers=False):
    """rows x cols values in a tensor whose rows are cols + pad apart."""
    x = torch.randn(rows, cols + pad, generator=g, device="cuda") * scale
    if outliers:  # a few channels far larger than the rest, as in trained networks
        ch = torch.randint(0, cols + pad, (max(1, cols // 256),), generator=g, device="cuda")
        x[:, ch] *= 8.0
    return x.to(dtype)[:, :cols]


def _quantize(x):
    """8-bit rows of a float matrix: q = round(x / s), s the smallest power of
    two with max|x| <= 127 s (at least 2^-126); rows with a non-finite value
    get q = 0, s = NaN."""
    x = x.float()
    amax = x.abs().amax(dim=1) if x.shape[1] else x.new_zeros(x.shape[0])
    fine = torch.isfinite(amax)
    m, e = torch.frexp(torch.where(fine, amax, torch.zeros_like(amax)))
    e = torch.where(m > 127.0 / 128.0, e - 6, e - 7)
    e = torch.where(amax > 0, e, torch.full_like(e, -126)).clamp(min=-126)
    s = torch.ldexp(torch.ones_like(amax), e)
    q = torch.round(torch.ldexp(x, -e[:, None]))
    q = torch.where(fine[:, None], q, torch.zeros_like(q))
    return q.to(torch.int8), torch.where(fine, s, torch.full_like(s, math.nan))


def _kept(x):
    """The 8-bit rows of x in the storage a program keeps them in: rows a
    multiple of 16 bytes apart, zeros behind the last column."""
    q, s = _quantize(x)
    rows, cols = q.shape
    store = torch.zeros(rows, (cols + 15) // 16 * 16, dtype=torch.int8, device=q.device)
    store[:, :cols] = q
    return store[:, :cols], s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt, pad, op = DT[case["dtype"]], case["pad"], case["op"]
    st = {"case": dict(case)}
    new = lambda *shape, dtype=dt: torch.empty(*shape, dtype=dtype, device="cuda")
    if op in ("norm_fwd", "norm_bwd", "keep"):
        r, c = case["rows"], case["cols"]
        st["x"] = _rows_of(g, r, c, pad, dt, 1.5, outliers=True)
        if op == "keep":
            st["q"] = new(r, (c + 15) // 16 * 16, dtype=torch.int8)[:, :c]
            st["scale"], st["out"] = new(r, dtype=torch.float32), new(r, c)
            return st
    else:
        t, n, k = case["tokens"], case["out"], case["in"]
        c = k
        if op == "wgrad":
            st["q"], st["scale"] = _kept(_rows_of(g, t, k, 0, torch.float32, 1.0, outliers=True))
            st["dy"] = _rows_of(g, t, n, pad, dt, 1e-3)
            st["dw"] = new(n, k)
            return st
        st["wq"], st["wscale"] = _kept(_rows_of(g, n, k, 0, torch.float32, 0.02))
        if op == "igrad":
            st["dy"] = _rows_of(g, t, n, pad, dt, 1e-3)
            st["dx"] = new(t, k)
            return st
        st["x"] = _rows_of(g, t, k, pad, dt, 1.0, outliers=True)
        st["bias"] = (torch.randn(n, generator=g, device="cuda") * 0.02).to(dt)
        st["q"] = new(t, (k + 15) // 16 * 16, dtype=torch.int8)[:, :k]
        st["scale"], st["y"] = new(t, dtype=torch.float32), new(t, n)
        if not case["norm"]:
            return st
    st["gamma"] = (1.0 + 0.1 * torch.randn(c, generator=g, device="cuda")).to(dt)
    layer = case.get("kind") == "layer"
    st["beta"] = (0.1 * torch.randn(c, generator=g, device="cuda")).to(dt) if layer else None
    if op == "norm_bwd":
        st["dy"] = _rows_of(g, case["rows"], c, pad, dt, 1e-3)
        xd = st["x"].double()
        mean = xd.mean(dim=1) if layer else torch.zeros_like(xd[:, 0])
        st["rstd"] = ((xd - mean[:, None]).square().mean(dim=1) + EPS).rsqrt().float()
        st["mean"] = mean.float() if layer else None
        st["dx"], st["dgamma"] = new(case["rows"], c), new(c)
        st["dbeta"] = new(c) if layer else None
    elif op == "norm_fwd":
        st["y"], st["rstd"] = new(case["rows"], c), new(case["rows"], dtype=torch.float32)
        st["mean"] = new(case["rows"], dtype=torch.float32) if layer else None
    return st


# ----------------------------------------------------------------- plain form

def _plain_norm(x, gamma, beta, layer):
    mean = x.mean(dim=1) if layer else None
    d = x - mean[:, None] if layer else x
    rstd = 1.0 / torch.sqrt((d * d).mean(dim=1) + EPS)
    y = d * rstd[:, None] * gamma.to(x.dtype)
    if beta is not None:
        y = y + beta.to(x.dtype)
    return y, mean, rstd


def _plain(st):
    case = st["case"]
    op, dt = case["op"], DT[case["dtype"]]
    layer = case.get("kind") == "layer"
    if op == "norm_fwd":
        y, mean, rstd = _plain_norm(st["x"].float(), st["gamma"], st["beta"], layer)
        return [y.to(dt), mean, rstd] if layer else [y.to(dt), rstd]
    if op == "norm_bwd":
        x, dy = st["x"].float(), st["dy"].float()
        xh = ((x - st["mean"][:, None]) if layer else x) * st["rstd"][:, None]
        gr = dy * st["gamma"].float()
        dx = gr - xh * (gr * xh).mean(dim=1, keepdim=True)
        if layer:
            dx = dx - gr.mean(dim=1, keepdim=True)
        dx = dx * st["rstd"][:, None]
        dg = (dy * xh).sum(dim=0)
        return [dx.to(dt), dg.to(dt)] + ([dy.sum(dim=0).to(dt)] if layer else [])
    if op == "keep":
        q, s = _quantize(st["x"])
        return (q.float() * s[:, None]).to(dt)
    if op == "wgrad":
        x = st["q"].float() * st["scale"][:, None]
        return (st["dy"].float().t() @ x).to(dt)
    w = st["wq"].float() * st["wscale"][:, None]
    if op == "igrad":
        return (st["dy"].float() @ w).to(dt)
    # the norm in 64 bits: its values are rounded to 8 bits next
    x = _plain_norm(st["x"].double(), st["gamma"], None, False)[0] if case["norm"] else st["x"]
    q, s = _quantize(x)
    y = (q.float() * s[:, None]) @ w.t() + st["bias"].float()
    return y.to(dt)


# ------------------------------------------------------------------- own form

def _own(st):
    import matrix_orthogonalizing_optimizer_amd as mo
    case = st["case"]
    op = case["op"]
    kind = mo.MUON_NORM_LAYER if case.get("kind") == "layer" else mo.MUON_NORM_RMS
    if op == "norm_fwd":
        mo.muon_norm_forward(st["x"], st["gamma"], st["beta"], eps=EPS, kind=kind, y=st["y"],
                             mean=st["mean"], rstd=st["rstd"])
        return [st["y"], st["mean"], st["rstd"]] if st["mean"] is not None else [st["y"], st["rstd"]]
    if op == "norm_bwd":
        mo.muon_norm_backward(st["dy"], st["x"], st["gamma"], st["mean"], st["rstd"], kind=kind, dx=st["dx"],
                              dgamma=st["dgamma"], dbeta=st["dbeta"])
        return [st["dx"], st["dgamma"]] + ([st["dbeta"]] if st["dbeta"] is not None else [])
    if op == "keep":
        mo.muon_rows8_quantize(st["x"], q=st["q"], scale=st["scale"])
        return mo.muon_rows8_dequantize(st["q"], st["scale"], out=st["out"])
    if op == "wgrad":
        return mo.muon_linear8_weight_grad(st["dy"], st["q"], st["scale"], dw=st["dw"])
    if op == "igrad":
        return mo.muon_linear8_input_grad(st["dy"], st["wq"], st["wscale"], dx=st["dx"])
    if case["norm"]:
        mo.muon_norm_forward(st["x"], st["gamma"], eps=EPS, kind=mo.MUON_NORM_RMS, q=st["q"], scale=st["scale"])
    else:
        mo.muon_rows8_quantize(st["x"], q=st["q"], scale=st["scale"])
    return mo.muon_linear8_forward(st["q"], st["scale"], st["wq"], st["wscale"], bias=st["bias"], y=st["y"])


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------- 64-bit definition

def _restore64(x):
    """The 64-bit values that the 8-bit rows of x stand for, by the definition:
    the power of two is searched from the largest magnitude of the row."""
    x = x.double()
    a = x.abs().max(dim=1).values
    p = torch.floor(torch.log2(torch.clamp(a, min=2.0 ** -140))) - 7
    for _ in range(3):  # at most two steps up from a quotient of at most 256
        p = torch.where(torch.pow(2.0, p) * 127.0 < a, p + 1, p)
    step = torch.pow(2.0, torch.clamp(p, min=-126.0))
    return torch.round(x / step[:, None]) * step[:, None]


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "keep":
        return _restore64(st["x"])
    if op == "wgrad":
        x = st["q"].double() * st["scale"].double().unsqueeze(1)
        return torch.matmul(st["dy"].double().t().contiguous(), x)
    if op == "igrad":
        w = st["wq"].double() * st["wscale"].double().unsqueeze(1)
        return torch.matmul(st["dy"].double(), w)
    x = st["x"].double()
    if op == "norm_fwd":
        layer = case["kind"] == "layer"
        mu = x.sum(1) / x.shape[1] if layer else torch.zeros_like(x[:, 0])
        var = ((x - mu.unsqueeze(1)) ** 2).sum(1) / x.shape[1]
        r = (var + EPS) ** -0.5
        y = (x - mu.unsqueeze(1)) * r.unsqueeze(1) * st["gamma"].double()
        return [y + st["beta"].double(), mu, r] if layer else [y, r]
    if op == "norm_bwd":
        layer = case["kind"] == "layer"
        n, r = x.shape[1], st["rstd"].double().unsqueeze(1)
        h = (x - st["mean"].double().unsqueeze(1)) * r if layer else x * r
        dy = st["dy"].double()
        g = dy * st["gamma"].double()
        s2 = (g * h).sum(1, keepdim=True) / n
        s1 = g.sum(1, keepdim=True) / n if layer else torch.zeros_like(s2)
        res = [r * (g - s1 - h * s2), (dy * h).sum(0)]
        return res + [dy.sum(0)] if layer else res
    if case["norm"]:
        x = x * ((x * x).sum(1, keepdim=True) / x.shape[1] + EPS) ** -0.5 * st["gamma"].double()
    w = st["wq"].double() * st["wscale"].double().unsqueeze(1)
    return torch.matmul(_restore64(x), w.t().contiguous()) + st["bias"].double()
