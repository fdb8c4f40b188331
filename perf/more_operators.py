"""The experts' matrix products and the AdamW update on 8-bit states, as they are timed.

Two groups, which a training or serving program of a mixture-of-experts model
calls around the optimizer:
  adamw8   the optimizer's step for AdamW parameters whose two moments are
           kept in 8 bits, over all the tensors of a shape table
  experts  matrix products grouped by expert over ragged groups of rows:
           forward, input gradient, weight gradient (the gradient of a Muon
           parameter of experts * out rows)
`run` computes them in elementary torch operations where `own` is false and
calls the package where it is true.
"""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HP = {"lr": 3e-4, "beta1": 0.9, "beta2": 0.95, "eps": 1e-8, "wd": 0.1, "t": 10}
BLOCK = 256


# --------------------------------------------------------------------- cases

def listed():
    return [
        # the norms and biases of a GPT-2-small model: many tiny tensors
        {"name": "adamw8_vectors", "op": "adamw8", "shapes": "74*1x768", "dtype": "bf16"},
        # every AdamW parameter of that model
        {"name": "adamw8_gpt2", "op": "adamw8", "shapes": "50257x768 74*1x768", "dtype": "bf16"},
        # 32-bit weights of odd and ragged sizes, blocks that end inside a tensor
        {"name": "adamw8_odd", "op": "adamw8", "shapes": "1x1 3x5 1x255 1x257 1001x33 777x1023 2049x511 5x4099", "dtype": "f32"},
        # the embedding of a 4096-wide model
        {"name": "adamw8_embedding", "op": "adamw8", "shapes": "128256x4096", "dtype": "bf16"},
        # one token decoded, 6 experts of 64: the experts' up projection
        {"name": "experts_token", "op": "experts_fwd", "rows": 6, "experts": 64, "out": 1408, "in": 2048, "skew": 0.0, "dtype": "bf16"},
        # 64 sequences decoded at once: a few rows for every expert
        {"name": "experts_decode", "op": "experts_fwd", "rows": 384, "experts": 64, "out": 1408, "in": 2048, "skew": 0.5, "dtype": "bf16"},
        # a training batch of 8192 tokens through the same layer, and its gradients
        {"name": "experts_fwd_64", "op": "experts_fwd", "rows": 49152, "experts": 64, "out": 1408, "in": 2048, "skew": 0.5, "dtype": "bf16"},
        {"name": "experts_igrad_64", "op": "experts_igrad", "rows": 49152, "experts": 64, "out": 1408, "in": 2048, "skew": 0.5, "dtype": "bf16"},
        {"name": "experts_wgrad_64", "op": "experts_wgrad", "rows": 49152, "experts": 64, "out": 1408, "in": 2048, "skew": 0.5, "dtype": "bf16"},
        # odd widths: rows that start at any 2-byte address, experts without rows
        {"name": "experts_igrad_odd", "op": "experts_igrad", "rows": 1531, "experts": 13, "out": 701, "in": 301, "skew": 2.0, "dtype": "bf16"},
        # 32-bit weight gradient, every size odd
        {"name": "experts_wgrad_odd", "op": "experts_wgrad", "rows": 3001, "experts": 7, "out": 513, "in": 767, "skew": 1.0, "dtype": "f32"},
        # 8192 tokens, 2 experts of 8, of a 4096 -> 14336 projection
        {"name": "experts_fwd_8", "op": "experts_fwd", "rows": 16384, "experts": 8, "out": 14336, "in": 4096, "skew": 0.5, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    """Log-uniform over [lo, hi]; half of the draws are multiples of 64 where that fits."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if n >= 64 and rng.random() < 0.5:
        n -= n % 64
    return max(lo, min(hi, n))


def draw(rng):
    dtype = "bf16" if rng.random() < 0.7 else "f32"
    op = rng.choice(["adamw8", "adamw8", "experts_fwd", "experts_fwd", "experts_igrad", "experts_wgrad"])
    if op == "adamw8":
        kinds, left, shapes = rng.randint(1, 6), 1 << 28, []
        for _ in range(kinds):
            cols = _log(rng, 1, 16384)
            rows = 1 if rng.random() < 0.4 else _log(rng, 1, max(1, left // kinds // cols))
            count = _log(rng, 1, max(1, min(48, left // kinds // (rows * cols))))
            shapes.append("%d*%dx%d" % (count, rows, cols) if count > 1 else "%dx%d" % (rows, cols))
        return {"op": op, "shapes": " ".join(shapes), "dtype": dtype}
    experts, out, inn = _log(rng, 1, 160), _log(rng, 16, 14336), _log(rng, 16, 14336)
    while experts * out * inn > 64 * 4096 * 4096:  # the weights of all experts within what the listed ones hold
        experts = (experts + 1) // 2
    most = 16384 * 14336 * 4096 // (1 if dtype == "bf16" else 4)
    rows = _log(rng, 1, max(1, min(49152, most // (out * inn))))
    # the plain form gives every expert as many rows as the fullest one has: no more of them than fit
    skew = rng.uniform(0.0, 2.0 if experts * rows * max(out, inn) < 1 << 31 else 0.7)
    return {"op": op, "rows": rows, "experts": experts, "out": out, "in": inn, "skew": round(skew, 2), "dtype": dtype}


def _sizes(case):
    """(rows, cols) of every tensor of "74*1x768 5x7"."""
    parts = [p.replace("*", "x").split("x") for p in case["shapes"].split()]
    return [(int(p[-2]), int(p[-1])) for p in parts for _ in range(int(p[0]) if len(p) == 3 else 1)]


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "adamw8":
        n = sum(r * c for r, c in _sizes(case))
        blocks = sum(-(-r * c // BLOCK) for r, c in _sizes(case))
        # w read and written, g read; the codes of m and v and their offsets read and written
        return {"bytes": n * (3 * es + 4) + blocks * 8, "flops": 40 * n}
    t, e, n, k = case["rows"], case["experts"], case["out"], case["in"]
    used = e if case["op"] == "experts_wgrad" else min(e, t)  # a weight gradient is written for every expert
    return {"bytes": (t * n + t * k + used * n * k) * es + 4 * (e + 1), "flops": 2 * t * n * k}


# -------------------------------------------------------------------- inputs

def _counts(case, seed):
    """Rows per expert: every row picks one by the same skewed chances."""
    g = torch.Generator().manual_seed(seed)
    chance = torch.softmax(case["skew"] * torch.randn(case["experts"], generator=g), 0)
    pick = torch.multinomial(chance, case["rows"], replacement=True, generator=g)
    return torch.bincount(pick, minlength=case["experts"])


def _mix(x):
    """32-bit integer hash of the integers of x (int64, 0 .. 2^32 - 1)."""
    x = x ^ (x >> 16)
    x = x * 0x6A09E667 & 0xFFFFFFFF
    x = x ^ (x >> 15)
    x = x * 0xBB67AE85 & 0xFFFFFFFF
    return x ^ (x >> 16)


def _key(t):
    return _mix((t & 0xFFFFFFFF) ^ _mix(t >> 32))


def _padded(t):
    return torch.nn.functional.pad(t.reshape(-1), (0, -t.numel() % BLOCK))


def _blocks(tensors):
    """All tensors' elements in rows of 256, each tensor from a row of its own."""
    return torch.cat([_padded(t) for t in tensors]).view(-1, BLOCK)


def _hash(numels, device, t):
    """Hash of every group of 4 elements, in rows of 64."""
    block = torch.cat([torch.arange(-(-n // BLOCK), device=device) for n in numels])
    group = block[:, None] * (BLOCK // 4) + torch.arange(BLOCK // 4, device=device)
    return _mix((group & 0xFFFFFFFF) ^ (((group >> 32) * 0x9E3779B1 & 0xFFFFFFFF) ^ _key(t)))


def _random(numels, device, t):
    """16 random bits for the first and for the second moment of every element: the
    halves of its group's hash, turned right by 8 bits per place in the group."""
    h = _hash(numels, device, t)[:, :, None]
    turn = torch.arange(0, 32, 8, device=device)
    h = ((h >> turn) | (h << (32 - turn))) & 0xFFFFFFFF
    h = h.view(-1, BLOCK)
    return (h & 0xFFFF).int(), (h >> 16).int()


def _encode(x, rand, top, signed):
    """Codes (rows of 256) and offsets of fp32 values, see the library's header."""
    a = x.abs()
    u = torch.where(a.isnan(), 0x7FC00000, a.view(torch.int32))
    off = (((u.amax(dim=1, keepdim=True) + 0xFFFFF) >> 20) - top).clamp(min=0)
    k = ((u + (rand << 4)) >> 20) - off
    lo = ((off + 1) << 20).view(torch.float32)
    low = (a > lo * ((rand.float() + 0.5) * 2.0 ** -16)) if signed else (a > 0)
    k = torch.where(u < ((off + 1) << 20), low.int(), k)
    if signed:
        k = k | (x.view(torch.int32) >> 24 & 0x80)
    return k.to(torch.uint8), off[:, 0].to(torch.int16)


def _decode(code, off, signed):
    k = code.int()
    mag = k & 127 if signed else k
    x = torch.where(mag > 0, (mag + off.int()[:, None]) << 20, 0).view(torch.float32)
    return torch.where(k > 127, -x, x) if signed else x


def _state(code, off, numels):
    """Kept moments, tensor by tensor: its codes in whole blocks, then the blocks' 16-bit offsets up to a multiple of 16 bytes."""
    nb = [-(-n // BLOCK) for n in numels]
    offs = [torch.nn.functional.pad(o.view(torch.uint8), (0, -2 * o.numel() % 16)) for o in off.split(nb)]
    return torch.cat([t for c, o in zip(code.split(nb), offs) for t in (c.reshape(-1), o)])


def _state_views(flat, numels):
    nb = [-(-n // BLOCK) for n in numels]
    return list(flat.split([b * BLOCK + (2 * b + 15) // 16 * 16 for b in nb]))


def _parts(states, numels):
    """(codes in rows of 256, offsets) of all buffers."""
    ends = [-(-n // BLOCK) * BLOCK for n in numels]
    code = torch.cat([s[:e] for s, e in zip(states, ends)]).view(-1, BLOCK)
    return code, torch.cat([s[e:e + e // BLOCK * 2].view(torch.int16) for s, e in zip(states, ends)])


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DT[case["dtype"]]
    st = {"case": dict(case)}
    rand = lambda *shape: torch.randn(*shape, generator=g, device="cuda")
    if case["op"] == "adamw8":
        sizes = _sizes(case)
        numels = [r * c for r, c in sizes]
        # gradients whose size differs from row to row; rows without any, as of an embedding's unseen tokens
        seen = [(torch.rand(r, 1, generator=g, device="cuda") < 0.8) if r > 1 else torch.ones(1, 1, device="cuda") for r, _ in sizes]
        size = [1e-3 * torch.exp(rand(r, 1)) for r, _ in sizes]
        # one buffer for all the weights and one for each moment, as programs keep them
        st["flat_w"] = torch.cat([torch.nn.functional.pad((rand(r, c) * 0.02).to(dt).view(-1), (0, -r * c % 64)) for r, c in sizes])
        st["w"] = [p[:r * c].view(r, c) for (r, c), p in zip(sizes, st["flat_w"].split([-(-n // 64) * 64 for n in numels]))]
        st["g"] = [(rand(r, c) * z * s).to(dt) for (r, c), z, s in zip(sizes, size, seen)]
        rm, rv = _random(numels, "cuda", HP["t"] - 1)
        code, off = _encode(_blocks([rand(r, c) * z * 0.3 for (r, c), z in zip(sizes, size)]), rm, 127, True)
        st["flat_m"] = _state(code, off, numels)
        st["m"] = _state_views(st["flat_m"], numels)
        code, off = _encode(_blocks([(rand(r, c) * z).square() * 0.5 for (r, c), z in zip(sizes, size)]), rv, 255, False)
        st["flat_v"] = _state(code, off, numels)
        st["v"] = _state_views(st["flat_v"], numels)
        if own:
            import matrix_orthogonalizing_optimizer_amd as mo
            code = mo.MUON_BF16 if dt == torch.bfloat16 else mo.MUON_F32
            st["plan"] = mo.muon_plan_create([(mo.MUON_KIND_ADAMW8, code, r, c, 0, 0) for r, c in sizes])
            st["hp"] = mo.make_hparams(adam_lr=HP["lr"], adam_beta1=HP["beta1"], adam_beta2=HP["beta2"], adam_eps=HP["eps"],
                                       adam_weight_decay=HP["wd"], adam_step=HP["t"])
            st["ws"] = torch.empty(mo.muon_plan_workspace_bytes(st["plan"]), dtype=torch.uint8, device="cuda")
        return st
    t, e, n, k = case["rows"], case["experts"], case["out"], case["in"]
    counts = _counts(case, seed)
    st["most"] = int(counts.max())  # the capacity a router plans with
    st["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)]).int().cuda()
    if case["op"] != "experts_igrad":
        st["x"] = rand(t, k).to(dt)
    if case["op"] != "experts_fwd":
        st["dy"] = (rand(t, n) * 1e-3).to(dt)
    if case["op"] != "experts_wgrad":
        st["w"] = torch.empty(e, n, k, dtype=dt, device="cuda")
        for i in range(e):
            st["w"][i] = rand(n, k) * 0.02
    shape = {"experts_fwd": (t, n), "experts_igrad": (t, k), "experts_wgrad": (e, n, k)}[case["op"]]
    st["o"] = torch.empty(*shape, dtype=dt, device="cuda")
    return st


# ----------------------------------------------------------------- plain form

def _scalars():
    f = np.float32
    return {"c1": float(f(1) - f(HP["beta1"])), "c2": float(f(1) - f(HP["beta2"])), "eps": float(f(HP["eps"])),
            "keep": float(f(1) - f(HP["lr"]) * f(HP["wd"])),
            "step": float(f(HP["lr"])) * math.sqrt(1 - float(f(HP["beta2"])) ** HP["t"]) / (1 - float(f(HP["beta1"])) ** HP["t"])}


def _plain_adamw8(st):
    s = _scalars()
    numels = [t.numel() for t in st["w"]]
    rm, rv = _random(numels, st["w"][0].device, HP["t"])
    g = _blocks(st["g"]).float()
    m = _decode(*_parts(st["m"], numels), True)
    m = m + (g - m) * s["c1"]
    code, off = _encode(m, rm, 127, True)
    st["flat_m"].copy_(_state(code, off, numels))
    v = _decode(*_parts(st["v"], numels), False)
    v = v + (g * g - v) * s["c2"]
    code, off = _encode(v, rv, 255, False)
    st["flat_v"].copy_(_state(code, off, numels))
    w = _blocks(st["w"]).float() * s["keep"] - s["step"] * (m / (s["eps"] + v.sqrt()))
    parts = w.view(-1).split([-(-n // BLOCK) * BLOCK for n in numels])
    torch._foreach_copy_(st["w"], [p[:n].view(t.shape).to(t.dtype) for p, n, t in zip(parts, numels, st["w"])])
    return {"w": st["flat_w"], "m": st["flat_m"], "v": st["flat_v"]}


def _plain_experts(st):
    """Every expert's rows in a block of the same height, zeros below them, for one batched product."""
    case, off, most = st["case"], st["offsets"].long(), st["most"]
    e = case["experts"]
    row = torch.arange(case["rows"], device=off.device)
    owner = torch.searchsorted(off[1:], row, right=True)
    place = owner * most + row - off[owner]

    def spread(t):
        out = torch.zeros(e * most, t.shape[1], device=t.device)
        out[place] = t.float()
        return out.view(e, most, -1)

    if case["op"] == "experts_wgrad":
        return torch.bmm(spread(st["dy"]).transpose(1, 2), spread(st["x"])).to(st["o"].dtype)
    w = st["w"].float()
    o = torch.bmm(spread(st["x"]), w.transpose(1, 2)) if case["op"] == "experts_fwd" else torch.bmm(spread(st["dy"]), w)
    return o.view(e * most, -1)[place].to(st["o"].dtype)


def run(st):
    op = st["case"]["op"]
    if own:
        import matrix_orthogonalizing_optimizer_amd as mo
        if op == "adamw8":
            mo.muon_step(st["plan"], st["w"], st["g"], [None] * len(st["w"]), st["m"], st["v"], st["hp"], st["ws"])
            return {"w": st["flat_w"], "m": st["flat_m"], "v": st["flat_v"]}
        if op == "experts_fwd":
            return mo.muon_experts_forward(st["x"], st["w"], st["offsets"], y=st["o"])
        if op == "experts_igrad":
            return mo.muon_experts_input_grad(st["dy"], st["w"], st["offsets"], dx=st["o"])
        return mo.muon_experts_weight_grad(st["dy"], st["x"], st["offsets"], dw=st["o"])
    return _plain_adamw8(st) if op == "adamw8" else _plain_experts(st)


# --------------------------------------------------------------- in 64 bits

def _exact_moment(state, n, signed):
    """The kept values, in 64 bits: code k of a block with offset o is 2^E (1 + F / 8), 8 (E + 127) + F = k + o."""
    end = -(-n // BLOCK) * BLOCK
    code = state[:end].view(-1, BLOCK).long()
    off = state[end:end + end // BLOCK * 2].view(torch.int16).long()[:, None]
    mag = code % 128 if signed else code
    at = mag + off
    size = torch.ldexp(torch.where(at >= 8, 1.0 + (at % 8).double() / 8, (at % 8).double() / 4), (at // 8 - 127))
    size = torch.where(mag > 0, size, torch.zeros_like(size))
    return (torch.where(code >= 128, -size, size) if signed else size).view(-1)[:n]


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "adamw8":
        s, out = _scalars(), []
        for w, g, m, v in zip(st["w"], st["g"], st["m"], st["v"]):
            n, g = w.numel(), g.double().view(-1)
            m, v = _exact_moment(m, n, True), _exact_moment(v, n, False)
            m, v = (1 - s["c1"]) * m + s["c1"] * g, (1 - s["c2"]) * v + s["c2"] * g ** 2
            w = s["keep"] * w.double().view(-1) - s["step"] * m / (v.sqrt() + s["eps"])
            out.append(torch.nn.functional.pad(w, (0, -n % 64)))
        return {"w": torch.cat(out), "m": None, "v": None}
    off = st["offsets"].tolist()
    o = torch.zeros(st["o"].shape, dtype=torch.float64, device="cuda")
    for e, (a, b) in enumerate(zip(off, off[1:])):
        if case["op"] == "experts_wgrad":
            o[e] = st["dy"][a:b].double().t() @ st["x"][a:b].double()
        elif case["op"] == "experts_fwd":
            o[a:b] = st["x"][a:b].double() @ st["w"][e].double().t()
        else:
            o[a:b] = st["dy"][a:b].double() @ st["w"][e].double()
    return o
