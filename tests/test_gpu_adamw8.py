"""GPU tests of AdamW on 8-bit moments against the numpy reference: the codes
have to be equal, bit for bit; the weights within their roundings.

Tolerance of a weight: keep = 1 - lr wd takes two fp32 roundings and its product
with w one, the difference one more, together 4 u |w|, u = 2^-24; the update takes
a square root and a reciprocal of 1 ulp = 2 u each and one rounding each in the
sum with eps, the product with m, the factor lr sqrt(1-b2^t)/(1-b1^t), the product
with it and the difference, together 9 u |update|, of which w - w0 also holds
lr wd w (9 u of that is in the slack of 4 u |w|, as its own error is u |w|):
4 u |w| + 10 u |update|, and half a step of the storage type."""
import numpy as np
import pytest
import torch

from oracle import adamw8_ref as R
from tests.gpu_util import dev, f64

mo = pytest.importorskip("matrix_orthogonalizing_optimizer_amd")

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32
HP = dict(lr=3e-4, beta1=0.9, beta2=0.95, eps=1e-8, wd=0.1)


def hparams(t, **kw):
    h = dict(HP, **kw)
    return mo.make_hparams(adam_lr=h["lr"], adam_beta1=h["beta1"], adam_beta2=h["beta2"], adam_eps=h["eps"],
                           adam_weight_decay=h["wd"], adam_step=t)


def code(dtype):
    return mo.MUON_F32 if dtype == F32 else mo.MUON_BF16


class Param:
    """One parameter on the host and on the device; `shift` elements into its storage."""

    def __init__(self, shape, dtype, seed, shift=0, fill=77, zero=False):
        rng = np.random.default_rng(seed)
        n = shape[0] * shape[1]
        self.shape, self.dtype, self.n = shape, dtype, n
        self.w = self.put(rng.standard_normal(n) * 0.02, shift)
        size = np.exp(rng.uniform(-12, 0, n))
        self.states = []
        for moment in (0, 1):
            x = rng.standard_normal(n) * 1e-3 * size
            x = (np.square(x) if moment else x * 0.3).astype(np.float32) * (0 if zero else 1)
            c, o = R.encode(x, seed, moment)
            # the buffers lie at 4-byte alignment in a wider one
            s = R.to_state(c, o, fill)
            base = torch.zeros(s.size + 4, dtype=torch.uint8)
            base[4:] = torch.from_numpy(s)
            self.states.append(base.to(dev())[4:])

    def put(self, x, shift):
        base = torch.zeros(self.n + shift + 3, dtype=self.dtype)
        base[shift:shift + self.n] = torch.from_numpy(np.asarray(x, dtype=np.float64)).to(self.dtype)
        return base.to(dev())[shift:shift + self.n].view(self.shape)

    def grad(self, seed, shift=0, scale=1e-3):
        rng = np.random.default_rng(seed)
        return self.put(rng.standard_normal(self.n) * scale * np.exp(rng.uniform(-12, 0, self.n)), shift)


def expect(p, g, t, hp):
    """(weights in fp64, their bound, the two buffers) of a step."""
    with np.errstate(all="ignore"):
        old = [R.decode(*R.from_state(s.cpu().numpy(), p.n), k) for k, s in enumerate(p.states)]
        gv = g.float().cpu().numpy().reshape(-1)
        m, v = R.moments(gv, old[0], old[1], hp["beta1"], hp["beta2"])
        w0 = f64(p.w).reshape(-1)
        w = R.weights(w0, m, v, t=t, **{k: hp[k] for k in ("lr", "beta1", "beta2", "eps", "wd")})
        bufs = []
        for k, x in enumerate((m, v)):
            s = p.states[k].cpu().numpy().copy()
            c, o = R.encode(x, t, k)
            nb = o.size
            s[:p.n] = c
            s[nb * 256:nb * 256 + 2 * nb] = o.view(np.uint8)
            bufs.append(s)
        bound = 4 * U * np.abs(w0) + 10 * U * np.abs(w - w0) + torch.finfo(p.dtype).eps / 2 * np.abs(w) * (p.dtype == BF)
        bound += (U * np.abs(w)) * (p.dtype == F32)
    return w, bound, bufs


def compare(p, want, what):
    w, bound, bufs = want
    for k in (0, 1):
        got = p.states[k].cpu().numpy()
        bad = np.nonzero(got != bufs[k])[0]
        assert bad.size == 0, f"{what}: moment {k}, {bad.size} bytes differ, first {bad[0]}: {got[bad[0]]} for {bufs[k][bad[0]]}"
    got = f64(p.w).reshape(-1)
    nan = np.isnan(w)
    assert np.array_equal(np.isnan(got), nan), what
    inf = np.isinf(w)
    assert np.array_equal(got[inf], w[inf]), what
    ok = ~nan & ~inf
    over = np.abs(got[ok] - w[ok]) - bound[ok]
    assert not over.size or over.max() <= 0, f"{what}: {over.max()} over the bound"


def step(ps, gs, hp, extra=()):
    plan = mo.muon_plan_create([(mo.MUON_KIND_ADAMW8, code(p.dtype), *p.shape, 0, 0) for p in ps])
    mo.muon_step(plan, [p.w for p in ps], gs, [None] * len(ps), [p.states[0] for p in ps], [p.states[1] for p in ps], hp,
                 None)


SIZES = [1, 2, 3, 4, 5, 7, 63, 255, 256, 257, 511, 1023, 1024, 1025, 4095, 4096, 4097, 10007]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n", SIZES)
def test_one_tensor(n, dtype):
    print("adamw8", n, dtype, flush=True)
    for shift in (0, 1, 2, 3):
        p = Param((1, n), dtype, n + shift, shift)
        g = p.grad(n + 100, (3 * shift) % 4)
        want = expect(p, g, 7, HP)
        around = p.w.untyped_storage()
        before = torch.empty(0, dtype=dtype, device=p.w.device).set_(around).clone()
        step([p], [g], hparams(7))
        compare(p, want, f"{n} {dtype} shift {shift}")
        after = torch.empty(0, dtype=dtype, device=p.w.device).set_(around)
        assert torch.equal(before[:shift], after[:shift]) and torch.equal(before[shift + n:], after[shift + n:])


def test_steps_follow_each_other():
    """Ten steps from zero moments, other gradients and hyperparameters each."""
    print("adamw8 ten steps", flush=True)
    ps = [Param((5, 101), BF, 1, zero=True), Param((33, 77), F32, 2, zero=True)]
    for t in range(1, 11):
        hp = dict(HP, beta1=0.9 if t % 2 else 0.0, beta2=0.999 if t % 3 else 0.5, wd=0.0 if t == 4 else 0.1,
                  eps=0.0 if t == 6 else 1e-8)
        gs = [p.grad(100 + 10 * t + i) for i, p in enumerate(ps)]
        want = [expect(p, g, t, hp) for p, g in zip(ps, gs)]
        step(ps, gs, hparams(t, **{k: hp[k] for k in ("beta1", "beta2", "wd", "eps")}))
        for p, w in zip(ps, want):
            compare(p, w, f"step {t}")


def test_many_tensors_and_empty_ones():
    """More than a launch takes, empty ones and large ones among them; and the
    same tensors in another order give the same results."""
    print("adamw8 many tensors", flush=True)
    shapes = [(1, 768)] * 70 + [(0, 5), (300, 257), (3, 0)] + [(1, 1 + 37 * i) for i in range(90)]
    ps = [Param(s, BF if i % 3 else F32, i) for i, s in enumerate(shapes) if s[0] * s[1]]
    gs = [p.grad(1000 + i) for i, p in enumerate(ps)]
    want = [expect(p, g, 3, HP) for p, g in zip(ps, gs)]
    again = [[p.w.clone(), p.states[0].clone(), p.states[1].clone()] for p in ps]
    table = [(3, mo.MUON_BF16, *s, 0, 0) for s in shapes[:0]]
    it = iter(zip(ps, gs))
    lists = [[], [], [], []]
    for i, s in enumerate(shapes):
        if s[0] * s[1]:
            p, g = next(it)
            table.append((3, code(p.dtype), *s, 0, 0))
            for lst, t in zip(lists, (p.w, g, p.states[0], p.states[1])):
                lst.append(t)
        else:
            table.append((3, mo.MUON_BF16, *s, 0, 0))
            for lst in lists:
                lst.append(None)
    plan = mo.muon_plan_create(table)
    mo.muon_step(plan, lists[0], lists[1], [None] * len(table), lists[2], lists[3], hparams(3), None)
    for i, (p, w) in enumerate(zip(ps, want)):
        compare(p, w, f"tensor {i}")
    order = list(range(len(ps)))[::-1]
    plan = mo.muon_plan_create([(3, code(ps[i].dtype), *ps[i].shape, 0, 0) for i in order])
    mo.muon_step(plan, [again[i][0] for i in order], [gs[i] for i in order], [None] * len(order),
                 [again[i][1] for i in order], [again[i][2] for i in order], hparams(3), None)
    for p, a in zip(ps, again):
        assert torch.equal(p.w, a[0]) and torch.equal(p.states[0], a[1]) and torch.equal(p.states[1], a[2])


def test_special_values():
    """NaN, infinities, zeros, the smallest and the largest floats in one block and alone."""
    print("adamw8 special values", flush=True)
    tiny, big = 1e-45, 3.4e38
    vals = [float("nan"), float("inf"), float("-inf"), 0.0, -0.0, tiny, -tiny, 1e-38, -1e-30, 1e-20, 1e18, -1e19, big, -big, 1.0]
    for dtype in (F32, BF):
        for case in range(len(vals) + 1):
            p = Param((2, 300), dtype, 50 + case, zero=case % 2 == 0)
            g = p.grad(60 + case)
            if case < len(vals):
                g.view(-1)[5] = vals[case]
                g.view(-1)[550] = vals[case]
            else:
                g.zero_()
                g.view(-1)[:len(vals)] = torch.tensor(vals, device=g.device, dtype=dtype)
            want = expect(p, g, 9, HP)
            step([p], [g], hparams(9))
            compare(p, want, f"case {case} {dtype}")
    # a block whose values are all under the smallest code of another
    p = Param((1, 256), F32, 3, zero=True)
    g = torch.full((1, 256), 1e-9, device=p.w.device)
    g[0, 17] = 1e3
    want = expect(p, g, 2, HP)
    step([p], [g], hparams(2))
    compare(p, want, "far below the largest")


@pytest.mark.parametrize("moment", [0, 1])
@pytest.mark.parametrize("n", [1, 4, 255, 256, 1000, 70001])
def test_pack_and_unpack(n, moment):
    print("adamw8 pack", n, moment, flush=True)
    rng = np.random.default_rng(n)
    x = (rng.standard_normal(n) * np.exp(rng.uniform(-40, 10, n))).astype(np.float32)
    x[rng.integers(0, n, n // 10)] = 0
    if n > 300:
        x[300] = np.nan
    if moment:
        x = np.abs(x)
    t = torch.from_numpy(x).to(dev())
    c, o = R.encode(x, 1 << 33, moment)
    state = mo.muon_adamw8_pack(t, moment, 1 << 33)
    assert np.array_equal(state.cpu().numpy(), R.to_state(c, o))
    out = mo.muon_adamw8_unpack(state, torch.full_like(t, 5.0), moment)
    assert np.array_equal(out.cpu().numpy(), R.decode(c, o, moment), equal_nan=True)
    # what a buffer stands for is kept by packing it again with any step
    if not np.isnan(x).any():
        assert torch.equal(mo.muon_adamw8_unpack(mo.muon_adamw8_pack(out, moment, 5), torch.empty_like(out), moment), out)


def test_next_to_the_other_kinds():
    """A table of Muon, AdamW and 8-bit AdamW parameters: each gets what it gets alone."""
    print("adamw8 mixed table", flush=True)
    d = dev()
    g = torch.Generator().manual_seed(1)
    rnd = lambda *s: (torch.randn(*s, generator=g) * 0.02).to(BF).to(d)
    p = Param((40, 301), BF, 8)
    pg = p.grad(9)
    want = expect(p, pg, 4, HP)
    muon, muon_g, mom = rnd(64, 96), rnd(64, 96), torch.zeros(64, 96, device=d)
    vec, vec_g, ea, es = rnd(1, 500), rnd(1, 500), torch.zeros(1, 500, device=d), torch.zeros(1, 500, device=d)
    alone = [t.clone() for t in (muon, mom, vec, ea, es)]
    hp = hparams(4)

    def run(table, *lists):
        plan = mo.muon_plan_create(table)
        ws = torch.empty(max(1, mo.muon_plan_workspace_bytes(plan)), dtype=torch.uint8, device=d)
        mo.muon_step(plan, *lists, hp, ws)

    run([(0, 1, 64, 96, 0, 0), (1, 1, 1, 500, 0, 0)], [alone[0], alone[2]], [muon_g, vec_g], [alone[1], None],
        [None, alone[3]], [None, alone[4]])
    run([(0, 1, 64, 96, 0, 0), (3, 1, 40, 301, 0, 0), (1, 1, 1, 500, 0, 0)], [muon, p.w, vec], [muon_g, pg, vec_g],
        [mom, None, None], [None, p.states[0], ea], [None, p.states[1], es])
    compare(p, want, "in a mixed table")
    for a, b in zip(alone, (muon, mom, vec, ea, es)):
        assert torch.equal(a, b)


def test_graph_replays_and_streams():
    """Captured into a graph and replayed with eager work between, on a stream of its own, and on two streams at once."""
    print("adamw8 under graph capture", flush=True)
    d = dev()
    ps = [Param((7, 999), BF, 1), Param((1, 5000), F32, 2)]
    gs = [p.grad(11 + i) for i, p in enumerate(ps)]
    init = [[p.w.clone(), p.states[0].clone(), p.states[1].clone()] for p in ps]
    want = [expect(p, g, 5, HP) for p, g in zip(ps, gs)]
    plan = mo.muon_plan_create([(3, code(p.dtype), *p.shape, 0, 0) for p in ps])
    args = ([p.w for p in ps], gs, [None, None], [p.states[0] for p in ps], [p.states[1] for p in ps], hparams(5), None)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mo.muon_step(plan, *args)

    def reset():
        for p, i in zip(ps, init):
            p.w.copy_(i[0])
            p.states[0].copy_(i[1])
            p.states[1].copy_(i[2])
        torch.cuda.synchronize()

    for replay in range(3):
        reset()
        graph.replay()
        torch.cuda.synchronize()
        for p, w in zip(ps, want):
            compare(p, w, f"replay {replay}")
    reset()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    mo.muon_step(plan, *args, stream=s)
    s.synchronize()
    for p, w in zip(ps, want):
        compare(p, w, "on a stream of its own")
    # one parameter on each of two streams
    reset()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for p, g, st in zip(ps, gs, streams):
        one = mo.muon_plan_create([(3, code(p.dtype), *p.shape, 0, 0)])
        mo.muon_step(one, [p.w], [g], [None], [p.states[0]], [p.states[1]], hparams(5), None, stream=st)
    torch.cuda.synchronize()
    for p, w in zip(ps, want):
        compare(p, w, "on two streams")


def test_offsets_past_34_bits():
    """A parameter of 2^34 + 1024 elements: its last block's result, whose
    groups' numbers pass 32 bits, and the first."""
    print("adamw8 2^34 elements", flush=True)
    d = dev()
    rows, cols = (1 << 24) + 1, 1024
    n = rows * cols
    nb = n // 256
    w, g = torch.zeros(rows, cols, dtype=BF, device=d), torch.zeros(rows, cols, dtype=BF, device=d)
    states = [torch.zeros(mo.muon_adamw8_state_bytes(n), dtype=torch.uint8, device=d) for _ in (0, 1)]
    tail = (torch.randn(512, generator=torch.Generator().manual_seed(1)) * 1e-3).to(BF)
    g.view(-1)[-512:] = tail.to(d)
    g.view(-1)[:512] = tail.to(d)
    plan = mo.muon_plan_create([(3, 1, rows, cols, 0, 0)])
    mo.muon_step(plan, [w], [g], [None], [states[0]], [states[1]], hparams(1), None)
    m, v = R.moments(tail.float().numpy(), np.zeros(512, np.float32), np.zeros(512, np.float32), 0.9, 0.95)
    want = R.weights(np.zeros(512), m, v, t=1, **HP)
    for first in (0, n - 512):
        for k, x in enumerate((m, v)):
            c, o = R.encode(x, 1, k, rand=R.random_bits(512, 1, k, first=first))
            assert np.array_equal(states[k][first:first + 512].cpu().numpy(), c), (first, k)
            at = n + 2 * (first // 256)
            assert np.array_equal(states[k][at:at + 4].cpu().numpy().view(np.uint16), o), (first, k)
        got = f64(w.view(-1)[first:first + 512])
        assert (np.abs(got - want) <= (10 * U + 2.0 ** -8) * np.abs(want)).all()
    assert states[0][512:n - 512].count_nonzero().item() == 0 and w.view(-1)[512:n - 512].count_nonzero().item() == 0
    assert nb * 256 == n


@pytest.mark.parametrize("eps", [1e-8, 0.0])
def test_a_large_tensor_by_its_blocks(eps):
    """60 M elements, which pass the caches: blocks from all over it against the reference."""
    print("adamw8 60 M elements", eps, flush=True)
    d = dev()
    rows, cols, t = 15001, 4001, 12
    n = rows * cols
    gen = torch.Generator(device=d).manual_seed(3)
    w = (torch.randn(rows, cols, generator=gen, device=d) * 0.02).to(BF)
    g = (torch.randn(rows, cols, generator=gen, device=d) * 1e-3).to(BF)
    states = [mo.muon_adamw8_pack(torch.randn(rows, cols, generator=gen, device=d).mul_(s).square_() if k else
                                  torch.randn(rows, cols, generator=gen, device=d).mul_(s), k, 11)
              for k, s in ((0, 3e-4), (1, 1e-3))]
    nb = -(-n // 256)
    blocks = sorted({0, 1, nb // 3, nb // 2 + 1, nb - 3, nb - 2, nb - 1})
    cut = lambda x, b: x.view(-1)[256 * b:min(n, 256 * b + 256)].cpu()
    offs = lambda s, b: s[nb * 256 + 2 * b:nb * 256 + 2 * b + 2].cpu().numpy().view(np.uint16)
    old = {b: (cut(w, b), cut(g, b), [(cut(s[:n], b).numpy(), offs(s, b)) for s in states]) for b in blocks}
    plan = mo.muon_plan_create([(3, 1, rows, cols, 0, 0)])
    mo.muon_step(plan, [w], [g], [None], [states[0]], [states[1]], hparams(t, eps=eps), None)
    for b in blocks:
        w0, gb, moments = old[b]
        m, v = R.moments(gb.float().numpy(), *[R.decode(c, o, k) for k, (c, o) in enumerate(moments)], 0.9, 0.95)
        for k, x in enumerate((m, v)):
            c, o = R.encode(x, t, k, rand=R.random_bits(x.size, t, k, first=256 * b))
            assert np.array_equal(cut(states[k][:n], b).numpy(), c) and np.array_equal(offs(states[k], b), o), (b, k)
        want = R.weights(w0.double().numpy(), m, v, t=t, **dict(HP, eps=eps))
        bound = 4 * U * np.abs(w0.double().numpy()) + 10 * U * np.abs(want - w0.double().numpy()) + 2.0 ** -8 * np.abs(want)
        assert (np.abs(f64(cut(w, b)) - want) <= bound).all(), b


def test_calls_that_the_quick_check_leaves_to_the_other():
    """Raw pointers, a tensor in a place its kind does not use, wrong dtypes and sizes."""
    print("adamw8 binding checks", flush=True)
    d = dev()
    p = Param((3, 100), BF, 1)
    g = p.grad(2)
    want = expect(p, g, 2, HP)
    plan = mo.muon_plan_create([(3, 1, 3, 100, 0, 0)])
    mo.muon_step(plan, [p.w.data_ptr()], [g.data_ptr()], [None], [p.states[0].data_ptr()], [p.states[1].data_ptr()],
                 hparams(2), None)
    compare(p, want, "raw pointers")
    want = expect(p, g, 3, HP)
    mo.muon_step(plan, [p.w], [g], [torch.zeros(1, device=d)], [p.states[0]], [p.states[1]], hparams(3), None)
    compare(p, want, "an unused tensor")
    before = [t.clone() for t in (p.w, *p.states)]
    cpu = torch.zeros(3, 100, dtype=BF)
    for bad in ([p.w.float()], [p.w[:2]], [cpu], [torch.zeros(100, 3, dtype=BF, device=d).t()]):
        with pytest.raises(ValueError):
            mo.muon_step(plan, bad, [g], [None], [p.states[0]], [p.states[1]], hparams(3), None)
    for bad in (p.states[0][:-1], p.states[0].float(), torch.zeros(3, 100, device=d)):
        with pytest.raises(ValueError):
            mo.muon_step(plan, [p.w], [g], [None], [bad], [p.states[1]], hparams(3), None)
    with pytest.raises(ValueError):
        mo.muon_step(plan, [p.w], [g], [cpu], [p.states[0]], [p.states[1]], hparams(3), None)
    with pytest.raises(mo.MuonError):
        mo.muon_step(plan, [p.w], [None], [None], [p.states[0]], [p.states[1]], hparams(3), None)
    assert all(torch.equal(a, b) for a, b in zip(before, (p.w, *p.states)))
