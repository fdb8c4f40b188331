"""A training step of a mixture-of-experts block with everything it uses: RMS
norm -> product by expert -> ReLU -> product by expert, the gradients of all of
them, then muon_step with the experts' weights as Muon parameters whose units
are the experts, and the norm's weight and an embedding on 8-bit AdamW moments.
Each result is compared with the fp64 reference fed with what the device read."""
import numpy as np
import pytest
import torch

import oracle
from oracle import adamw8_ref as A8
from oracle import cref, ops_ref
from oracle import experts_ref as R
from tests.gpu_util import StepRunner, dev, f64, rel, stored

mo = pytest.importorskip("matrix_orthogonalizing_optimizer_amd")

pytestmark = pytest.mark.gpu

U, HALF = 2.0 ** -24, 2.0 ** -8
BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-5


def routing(tokens, experts, seed, empty):
    g = np.random.default_rng(seed)
    p = g.random(experts) + 0.1
    p[empty] = 0
    n = g.multinomial(tokens, p / p.sum())
    return torch.tensor(np.concatenate([[0], np.cumsum(n)]).astype(np.int32))


class Block:
    def __init__(self, tokens, experts, width, hidden, vocabulary, seed):
        g = torch.Generator().manual_seed(seed)
        d = dev()
        rnd = lambda *s, k=1.0: (torch.randn(*s, generator=g) * k).to(BF).to(d)
        self.T, self.E, self.D, self.H, self.V = tokens, experts, width, hidden, vocabulary
        self.x, self.dy = rnd(tokens, width), rnd(tokens, width, k=1e-2)
        self.up, self.down = rnd(experts * hidden, width, k=width ** -0.5), rnd(experts * width, hidden, k=hidden ** -0.5)
        self.gamma, self.table = 1 + rnd(1, width, k=0.1), rnd(vocabulary, width, k=0.02)
        self.gtable = rnd(vocabulary, width, k=1e-3)
        self.off = torch.zeros(experts + 1, dtype=torch.int32, device=d)
        z = lambda *s: torch.zeros(*s, device=d, dtype=BF)
        self.h, self.a, self.y = z(tokens, width), z(tokens, hidden), z(tokens, width)
        self.da, self.dh, self.dx = z(tokens, hidden), z(tokens, width), z(tokens, width)
        self.rstd = torch.zeros(tokens, device=d)
        self.gup, self.gdown, self.ggamma = torch.zeros_like(self.up), torch.zeros_like(self.down), torch.zeros_like(self.gamma)
        rows = [(0, 1, experts * hidden, width, hidden, 0), (0, 1, experts * width, hidden, width, 0),
                (mo.MUON_KIND_ADAMW8, 1, 1, width, 0, 0), (mo.MUON_KIND_ADAMW8, 1, vocabulary, width, 0, 0)]
        self.rows = rows
        # Newton-Schulz in fp32: these gradients have full rank, and bf16
        # amplifies its rounding at singular values near zero
        self.run = StepRunner(rows, mo.MUON_NS_STANDARD, mo.MUON_F32)
        self.P = [self.up, self.down, self.gamma, self.table]
        self.G = [self.gup, self.gdown, self.ggamma, self.gtable]
        self.M = [torch.zeros(*self.up.shape, device=d), torch.zeros(*self.down.shape, device=d), None, None]
        state = lambda t: torch.zeros(mo.muon_adamw8_state_bytes(t.numel()), dtype=torch.uint8, device=d)
        self.S = [[None, None, state(self.gamma), state(self.table)] for _ in (0, 1)]
        n = max(mo.muon_experts_workspace_bytes(op, tokens, experts, *oi, mo.MUON_BF16)
                for op in range(3) for oi in ((hidden, width), (width, hidden)))
        self.ws = torch.empty(n + 256, dtype=torch.uint8, device=d)

    def train(self, step):
        ws = dict(workspace=self.ws)
        mo.muon_norm_forward(self.x, self.gamma.view(-1), None, EPS, mo.MUON_NORM_RMS, y=self.h, rstd=self.rstd)
        mo.muon_experts_forward(self.h, self.up, self.off, y=self.a, **ws)
        self.a.relu_()
        mo.muon_experts_forward(self.a, self.down, self.off, y=self.y, **ws)
        mo.muon_experts_weight_grad(self.dy, self.a, self.off, dw=self.gdown, **ws)
        mo.muon_experts_input_grad(self.dy, self.down, self.off, dx=self.da, **ws)
        self.da.mul_(self.a > 0)
        mo.muon_experts_weight_grad(self.da, self.h, self.off, dw=self.gup, **ws)
        mo.muon_experts_input_grad(self.da, self.up, self.off, dx=self.dh, **ws)
        mo.muon_norm_backward(self.dh, self.x, self.gamma.view(-1), None, self.rstd, mo.MUON_NORM_RMS, dx=self.dx,
                              dgamma=self.ggamma.view(-1))
        self.run.step(self.P, self.G, self.M, *self.S, self.hparams(step))

    def hparams(self, step):
        return mo.make_hparams(lr=2e-2, momentum=0.95, weight_decay=0.1, nesterov=True, ns_steps=5, adam_lr=3e-4,
                               adam_beta1=0.9, adam_beta2=0.95, adam_eps=1e-8, adam_weight_decay=0.1, adam_step=step)

    def all(self):
        return self.P + self.G + [m for m in self.M if m is not None] + [s for k in self.S for s in k if s is not None] + [
            self.h, self.a, self.y, self.da, self.dh, self.dx]


def product(got, ref, terms, K, what):
    """The bound of a product of K terms rounded to bf16 (K + 41 fp32 roundings)."""
    over = np.abs(f64(got).reshape(ref.shape) - ref) - ((K + 41) * U * terms + HALF * np.abs(ref) * (1 + (K + 41) * U))
    assert over.max() <= 0, (what, over.max())


def check(b, before, step):
    """b after a step against the reference fed with `before` (the weights and
    states) and with the rounded results that the device handed on."""
    P0, M0, S0 = before
    T, E, D, H = b.T, b.E, b.D, b.H
    o = b.off.cpu().numpy()
    up, down = P0[0].reshape(E, H, D), P0[1].reshape(E, D, H)
    h, a, dy, da, dh = (f64(t) for t in (b.h, b.a, b.dy, b.da, b.dh))
    zero = lambda n: np.zeros((T, n))
    rh = ops_ref.norm_forward(f64(b.x), P0[2].reshape(-1), None, EPS, layer=False)[0]
    assert np.abs(h - rh).max() <= (HALF + 16 * U) * np.abs(rh).max()
    ra, terms = R.forward(h, up, o, zero(H)), R.forward(np.abs(h), np.abs(up), o, zero(H))
    product(b.a, np.maximum(ra, 0), terms, D, "up")
    product(b.y, R.forward(a, down, o, zero(D)), R.forward(a, np.abs(down), o, zero(D)), H, "down")
    product(b.gdown, R.weight_grad(dy, a, o), R.weight_grad(np.abs(dy), a, o), T, "down's gradient")
    live = a > 0
    product(b.da, R.input_grad(dy, down, o, zero(H)) * live, R.input_grad(np.abs(dy), np.abs(down), o, zero(H)), D, "to the ReLU")
    product(b.gup, R.weight_grad(da, h, o), R.weight_grad(np.abs(da), np.abs(h), o), T, "up's gradient")
    product(b.dh, R.input_grad(da, up, o, zero(D)), R.input_grad(np.abs(da), np.abs(up), o, zero(D)), H, "to the norm")
    rdx, rg, _ = ops_ref.norm_backward(dh, f64(b.x), P0[2].reshape(-1), None, f64(b.rstd), layer=False)
    assert rel(f64(b.dx), rdx) <= 1.01 * HALF and rel(f64(b.ggamma).reshape(-1), rg) <= 1.01 * HALF
    # the Muon parameters, expert by expert
    hp = oracle.OracleHparams(lr=2e-2, momentum=0.95, weight_decay=0.1, nesterov=True, ns_steps=5)
    ref = cref.muon_step(b.rows[:2], P0[:2], [f64(g) for g in b.G[:2]], M0, [None] * 2, [None] * 2, hp)
    for i, unit in ((0, H), (1, D)):
        got, old, want = f64(b.P[i]), P0[i], stored(ref["W"][i], BF)
        for e in range(E):
            s = slice(e * unit, (e + 1) * unit)
            assert rel(got[s] - old[s], want[s] - old[s]) <= 2e-2, (i, e)
        assert rel(f64(b.M[i]), ref["M"][i]) <= 1e-6
    # 8-bit AdamW: the codes bit for bit, the weights within their roundings
    for i in (2, 3):
        n = P0[i].size
        m, v = A8.moments(f64(b.G[i]).reshape(-1), *[A8.decode(*A8.from_state(S0[k][i], n), k) for k in (0, 1)], 0.9, 0.95)
        for k, x in enumerate((m, v)):
            c, off = A8.from_state(b.S[k][i].cpu().numpy(), n)
            rc, roff = A8.encode(x, step, k)
            assert np.array_equal(c, rc) and np.array_equal(off, roff), (i, k)
        w0 = P0[i].reshape(-1)
        want = A8.weights(w0, m, v, lr=3e-4, beta1=0.9, beta2=0.95, eps=1e-8, wd=0.1, t=step)
        bound = 4 * U * np.abs(w0) + 10 * U * np.abs(want - w0) + HALF * np.abs(want)
        assert (np.abs(f64(b.P[i]).reshape(-1) - want) <= bound).all(), i


def keep(b):
    return ([f64(p) for p in b.P], [f64(m) for m in b.M[:2]], [[None if s is None else s.cpu().numpy() for s in k] for k in b.S])


@pytest.mark.parametrize("tokens,experts,width,hidden", [(400, 5, 96, 160), (37, 9, 64, 130)])
def test_training_steps(tokens, experts, width, hidden):
    """Two steps with other routings, an expert without tokens in each; the
    second also captured into a graph and replayed from the same state."""
    print("experts training step", tokens, experts, width, hidden, flush=True)
    b = Block(tokens, experts, width, hidden, 50, tokens)
    b.off.copy_(routing(tokens, experts, 1, 2))
    before = keep(b)
    b.train(1)
    torch.cuda.synchronize()
    check(b, before, 1)

    b.off.copy_(routing(tokens, experts, 2, 0))
    start = [t.clone() for t in b.all()]
    before = keep(b)
    b.train(2)
    torch.cuda.synchronize()
    check(b, before, 2)
    want = [t.clone() for t in b.all()]

    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        b.train(2)
    for replay in range(3):
        for t, s in zip(b.all(), start):
            t.copy_(s)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for i, (t, w) in enumerate(zip(b.all(), want)):
            assert torch.equal(t, w), (replay, i)
    # the same graph with another routing, which only the device knows
    for t, s in zip(b.all(), start):
        t.copy_(s)
    b.off.copy_(routing(tokens, experts, 3, 1))
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    check(b, before, 2)
