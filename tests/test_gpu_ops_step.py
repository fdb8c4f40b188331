"""The operators around the step together with the step: a two-block network
(layer norm -> 8-bit linear layer) is run forward and backward, its gradients
go to muon_step, and everything is compared with the fp64 reference fed with
the same 8-bit rows."""
import numpy as np
import pytest
import torch

import oracle
from oracle import ops_ref as R
from tests.gpu_util import dev, f64, hp_from, rel, stored
from workloads import configs

mo = pytest.importorskip("matrix_orthogonalizing_optimizer_amd")

pytestmark = pytest.mark.gpu

EPS = 1e-5


@pytest.mark.parametrize("tokens,width,out", [(512, 768, 768), (300, 320, 512)])
def test_training_step(tokens, width, out):
    print("training step", tokens, width, out, flush=True)
    d = dev()
    g = torch.Generator().manual_seed(tokens)
    rnd = lambda *s, k=1.0: (torch.randn(*s, generator=g) * k).to(torch.bfloat16).to(d)
    x = rnd(tokens, width)
    W, gamma, beta = rnd(out, width, k=0.02), (1 + rnd(width, k=0.1)), rnd(width, k=0.1)
    # forward: the norm's output exists as 8-bit rows only; they are kept
    q, s = mo._lib._empty_rows8(0, None, tokens, width)
    mean, rstd = torch.empty(tokens, device=d), torch.empty(tokens, device=d)
    mo.muon_norm_forward(x, gamma, beta, EPS, q=q, scale=s, mean=mean, rstd=rstd)
    wq, ws = mo.muon_rows8_quantize(W)
    y = mo.muon_linear8_forward(q, s, wq, ws)
    # loss = sum(y * target): dy is the target
    dy = rnd(tokens, out, k=1e-2)
    # backward
    gW = mo.muon_linear8_weight_grad(dy, q, s)
    dh = mo.muon_linear8_input_grad(dy, wq, ws)
    gg, gb = torch.empty_like(gamma), torch.empty_like(beta)
    dx = mo.muon_norm_backward(dh, x, gamma, mean, rstd, dgamma=gg, dbeta=gb)

    # the same in fp64 from the same 8-bit rows and statistics
    Q, S, WQ, WS = q.cpu().numpy(), f64(s), wq.cpu().numpy(), f64(ws)
    rh = R.norm_forward(f64(x), f64(gamma), f64(beta), EPS)[0]
    assert np.abs(R.restore(Q, S) - rh).max() <= (S.max() / 2) * 1.001
    half = 2.0 ** -8  # one rounding to bf16
    assert rel(f64(y), R.linear8_forward(Q, S, WQ, WS)) <= half
    assert rel(f64(gW), R.linear8_weight_grad(f64(dy), Q, S)) <= half
    rdh = R.linear8_input_grad(f64(dy), WQ, WS)
    assert rel(f64(dh), rdh) <= half
    rdx, rg, rb = R.norm_backward(rdh, f64(x), f64(gamma), f64(mean), f64(rstd))
    # dh was rounded on the way; its rounding enters dx and the sums once more
    assert rel(f64(dx), rdx) <= 2 * half and rel(f64(gg), rg) <= 2 * half and rel(f64(gb), rb) <= 2 * half

    # the step takes the gradients as they are
    table = [(0, 1, out, width, 0, 0), (1, 1, 1, width, 0, 0), (1, 1, 1, width, 0, 0)]
    P = [W.clone(), gamma.clone().view(1, -1), beta.clone().view(1, -1)]
    G = [gW, gg.view(1, -1), gb.view(1, -1)]
    M = [torch.zeros(out, width, device=d), None, None]
    EA = [None, torch.zeros(1, width, device=d), torch.zeros(1, width, device=d)]
    ES = [None, torch.zeros(1, width, device=d), torch.zeros(1, width, device=d)]
    # Newton-Schulz in fp32: this gradient has full rank, and in bf16 the
    # iteration amplifies rounding at singular values near zero (0.03 measured
    # against 2e-2, which holds for the low-rank gradients of the workloads)
    plan = mo.muon_plan_create(table, mo.MUON_NS_STANDARD, mo.MUON_F32)
    wsp = torch.empty(mo.muon_plan_workspace_bytes(plan), dtype=torch.uint8, device=d)
    W0 = [f64(p) for p in P]
    hp = configs._hp()
    mo.muon_step(plan, P, G, M, EA, ES, hp_from(hp), wsp)
    z = [np.zeros((1, width)) if r[0] == 1 else None for r in table]
    ref = oracle.muon_step(table, W0, [f64(t) for t in G], [np.zeros((out, width)), None, None], z,
                           [None if a is None else a.copy() for a in z], oracle.OracleHparams())
    for i in range(3):
        want = stored(ref["W"][i], torch.bfloat16)
        assert rel(f64(P[i]) - W0[i], want - W0[i]) <= 2e-2, i
    # the next forward pass uses the updated weight's 8-bit rows
    wq2, ws2 = mo.muon_rows8_quantize(P[0])
    y2 = mo.muon_linear8_forward(q, s, wq2, ws2)
    assert rel(f64(y2), R.linear8_forward(Q, S, wq2.cpu().numpy(), f64(ws2))) <= half


def test_gradients_of_microbatches_add_up():
    """fp32 gradients accumulated over microbatches equal those of the whole
    batch up to fp32 rounding: 1200 terms in another grouping, a random walk
    of at most sqrt(1200) u = 2e-6 of the norm."""
    d = dev()
    g = torch.Generator().manual_seed(3)
    T, N, K = 1200, 130, 200
    x = torch.randn(T, K, generator=g).to(torch.bfloat16).to(d)
    dy = (torch.randn(T, N, generator=g) * 1e-3).to(d)
    q, s = mo.muon_rows8_quantize(x)
    whole = mo.muon_linear8_weight_grad(dy, q, s)
    parts = torch.empty_like(whole)
    for i, lo in enumerate(range(0, T, 400)):
        mo.muon_linear8_weight_grad(dy[lo:lo + 400], q[lo:lo + 400], s[lo:lo + 400], dw=parts, accumulate=i > 0)
    assert float((whole - parts).norm() / whole.norm()) <= 2e-6
