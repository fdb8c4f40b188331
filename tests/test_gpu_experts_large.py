"""GPU tests of the large products grouped by expert where their results are no
whole 16-byte pieces, where their operands or results reach past 2^31 elements
(every kernel of the products), with values that are not finite, after offsets
that go back, under graph replays and on two streams.  Operands are small whole
numbers: results are equal to products in fp64, rounded once."""
import pytest
import torch

from oracle import experts_ref as R
from tests import experts_cases as C
from tests.gpu_util import dev
from tests.test_gpu_experts import BF, F32, split_rows

mo = pytest.importorskip("matrix_orthogonalizing_optimizer_amd")

pytestmark = pytest.mark.gpu


def whole(gen, shape, dtype=BF, row=None, stride=None, shift=0):
    """Whole numbers from -3 to 3; rows `row` elements apart, matrices `stride`,
    from element `shift` on of a buffer whose other elements are not set."""
    *lead, cols = shape
    row = cols if row is None else row
    strides = [row, 1] if len(lead) == 1 else [stride or lead[1] * row, row, 1]
    n = shift + sum((s - 1) * st for s, st in zip(shape, strides)) + 1
    t = torch.empty(n, dtype=dtype, device=dev()).as_strided(shape, strides, shift)
    t.copy_(torch.randint(-3, 4, shape, generator=gen, device=dev()))
    return t


def product(a, b):
    return a.double().contiguous() @ b.double().contiguous()


def references(which, off, rows, A, B):
    """(expert, rows or None, its result in fp64) of a pass on its two operands."""
    for e, a, b in R.groups(off.tolist(), rows):
        if which == C.WEIGHT:
            yield e, None, product(A[a:b].t(), B[a:b])
        elif b > a:
            yield e, slice(a, b), product(A[a:b], B[e].t() if which == C.FORWARD else B[e])


def call(which, A, B, off, o, **kw):
    if which == C.FORWARD:
        return mo.muon_experts_forward(A, B, off, y=o, **kw)
    if which == C.INPUT:
        return mo.muon_experts_input_grad(A, B, off, dx=o, **kw)
    return mo.muon_experts_weight_grad(A, B, off, dw=o, **kw)


def shapes(which, rows, experts, out, in_):
    """Shapes of the two operands and of the result."""
    x, dy, w = (rows, in_), (rows, out), (experts, out, in_)
    return {C.FORWARD: (x, w, dy), C.INPUT: (dy, w, x), C.WEIGHT: (dy, x, w)}[which]


def check(which, off, rows, A, B, o, odt, what):
    for e, r, ref in references(which, off, rows, A, B):
        assert torch.equal(o[e if r is None else r], ref.to(odt)), (what, e)


@pytest.mark.parametrize("odt", [BF, F32])
@pytest.mark.parametrize("case", C.LARGE[:9], ids=lambda c: "-".join(map(str, c)))
def test_results_that_are_not_whole_pieces(case, odt):
    """Odd widths, rows an odd number of elements apart, results that start at any
    element; what lies around and between the rows stays."""
    which, rows, experts, out, in_ = case
    gen = torch.Generator(device=dev()).manual_seed(1)
    sa, sb, so = shapes(*case)
    A, B = whole(gen, sa), whole(gen, sb)
    for pad, shift in ((0, 0), (0, 1), (3, 0), (1, 5), (8, 8)):
        print("experts large results", case, odt, pad, shift, flush=True)
        off = split_rows(rows, experts, 7 + pad + shift, empty=0.3, lead=2, tail=3)
        row = so[-1] + pad
        n = shift + so[0] * (so[1] if len(so) == 3 else 1) * row + 64
        base = torch.full((n,), 77.0, dtype=odt, device=dev())
        strides = (so[1] * row, row, 1) if len(so) == 3 else (row, 1)
        o = base.as_strided(so, strides, shift)
        call(which, A, B, off, o)
        check(which, off, rows, A, B, o, odt, (case, pad, shift))
        if which != C.WEIGHT:
            assert (o[:2] == 77).all() and (o[rows - 3:] == 77).all()
        o.fill_(77.0)
        assert (base == 77).all(), (case, pad, shift)


@pytest.mark.parametrize("case", C.LARGE[3:9], ids=lambda c: "-".join(map(str, c)))
def test_values_that_are_not_finite(case):
    """NaN in a row that is an expert's, in rows of nobody, in the weights of
    experts without rows: only the results that take them are NaN."""
    which, rows, experts, out, in_ = case
    print("experts large not finite", case, flush=True)
    gen = torch.Generator(device=dev()).manual_seed(2)
    off = split_rows(rows, experts, 5, empty=0.3, lead=2, tail=3)
    groups = R.groups(off.tolist(), rows)
    sa, sb, so = shapes(*case)
    A, B = whole(gen, sa), whole(gen, sb)
    longest = max(groups, key=lambda g: g[2] - g[1])
    bad = (longest[1] + longest[2]) // 2
    for t in (A, B):
        if t.dim() == 2:
            t[:2] = t[rows - 3:] = float("nan")
    if which != C.WEIGHT:
        for e, a, b in groups:
            if a == b:
                B[e] = float("nan")
    A[bad, 5] = float("nan")
    o = torch.full(so, 77.0, device=dev())
    call(which, A, B, off, o)
    for e, r, ref in references(which, off, rows, A, B):
        got = o[e if r is None else r]
        assert torch.equal(got.isnan(), ref.isnan()), (case, e)
        assert torch.equal(got.nan_to_num(5.0), ref.float().nan_to_num(5.0)), (case, e)
        assert ref.isnan().any() == (e == longest[0])
    if which != C.WEIGHT:
        assert (o[:2] == 77).all() and (o[rows - 3:] == 77).all()


FAR = [  # pass, rows, experts, out, in, dtype of the operands, apart: rows in memory
    # few rows (two tiles), few rows (four tiles), tiles of 128 directly, through registers, in fp32, large tiles
    (C.FORWARD, 2400, 200, 96, 64, BF, 1 << 20), (C.FORWARD, 2400, 200, 40, 70, BF, 1 << 20),
    (C.FORWARD, 5000, 3, 136, 72, BF, 1 << 19), (C.FORWARD, 5000, 3, 136, 71, BF, 1 << 19),
    (C.FORWARD, 5000, 3, 136, 72, F32, 1 << 19),
    (C.INPUT, 5000, 3, 136, 72, BF, 1 << 19), (C.INPUT, 5000, 3, 137, 71, BF, 1 << 19), (C.INPUT, 5000, 3, 136, 72, F32, 1 << 19),
    (C.WEIGHT, 5000, 3, 136, 72, BF, 1 << 19), (C.WEIGHT, 5000, 3, 137, 71, BF, 1 << 19),
    (C.WEIGHT, 5000, 3, 136, 72, F32, 1 << 19),
] + [c + (BF, 1 << 19) for c in C.LARGE[9:]]


@pytest.mark.parametrize("case", FAR, ids=lambda c: "-".join(map(str, c)))
def test_past_31_bits(case):
    """Rows of the operands and of the result whose elements are numbered past
    2^31, then weights of experts that are."""
    which, rows, experts, out, in_, dtype, apart = case
    print("experts past 31 bits", case, flush=True)
    gen = torch.Generator(device=dev()).manual_seed(3)
    off = split_rows(rows, experts, 4, lead=1, tail=1)
    sa, sb, so = shapes(which, rows, experts, out, in_)
    far = (1 << 31) // max(1, min(experts, 3) - 1) + 8  # between experts
    for wide in ("rows", "experts"):
        def make(shape):
            if len(shape) == 2:
                return whole(gen, shape, dtype, row=apart if wide == "rows" else None)
            return whole(gen, shape, dtype, stride=far if wide == "experts" else None)
        if wide == "experts" and experts > 3:
            off = split_rows(rows := 20, experts := 3, 4, lead=1, tail=1)
            sa, sb, so = shapes(which, rows, experts, out, in_)
        A, B, o = make(sa), make(sb), make(so)
        last = [(s.size(0) - 1) * s.stride(0) for s in (A, B, o)]
        assert max(last) >= 1 << 31
        call(which, A, B, off, o)
        check(which, off, rows, A, B, o, dtype, (case, wide))
        del A, B, o


@pytest.mark.parametrize("back", [(0, 40000, 0, 30000), (39000, 40000, 0, 40000), (0, 20000, 15000, 40000)])
def test_the_call_after_offsets_that_go_back(back):
    """All three products are right after a call whose groups overlapped, on the
    same workspace."""
    print("experts after offsets back", back, flush=True)
    rows, e, out, in_ = 40000, 30, 2560, 520
    gen = torch.Generator(device=dev()).manual_seed(1)
    good = split_rows(rows, e, 3, lead=1)
    bad = torch.tensor(list(back) + [rows] * (e + 1 - len(back)), dtype=torch.int32, device=dev())
    for which in (C.FORWARD, C.WEIGHT, C.INPUT):
        sa, sb, so = shapes(which, rows, e, out, in_)
        A, B = whole(gen, sa), whole(gen, sb)
        o = torch.full(so, 77.0, dtype=BF, device=dev())
        ws = torch.empty(mo.muon_experts_workspace_bytes(which, rows, e, out, in_, mo.MUON_BF16), dtype=torch.uint8, device=dev())
        for off in (bad, good):
            call(which, A, B, off, o, workspace=ws)
        check(which, good, rows, A, B, o, BF, (which, back))


def test_graph_replays_and_two_streams():
    """The three large products captured into one graph on one workspace, replayed
    with other offsets; then on two streams at once, a workspace each."""
    print("experts large graph", flush=True)
    _, rows, e, out, in_ = C.LARGE[6]
    gen = torch.Generator(device=dev()).manual_seed(6)
    x, w, dy = whole(gen, (rows, in_)), whole(gen, (e, out, in_)), whole(gen, (rows, out))
    passes = ((C.FORWARD, x, w), (C.WEIGHT, dy, x), (C.INPUT, dy, w))
    off = split_rows(rows, e, 1)
    results = {p[0]: torch.zeros(shapes(p[0], rows, e, out, in_)[2], dtype=BF, device=dev()) for p in passes}
    size = max(mo.muon_experts_workspace_bytes(k, rows, e, out, in_, mo.MUON_BF16) for k in range(3))
    ws = [torch.empty(size, dtype=torch.uint8, device=dev()) for _ in range(2)]

    def run():
        for which, A, B in passes:
            call(which, A, B, off, results[which], workspace=ws[0])

    def verify(which, o, what):
        A, B = next(p[1:] for p in passes if p[0] == which)
        check(which, off, rows, A, B, o, BF, what)

    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    one = torch.tensor([0] + [rows] * e, dtype=torch.int32, device=dev())
    for replay, o in enumerate((split_rows(rows, e, 2, lead=3), one, torch.zeros_like(one), split_rows(rows, e, 3, empty=0.8))):
        off.copy_(o)
        for r in results.values():
            r.fill_(9)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for which, r in results.items():
            verify(which, r, f"replay {replay}")
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    many = []
    torch.cuda.synchronize()
    for i in range(6):
        which, A, B = passes[i % 3]
        o = torch.empty_like(results[which])
        torch.cuda.synchronize()
        many.append((which, o))
    for i, (which, o) in enumerate(many):
        A, B = next(p[1:] for p in passes if p[0] == which)
        call(which, A, B, off, o, workspace=ws[i % 2], stream=streams[i % 2])
    torch.cuda.synchronize()
    for i, (which, o) in enumerate(many):
        verify(which, o, f"stream {i}")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("experts,out,in_", [(65535, 8, 16), (65536, 8, 16), (65536, 5, 9)])
def test_as_many_experts_as_there_may_be(experts, out, in_, dtype):
    """2^16 experts, most of them with a row or none, a few with many."""
    print("experts at their limit", experts, out, in_, dtype, flush=True)
    rows = 70001
    gen = torch.Generator(device=dev()).manual_seed(9)
    n = torch.ones(experts, dtype=torch.int64, device=dev())
    n[torch.randint(0, experts, (30000,), generator=gen, device=dev())] = 0
    n[experts // 2], n[experts - 1] = 20000, 300
    off = torch.cat([n.new_zeros(1), n.cumsum(0)])
    assert off[-1] < rows
    mine = torch.repeat_interleave(torch.arange(experts, device=dev()), n)
    live = mine.numel()
    off = off.to(torch.int32)
    x, w, dy = whole(gen, (rows, in_), dtype), whole(gen, (experts, out, in_), dtype), whole(gen, (rows, out), dtype)
    y = mo.muon_experts_forward(x, w, off, y=torch.full((rows, out), 77.0, device=dev()))
    assert torch.equal(y[:live], (w[mine].double() * x[:live].double().unsqueeze(1)).sum(2).float()) and (y[live:] == 77).all()
    dx = mo.muon_experts_input_grad(dy, w, off, dx=torch.full((rows, in_), 77.0, device=dev()))
    assert torch.equal(dx[:live], (w[mine].double() * dy[:live].double().unsqueeze(2)).sum(1).float()) and (dx[live:] == 77).all()
    dw = mo.muon_experts_weight_grad(dy, x, off, dtype=F32)
    each = dy[:live].double().unsqueeze(2) * x[:live].double().unsqueeze(1)
    assert torch.equal(dw, torch.zeros(experts, out, in_, dtype=torch.float64, device=dev()).index_add_(0, mine, each).float())
