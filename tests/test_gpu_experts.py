"""GPU tests of the products grouped by expert against the fp64 reference.

Operands of small whole numbers make every partial sum exact in fp32 whatever
its order, so fp32 results have to be equal, and bf16 ones the nearest bf16 of
the reference: a product that takes one element too many or too few shows.
Operands of any values: u = 2^-24 bounds one fp32 rounding, a sum of K products
passes K additions and at most 40 more where its parts are joined, each product
is rounded once in fp32 (bf16 products are exact): (K + 41) u sum |terms|, and
half a step of the result's type."""
import numpy as np
import pytest
import torch

from oracle import experts_ref as R
from tests.gpu_util import dev, f64

mo = pytest.importorskip("matrix_orthogonalizing_optimizer_amd")

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


def tensor(shape, dtype, seed, pad=0, shift=0, whole=True, scale=1.0):
    """A device tensor whose rows lie pad elements further apart than they are
    long, shift elements into its storage."""
    g = torch.Generator().manual_seed(seed)
    *lead, cols = shape
    rows = int(np.prod(lead))
    n = rows * (cols + pad) + shift + pad
    v = torch.randint(-3, 4, (n,), generator=g).float() if whole else torch.randn(n, generator=g) * scale
    return v.to(dtype).to(dev())[shift:shift + rows * (cols + pad)].view(*lead, cols + pad)[..., :cols]


def split_rows(rows, experts, seed, empty=0.2, lead=0, tail=0):
    """Offsets of ragged groups, some empty, `lead` and `tail` rows of nobody's."""
    g = np.random.default_rng(seed)
    p = g.random(experts) ** 3 * (g.random(experts) > empty)
    if p.sum() == 0:
        p[-1] = 1
    n = g.multinomial(rows - lead - tail, p / p.sum())
    return torch.from_numpy(np.concatenate([[lead], lead + np.cumsum(n)]).astype(np.int32)).to(dev())


def nearest(ref, dtype):
    return torch.from_numpy(ref).to(dtype).double().numpy()


def same(got, ref, dtype, what):
    got = f64(got)
    want = nearest(ref, dtype)
    bad = np.argwhere(got != want)
    assert bad.size == 0, f"{what}: {len(bad)} differ, first at {bad[0]}: {got[tuple(bad[0])]} for {want[tuple(bad[0])]}"


def run_all(rows, experts, out, in_, dtype, off, seed=0, pads=(0, 0, 0), shifts=(0, 0, 0), odtypes=(BF, F32), what=""):
    x = tensor((rows, in_), dtype, seed + 1, pads[0], shifts[0])
    w = tensor((experts, out, in_), dtype, seed + 2, pads[1], shifts[1])
    dy = tensor((rows, out), dtype, seed + 3, pads[2], shifts[2])
    o = off.cpu().numpy()
    fx, fw, fdy = f64(x), f64(w), f64(dy)
    for odt in odtypes:
        y0 = tensor((rows, out), odt, 9, pads[2], shifts[1])
        ref = R.forward(fx, fw, o, f64(y0))
        same(mo.muon_experts_forward(x, w, off, y=y0), ref, odt, f"forward {what} {odt}")
        dx0 = tensor((rows, in_), odt, 8, pads[1], shifts[0])
        ref = R.input_grad(fdy, fw, o, f64(dx0))
        same(mo.muon_experts_input_grad(dy, w, off, dx=dx0), ref, odt, f"input grad {what} {odt}")
        dw0 = tensor((experts, out, in_), odt, 7, pads[0], shifts[2])
        ref = R.weight_grad(fdy, fx, o)
        old = f64(dw0)
        same(mo.muon_experts_weight_grad(dy, x, off, dw=dw0), ref, odt, f"weight grad {what} {odt}")
        if odt == F32:
            dw0 = tensor((experts, out, in_), odt, 7, pads[0], shifts[2])
            mo.muon_experts_weight_grad(dy, x, off, dw=dw0, accumulate=True)
            same(dw0, ref + old, odt, f"weight grad added {what}")


SHAPES = [  # rows, experts, out, in
    (1, 1, 1, 1), (1, 1, 8, 8), (2, 3, 5, 7), (5, 2, 16, 8), (7, 7, 3, 129), (16, 4, 64, 64), (17, 4, 65, 63), (31, 5, 24, 40),
    (64, 2, 128, 128), (65, 3, 127, 129), (100, 1, 136, 200), (128, 8, 130, 66), (129, 2, 256, 64), (200, 65, 40, 48),
    (257, 130, 33, 31), (300, 64, 72, 136), (513, 6, 264, 120), (777, 5, 301, 129), (1000, 200, 16, 24), (1531, 13, 701, 301),
]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", SHAPES)
def test_ragged_groups(shape, dtype):
    rows, experts, out, in_ = shape
    print("experts", shape, dtype, flush=True)
    run_all(*shape, dtype, split_rows(rows, experts, rows + experts), what=shape)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_strides_and_alignment(dtype):
    """Rows apart and anywhere in their storage: of whole 16-byte pieces and not."""
    print("experts strides", dtype, flush=True)
    off = split_rows(300, 5, 3, lead=7, tail=9)
    for pads, shifts in (((8, 16, 24), (0, 0, 0)), ((8, 16, 24), (8, 16, 8)), ((1, 0, 0), (0, 0, 0)), ((0, 3, 0), (0, 1, 0)),
                         ((0, 0, 5), (0, 0, 3)), ((2, 4, 6), (1, 2, 3)), ((0, 0, 0), (1, 0, 0)), ((0, 0, 0), (0, 0, 4))):
        run_all(300, 5, 136, 72, dtype, off, 4, pads, shifts, what=(pads, shifts))
    run_all(90, 5, 5, 3, dtype, split_rows(90, 5, 1, lead=1), 5, (1, 2, 3), (3, 2, 1), what="narrow")


@pytest.mark.parametrize("counts", [[0, 0, 300, 0], [300, 0, 0, 0], [0, 0, 0, 300], [75, 75, 75, 75], [128, 128, 44, 0],
                                    [1, 1, 1, 297], [0, 0, 0, 0], [129, 0, 171, 0]])
def test_who_gets_the_rows(counts):
    print("experts counts", counts, flush=True)
    off = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device=dev())
    run_all(300, 4, 264, 136, BF, off, 6, what=counts)
    run_all(300, 4, 33, 35, F32, off, 6, what=counts)


def test_rows_of_nobody_are_not_read_or_written():
    print("experts rows of nobody", flush=True)
    d = dev()
    off = torch.tensor([3, 10, 10, 40], dtype=torch.int32, device=d)
    x, w, dy = tensor((50, 72), BF, 1), tensor((3, 136, 72), BF, 2), tensor((50, 136), BF, 3)
    for t in (x, dy):
        t[:3] = float("nan")
        t[40:] = float("nan")
    w[1] = float("nan")  # an expert without rows
    y = torch.full((50, 136), 7.0, dtype=BF, device=d)
    mo.muon_experts_forward(x, w, off, y=y)
    assert (y[:3] == 7).all() and (y[40:] == 7).all()
    fw, fx, fdy, o = np.nan_to_num(f64(w)), np.nan_to_num(f64(x)), np.nan_to_num(f64(dy)), off.cpu().numpy()
    same(y, R.forward(fx, fw, o, np.full((50, 136), 7.0)), BF, "forward")
    dx = torch.full((50, 72), 5.0, dtype=F32, device=d)
    mo.muon_experts_input_grad(dy, w, off, dx=dx)
    same(dx, R.input_grad(fdy, fw, o, np.full((50, 72), 5.0)), F32, "input grad")
    same(mo.muon_experts_weight_grad(dy, x, off, dtype=F32), R.weight_grad(fdy, fx, o), F32, "weight grad")


def test_values_that_are_not_finite_stay_with_their_rows():
    """NaN and infinities in one row, one weight row: only the results that take them have them."""
    print("experts not finite", flush=True)
    off = torch.tensor([0, 40, 90], dtype=torch.int32, device=dev())
    for dtype in (BF, F32):
        x, w, dy = tensor((90, 136), dtype, 1), tensor((2, 264, 136), dtype, 2), tensor((90, 264), dtype, 3)
        x[45, 7], w[0, 100, 50], dy[10, 200] = float("nan"), float("inf"), float("-inf")
        args = f64(x), f64(w), f64(dy), off.cpu().numpy()
        with np.errstate(all="ignore"):
            refs = (R.forward(args[0], args[1], args[3], np.zeros((90, 264))),
                    R.input_grad(args[2], args[1], args[3], np.zeros((90, 136))), R.weight_grad(args[2], args[0], args[3]))
        gots = (mo.muon_experts_forward(x, w, off, dtype=F32), mo.muon_experts_input_grad(dy, w, off, dtype=F32),
                mo.muon_experts_weight_grad(dy, x, off, dtype=F32))
        for got, ref, what in zip(gots, refs, ("forward", "input grad", "weight grad")):
            got = f64(got)
            assert np.array_equal(np.isnan(got), np.isnan(ref)), (what, dtype)
            ok = ~np.isnan(ref)
            assert np.array_equal(got[ok], ref[ok]), (what, dtype)


def test_offsets_outside_the_rows():
    """Offsets below 0 and above the rows count as the nearest; ones that go back keep inside the buffers."""
    print("experts offsets outside", flush=True)
    d = dev()
    off = torch.tensor([-5, 20, 20, 1 << 30, (1 << 31) - 1], dtype=torch.int32, device=d)
    run_all(60, 4, 136, 72, BF, off, 3, what="outside")
    x, w, dy = tensor((60, 72), BF, 1), tensor((4, 136, 72), BF, 2), tensor((60, 136), BF, 3)
    for back in ([50, 10, 60, 0, 60], [60, 0, 60, 0, 60], [0, 60, 0, 60, 30], [-1, -7, 3, -9, 2]):
        o = torch.tensor(back, dtype=torch.int32, device=d)
        around = torch.full((80, 136), 3.0, dtype=BF, device=d)
        mo.muon_experts_forward(x, w, o, y=around[10:70])
        assert (around[:10] == 3).all() and (around[70:] == 3).all()
        around = torch.full((80, 72), 3.0, dtype=BF, device=d)
        mo.muon_experts_input_grad(dy, w, o, dx=around[10:70])
        assert (around[:10] == 3).all() and (around[70:] == 3).all()
        around = torch.full((6, 136, 72), 3.0, dtype=BF, device=d)
        mo.muon_experts_weight_grad(dy, x, o, dw=around[1:5])
        assert (around[0] == 3).all() and (around[5] == 3).all()


LARGE = [  # large tiles, sums that are split, many experts
    (4096, 8, 2560, 264), (5000, 3, 1408, 2048), (20000, 1, 72, 136), (40000, 2, 8, 16), (64, 2, 40, 14336), (3000, 40, 520, 776),
    (9000, 300, 264, 136),
]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", LARGE)
def test_large_and_long(shape, dtype):
    rows, experts, out, in_ = shape
    print("experts large", shape, dtype, flush=True)
    run_all(*shape, dtype, split_rows(rows, experts, experts, lead=3, tail=5), what=shape)
    if shape[0] == 5000 or shape[1] == 40:
        run_all(rows, experts, out - 1, in_ - 3, dtype, split_rows(rows, experts, experts), what="odd")


@pytest.mark.parametrize("shape", [(3000, 60, 1152, 1032), (9000, 12, 5128, 1288), (700, 1000, 264, 264), (2600, 2048, 264, 136),
                                   (40000, 30, 2560, 520)])
def test_many_tiles(shape):
    """Each workgroup computes many tiles one after the other, of experts with no
    row, of one stage of K, and of many; every value against products in fp64 on
    the device (whole numbers: exact)."""
    rows, experts, out, in_ = shape
    print("experts many tiles", shape, flush=True)
    d = dev()
    off = split_rows(rows, experts, 3, empty=0.3, lead=1, tail=2)
    gen = torch.Generator(device=d).manual_seed(1)
    whole = lambda *s: torch.randint(-3, 4, s, generator=gen, device=d).to(BF)
    x, w, dy = whole(rows, in_), whole(experts, out, in_), whole(rows, out)
    nan = float("nan")
    for odt in (F32, BF):
        y = torch.full((rows, out), nan, dtype=odt, device=d)
        dx = torch.full((rows, in_), nan, dtype=odt, device=d)
        dw = torch.full((experts, out, in_), nan, dtype=odt, device=d)
        mo.muon_experts_forward(x, w, off, y=y)
        mo.muon_experts_input_grad(dy, w, off, dx=dx)
        mo.muon_experts_weight_grad(dy, x, off, dw=dw)
        for e, a, b in R.groups(off.tolist(), rows):
            ref = dy[a:b].double().t().contiguous() @ x[a:b].double()
            assert torch.equal(dw[e], ref.to(odt)), ("weight grad", e, odt)
            if b > a:
                assert torch.equal(y[a:b], (x[a:b].double() @ w[e].double().t().contiguous()).to(odt)), ("forward", e, odt)
                assert torch.equal(dx[a:b], (dy[a:b].double() @ w[e].double()).to(odt)), ("input grad", e, odt)
        for t in (y, dx):
            assert t[0].isnan().all() and t[rows - 2:].isnan().all()
    before = dw.clone()
    mo.muon_experts_weight_grad(dy, x, off, dw=dw, accumulate=True)
    for e, a, b in R.groups(off.tolist(), rows):
        ref = dy[a:b].double().t().contiguous() @ x[a:b].double() + before[e].double()
        assert torch.equal(dw[e], ref.to(BF)), ("weight grad added", e)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", [(777, 5, 301, 129), (600, 4, 512, 1024), (64, 8, 128, 4096), (3000, 2, 136, 72)])
def test_any_values(shape, dtype):
    rows, experts, out, in_ = shape
    print("experts any values", shape, dtype, flush=True)
    off = split_rows(rows, experts, 5)
    x, w = tensor((rows, in_), dtype, 1, whole=False), tensor((experts, out, in_), dtype, 2, whole=False, scale=0.02)
    dy = tensor((rows, out), dtype, 3, whole=False, scale=1e-3)
    o, fx, fw, fdy = off.cpu().numpy(), f64(x), f64(w), f64(dy)
    for odt in (BF, F32):
        half = torch.finfo(odt).eps / 2
        cases = ((mo.muon_experts_forward(x, w, off, dtype=odt), lambda a, b, c: R.forward(a, b, o, np.zeros((rows, out))), in_),
                 (mo.muon_experts_input_grad(dy, w, off, dtype=odt),
                  lambda a, b, c: R.input_grad(c, b, o, np.zeros((rows, in_))), out),
                 (mo.muon_experts_weight_grad(dy, x, off, dtype=odt), lambda a, b, c: R.weight_grad(c, a, o), rows))
        for got, f, K in cases:
            ref, terms = f(fx, fw, fdy), f(np.abs(fx), np.abs(fw), np.abs(fdy))
            over = np.abs(f64(got) - ref) - ((K + 41) * U * terms + half * np.abs(ref) * (1 + (K + 41) * U))
            assert over.max() <= 0, (shape, dtype, odt, K, over.max())


def test_graphs_streams_and_changing_offsets():
    """Captured once and replayed with other offsets, which only the device
    sees; on a stream of its own; two calls on two streams at once."""
    print("experts under graph capture", flush=True)
    d = dev()
    rows, experts, out, in_ = 700, 6, 264, 136
    x, w, dy = tensor((rows, in_), BF, 1), tensor((experts, out, in_), BF, 2), tensor((rows, out), BF, 3)
    fx, fw, fdy = f64(x), f64(w), f64(dy)
    off = split_rows(rows, experts, 1)
    bufs = dict(y=torch.zeros(rows, out, device=d), dx=torch.zeros(rows, in_, device=d), dw=torch.zeros(experts, out, in_, device=d))
    ws = torch.empty(max(mo.muon_experts_workspace_bytes(k, rows, experts, out, in_, mo.MUON_BF16) for k in range(3)) + 1,
                     dtype=torch.uint8, device=d)

    def call(stream=None):
        mo.muon_experts_forward(x, w, off, y=bufs["y"], workspace=ws, stream=stream)
        mo.muon_experts_input_grad(dy, w, off, dx=bufs["dx"], workspace=ws, stream=stream)
        mo.muon_experts_weight_grad(dy, x, off, dw=bufs["dw"], workspace=ws, stream=stream)

    def verify(what):
        o = off.cpu().numpy()
        same(bufs["y"], R.forward(fx, fw, o, np.zeros((rows, out))), F32, what)
        same(bufs["dx"], R.input_grad(fdy, fw, o, np.zeros((rows, in_))), F32, what)
        same(bufs["dw"], R.weight_grad(fdy, fx, o), F32, what)

    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for replay in range(4):
        off.copy_(split_rows(rows, experts, 20 + replay, lead=5 * replay, tail=replay))
        for b in bufs.values():
            b.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        verify(f"replay {replay}")
    for b in bufs.values():
        b.zero_()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    call(s)
    s.synchronize()
    verify("stream of its own")
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    results = []
    for i in range(4):
        results.append(mo.muon_experts_weight_grad(dy, x, off, dtype=F32, stream=streams[i % 2]))
        results.append(mo.muon_experts_forward(x, w, off, dtype=F32, stream=streams[1 - i % 2]))
    torch.cuda.synchronize()
    o = off.cpu().numpy()
    for i, r in enumerate(results):
        if i % 2 == 0:
            same(r, R.weight_grad(fdy, fx, o), F32, f"two streams {i}")
        else:
            live = np.r_[tuple(slice(a, b) for _, a, b in R.groups(o, rows))]
            assert np.array_equal(f64(r)[live], R.forward(fx, fw, o, np.zeros((rows, out)))[live])


def test_same_result_every_time():
    print("experts repeated", flush=True)
    off = split_rows(3001, 7, 2)
    x, dy = tensor((3001, 513), F32, 1, whole=False), tensor((3001, 767), F32, 2, whole=False)
    first = mo.muon_experts_weight_grad(dy, x, off)
    for _ in range(3):
        assert torch.equal(first, mo.muon_experts_weight_grad(dy, x, off))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", [(300, 3, 3, 129), (300, 3, 129, 3), (500, 2, 1, 300), (500, 2, 300, 5), (400, 2, 8, 7),
                                   (400, 2, 7, 8), (5000, 3, 2, 2)])
def test_one_width_shorter_than_a_piece(shape, dtype):
    """One operand's rows are shorter than 16 bytes, the other's are not."""
    print("experts short rows", shape, dtype, flush=True)
    run_all(*shape, dtype, split_rows(shape[0], shape[1], 2, lead=1), 5, (1, 2, 3), (3, 2, 1), what=shape)
    run_all(*shape, dtype, split_rows(shape[0], shape[1], 2), 5, what=shape)


def test_sums_over_nothing_need_no_workspace():
    """No rows at all in the weight gradient (a rank that got no tokens), no inputs
    in the forward product, no outputs in the other, at sizes of large products."""
    print("experts sums over nothing", flush=True)
    d = dev()
    e, out, in_ = 40, 1408, 2048
    off = torch.zeros(e + 1, dtype=torch.int32, device=d)
    none = torch.empty(0, dtype=torch.uint8, device=d)
    for dt in (BF, F32):
        dw = torch.full((e, out, in_), 3.0, dtype=dt, device=d)
        dy, x = torch.empty(0, out, dtype=dt, device=d), torch.empty(0, in_, dtype=dt, device=d)
        mo.muon_experts_weight_grad(dy, x, off, dw=dw, accumulate=True)
        assert (dw == 3).all()
        mo.muon_experts_weight_grad(dy, x, off, dw=dw, workspace=none)
        assert not dw.any()
        rows = 9000
        off2 = split_rows(rows, e, 1)
        y = mo.muon_experts_forward(torch.empty(rows, 0, dtype=dt, device=d), torch.empty(e, out, 0, dtype=dt, device=d), off2)
        dx = mo.muon_experts_input_grad(torch.empty(rows, 0, dtype=dt, device=d), torch.empty(e, 0, in_, dtype=dt, device=d), off2)
        assert not y.any() and not dx.any()


@pytest.mark.parametrize("back", [(0, 40000, 0, 30000), (0, 30000, 10000, 40000, 5000, 39000), (39000, 40000, 0, 40000),
                                  (0, 20000, 15000, 40000)])
def test_offsets_that_go_back_in_a_large_product(back):
    """Groups that overlap, at sizes of the large products: whatever the results,
    nothing outside dw and the workspace is written, and the next call is right."""
    print("experts offsets back", back, flush=True)
    d = dev()
    rows, e, out, in_ = 40000, 30, 2560, 520
    gen = torch.Generator(device=d).manual_seed(1)
    whole = lambda *s: torch.randint(-3, 4, s, generator=gen, device=d).to(BF)
    x, w, dy = whole(rows, in_), whole(e, out, in_), whole(rows, out)
    n = [mo.muon_experts_workspace_bytes(k, rows, e, out, in_, mo.MUON_BF16) for k in range(3)]
    ws = [torch.full((b + 4096,), 91, dtype=torch.uint8, device=d) for b in n]
    guard = lambda r, c: torch.full((r + 2, c), 7.0, dtype=BF, device=d)
    y, dx, dw = guard(rows, out), guard(rows, in_), guard(e * out, in_)
    bad = torch.tensor(list(back) + [rows] * (e + 1 - len(back)), dtype=torch.int32, device=d)
    good = split_rows(rows, e, 3)
    for off in (bad, good):
        mo.muon_experts_forward(x, w, off, y=y[1:-1], workspace=ws[0][:n[0]])
        mo.muon_experts_weight_grad(dy, x, off, dw=dw[1:-1], workspace=ws[1][:n[1]])
        mo.muon_experts_input_grad(dy, w, off, dx=dx[1:-1], workspace=ws[2][:n[2]])
        torch.cuda.synchronize()
        for b, t in zip(n, ws):
            assert b > 0 and (t[b:] == 91).all(), b
        for t in (y, dx, dw):
            assert (t[0] == 7).all() and (t[-1] == 7).all()
    for g, a, b in R.groups(good.tolist(), rows):
        assert torch.equal(dw[1:-1].view(e, out, in_)[g], (dy[a:b].double().t().contiguous() @ x[a:b].double()).to(BF)), g
