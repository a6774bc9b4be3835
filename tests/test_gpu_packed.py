"""Products over packed rows and the 8-bit quantiser on the GPU against plain
64-bit forms, at the sizes and in the places where they can go wrong."""
import math

import pytest

import packed
from packed import check_close, offsets_of

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def bk():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import two_sided_gptq_b200 as bk

    bk._lib()
    return bk


def rand(shape, seed, dtype=F32, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype)


def rows_of(x, multiple):
    """On the GPU, with rows that start on 16-byte boundaries; what lies between
    the rows is NaN."""
    pad = -x.shape[-1] % multiple + multiple
    wide = torch.full(x.shape[:-1] + (x.shape[-1] + pad,), float("nan"), dtype=F32).to(x.dtype)
    wide[..., : x.shape[-1]] = x
    return wide.cuda()[..., : x.shape[-1]]


def bounds(o):
    return torch.tensor(o, dtype=torch.int32, device="cuda")


def poison(x, o, value=float("nan")):
    """The rows outside every group."""
    x[: o[0]] = value
    x[o[-1]:] = value
    return x


# ---------------------------------------------------------------- quantiser
QUANT_SHAPES = [(1, 1), (1, 128), (3, 129), (128, 128), (129, 7), (130, 1000), (300, 257), (257, 640)]


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("shape", QUANT_SHAPES)
def test_quantize_is_the_definition(bk, shape, block_rows, dtype):
    x = rand(shape, sum(shape) + block_rows)
    x *= torch.exp(3 * rand((shape[0], 1), 5))
    x[0, 0] = 0.0
    if shape[0] > 2:
        x[2] = 0.0  # a row (and, in blocks of rows, part of a block) of zeros
    if shape[0] > 100:
        x[100, : min(64, shape[1])] *= 2.0 ** -12  # values far below their block's step
    x = x.to(dtype)
    q, s = bk.quantize_blocks(x.cuda(), block_rows)
    want_q, want_s = packed.quantize(x, block_rows)
    assert q.dtype == E4M3 and q.shape == x.shape and q.stride(0) % 16 == 0
    assert torch.equal(s.double().cpu(), want_s)
    assert torch.equal(q.float().double().cpu(), want_q)


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_extremes(bk, block_rows):
    """Ties, subnormal steps, steps that underflow, the largest values."""
    ties = torch.tensor([448.0, 0.5 * 2 ** -9, 1.5 * 2 ** -9, 2.5 * 2 ** -9, 17.0, 19.0, 0.53125, -17.0, 0.0, -0.0,
                         2.0 ** -9, 432.0, 240.0, 1.0625])
    rows = torch.zeros((7, 128))
    rows[0, : len(ties)] = ties
    rows[1] = rows[0] * 2.0 ** -130          # a subnormal step
    rows[2, :3] = torch.tensor([2.0 ** -149, -(2.0 ** -148), 2.0 ** -140])  # a step of zero or one unit
    rows[3] = rows[0] * 2.0 ** 119           # close to the largest finite values
    rows[4, 5] = torch.finfo(F32).max
    rows[5] = rows[0] * 2.0 ** -70
    for r in range(7):
        x = rows[r: r + 1]
        q, s = bk.quantize_blocks(x.cuda(), block_rows)
        want_q, want_s = packed.quantize(x, block_rows)
        assert torch.equal(s.double().cpu(), want_s), r
        assert torch.equal(q.float().double().cpu(), want_q), r


def test_quantize_batches_strides_and_views(bk):
    x = rand((3, 200, 333), 4)
    wide = torch.full((3, 210, 400), float("nan"))
    wide[:, :200, :333] = x
    view = wide.cuda()[:, :200, :333]
    for block_rows in (1, 128):
        q, s = bk.quantize_blocks(view, block_rows)
        for e in range(3):
            want_q, want_s = packed.quantize(x[e], block_rows)
            assert torch.equal(s[e].double().cpu(), want_s)
            assert torch.equal(q[e].float().double().cpu(), want_q)
        # a view that starts off the vector loads' alignment grid
        y = wide.cuda()[1, 3:150, 8:301]
        q, s = bk.quantize_blocks(y[:, :290], block_rows)
        want_q, want_s = packed.quantize(wide[1, 3:150, 8:298], block_rows)
        assert torch.equal(s.double().cpu(), want_s) and torch.equal(q.float().double().cpu(), want_q)
    # bytes between the codes' columns and their row stride are left alone
    buf = torch.full((200, 352), 77, dtype=torch.uint8, device="cuda")
    codes = buf.view(E4M3)[:, :333]
    bk.quantize_blocks(view[0], 1, out=(codes, torch.empty((200, 3), device="cuda")))
    assert (buf[:, 333:] == 77).all()


def test_quantize_nothing_and_nonfinite(bk):
    q, s = bk.quantize_blocks(torch.zeros((0, 40), device="cuda"))
    assert q.shape == (0, 40) and s.shape == (0, 1)
    for block_rows in (1, 128):
        for bad in (float("nan"), float("inf"), -float("inf")):
            x = rand((150, 300), 1)
            x[140, 299] = bad
            with pytest.raises(bk.BakronError) as e:
                bk.quantize_blocks(x.cuda(), block_rows)
            assert e.value.status == bk.Status.ERR_NONFINITE
    bk.quantize_blocks(rand((150, 300), 1).cuda())  # the next call starts clean


@pytest.mark.parametrize("block_rows,few,many", [(1, (1984, 130), (1985, 130)), (1, (992, 1025), (993, 1025)),
                                                 (128, (260, 8000), (260, 10700)), (1, (1, 1), (70, 30000))])
def test_quantize_reports_from_any_block(bk, block_rows, few, many):
    """Grids of one, a few hundred and more blocks of threads on one workspace."""
    ws = bk.workspace(256).fill_(255)  # a fresh workspace holds anything
    for shape in (few, many, few):
        x = rand(shape, 1).cuda()
        q, s = bk.quantize_blocks(x, block_rows, ws=ws)
        want_q, want_s = packed.quantize(x.cpu(), block_rows)
        assert torch.equal(s.double().cpu(), want_s)
        assert torch.equal(q.float().double().cpu(), want_q)
        for at in {(0, 0), (shape[0] - 1, shape[1] - 1), (shape[0] // 2, shape[1] // 3)}:
            y = x.clone()
            y[at] = float("nan")
            with pytest.raises(bk.BakronError) as e:
                bk.quantize_blocks(y, block_rows, ws=ws)
            assert e.value.status == bk.Status.ERR_NONFINITE
            assert bk.get_status(ws) == bk.Status.OK
            bk.quantize_blocks(y, block_rows, ws=ws, check_status=False)
            bk.quantize_blocks(x, block_rows, ws=ws)  # the next call starts clean


# ------------------------------------------------------------ 8-bit products
def eight(rows, k, seed):
    """Codes over the whole range, steps over several powers of two."""
    g = torch.Generator().manual_seed(seed)
    q = torch.randn((rows, k), generator=g) * 100
    q = q.clamp(-448, 448).to(E4M3)
    s = torch.exp(torch.randn((rows, -(-k // 128)), generator=g)) * 0.01
    return q, s


def weights(n, k, per_row, seed):
    g = torch.Generator().manual_seed(seed)
    if per_row:
        return torch.randint(-7, 8, (n, k), generator=g).float().to(E4M3), torch.rand(n, generator=g) * 0.01 + 1e-3
    q = (torch.randn((n, k), generator=g) * 100).clamp(-448, 448).to(E4M3)
    return q, torch.rand((-(-n // 128), -(-k // 128)), generator=g) * 0.01 + 1e-4


def blocks_reference(x, xs, w, ws):
    k, n = x.shape[1], w.shape[0]
    a = x.float().double() * packed.spread(xs, k)
    steps = ws.double()[:, None] if ws.dim() == 1 else packed.spread(ws, k).repeat_interleave(128, 0)[:n]
    b = w.float().double() * steps
    a, b = a.cuda(), b.cuda()
    return (a @ b.T).cpu(), (a.abs() @ b.abs().T).cpu()


def rows8(x):
    pad = -x.shape[-1] % 16 + 16
    wide = torch.full(x.shape[:-1] + (x.shape[-1] + pad,), 0x7F, dtype=torch.uint8)  # NaN codes between the rows
    wide[..., : x.shape[-1]] = x.view(torch.uint8)
    return wide.cuda().view(E4M3)[..., : x.shape[-1]]


@pytest.mark.parametrize("per_row", [False, True])
@pytest.mark.parametrize("out", [BF16, F16, F32])
@pytest.mark.parametrize("rows,n,k", [(1, 1, 1), (1, 128, 128), (2, 130, 300), (16, 257, 129), (17, 1000, 640),
                                      (64, 384, 2000), (65, 300, 256), (127, 100, 1000), (129, 513, 384),
                                      (300, 260, 4096), (1, 4096, 4096), (33, 640, 11008), (700, 1024, 512)])
def test_matmul_blocks(bk, rows, n, k, out, per_row):
    x, xs = eight(rows, k, rows + k)
    w, ws = weights(n, k, per_row, n + k)
    if out == F16:
        ws = ws * 0.01  # results inside the type's range
    want, size = blocks_reference(x, xs, w, ws)
    got = bk.matmul_blocks(rows8(x), xs.cuda(), rows8(w), ws.cuda(), out_dtype=out)
    check_close(got.cpu(), want, size, k, 4, 128, f"blocks {rows}x{n}x{k} {out}")


GROUPS = [
    ([5], 0, 0), ([0, 0, 0], 2, 3), ([1, 0, 17, 64, 0, 33], 0, 9), ([130, 1, 0, 256, 300], 3, 40),
    ([1] * 40, 0, 0), ([0] * 63 + [70], 0, 1), ([128, 128, 257], 0, 0), ([600, 2], 0, 0),
]


@pytest.mark.parametrize("n,k", [(200, 136), (257, 1000), (128, 128)])
@pytest.mark.parametrize("lens,lead,tail", GROUPS)
@pytest.mark.parametrize("per_row", [False, True])
def test_matmul_blocks_grouped(bk, lens, lead, tail, n, k, per_row):
    o = offsets_of(lens, lead)
    rows = o[-1] + tail
    x, xs = eight(rows, k, rows + k)
    xs = poison(xs, o)
    xb = x.view(torch.uint8)
    x = poison(xb, o, 0x7F).view(E4M3)
    w, ws = zip(*[weights(n, k, per_row, 31 * e + n) for e in range(len(lens))])
    keep = torch.full((rows, n), 3.25, dtype=BF16, device="cuda")
    got = bk.matmul_blocks(rows8(x), xs.cuda(), rows8(torch.stack(w)), torch.stack(ws).cuda(), bounds(o), out=keep)
    assert got is keep
    assert (got[: o[0]] == 3.25).all() and (got[o[-1]:] == 3.25).all()
    for e, n_e in enumerate(lens):
        if n_e:
            a, b = o[e], o[e + 1]
            want, size = blocks_reference(x[a:b], xs[a:b], w[e], ws[e])
            check_close(got[a:b].cpu(), want, size, k, 4, 128, f"expert {e}")


@pytest.mark.parametrize("per_row", [False, True])
@pytest.mark.parametrize("rows,n,k", [(1500, 5000, 300), (300, 4100, 520), (100, 130, 1100), (200, 260, 900),
                                      (2100, 1030, 130), (50, 1000, 2000), (520, 3000, 1300)])
def test_matmul_blocks_every_tile_shape(bk, rows, n, k, per_row):
    """Sizes that reach the 256 x 256, 256 x 128 and 128 x 128 tiles, whole and
    split along the contraction, with ragged edges and uneven parts."""
    x, xs = eight(rows, k, rows + k)
    w, ws = weights(n, k, per_row, n + k)
    want, size = blocks_reference(x, xs, w, ws)
    y = bk.matmul_blocks(rows8(x), xs.cuda(), rows8(w), ws.cuda(), out_dtype=F32)
    check_close(y.cpu(), want, size, k, 4, 128, f"blocks {rows}x{n}x{k}")
    y = bk.matmul_blocks(rows8(x), xs.cuda(), rows8(w), ws.cuda())
    check_close(y.cpu(), want, size, k, 4, 128, f"blocks {rows}x{n}x{k} bf16")


def test_matmul_blocks_grouped_large(bk):
    lens, n, k = [700, 0, 1900, 33], 3000, 400
    o = offsets_of(lens, 5)
    rows = o[-1] + 6
    x, xs = eight(rows, k, 1)
    w, ws = zip(*[weights(n, k, False, e) for e in range(len(lens))])
    y = torch.full((rows, n), 3.25, dtype=F32, device="cuda")
    bk.matmul_blocks(rows8(x), poison(xs, o).cuda(), rows8(torch.stack(w)), torch.stack(ws).cuda(), bounds(o), out=y)
    assert (y[: o[0]] == 3.25).all() and (y[o[-1]:] == 3.25).all()
    for e, n_e in enumerate(lens):
        if n_e:
            a, b = o[e], o[e + 1]
            want, size = blocks_reference(x[a:b], xs[a:b], w[e], ws[e])
            check_close(y[a:b].cpu(), want, size, k, 4, 128, f"expert {e}")


def test_matmul_blocks_of_solver_codes(bk):
    """The solver's codes and steps as an 8-bit operand: the product with V."""
    import oracle
    import workloads

    m, n = 200, 264
    W, A, B = workloads.random_problem(m, n, seed=3)
    LA, LB = bk.factor(torch.from_numpy(A).cuda(), torch.from_numpy(B).cuda())
    for bits in (2, 3, 4, 5):
        V, codes, scales = bk.solve(torch.from_numpy(W).cuda(), LA, LB, bits=bits)
        w = codes.float().to(E4M3)
        assert torch.equal(w.float(), codes.float())
        x = rand((37, n), bits)
        q, s = bk.quantize_blocks(x.cuda())
        y = bk.matmul_blocks(q, s, rows8(w.cpu()), scales, out_dtype=F32)
        a = q.float().double() * packed.spread(s, n)
        want, size = a @ V.double().T, a.abs() @ V.double().abs().T
        # V is the fp32 product of code and step: half a unit more per term
        check_close(y.cpu(), want.cpu(), size.cpu(), n, 5, 128, f"codes of {bits} bits")


# ----------------------------------------------------- products by expert
NK = [(1, 1), (7, 9), (130, 72), (257, 1000), (64, 384)]


@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (F16, F16), (BF16, F32), (F16, F32)])
@pytest.mark.parametrize("n,k", NK)
@pytest.mark.parametrize("lens,lead,tail", GROUPS)
def test_matmul_grouped_and_gradients(bk, lens, lead, tail, n, k, dtype, out):
    o = offsets_of(lens, lead)
    rows = o[-1] + tail
    x = poison(rand((rows, k), 1 + k, dtype), o)
    dy = poison(rand((rows, n), 2 + n, dtype), o, float("inf"))
    w = rand((len(lens), n, k), 3, dtype)
    X, DY, W, O = rows_of(x, 8), rows_of(dy, 8), rows_of(w, 8), bounds(o)
    mark = lambda *shape: torch.full(shape, 3.25, dtype=out, device="cuda")  # noqa: E731
    y = bk.matmul_grouped(X, W, O, out=mark(rows, n))
    dx = bk.matmul_grouped_dx(DY, W, O, out=mark(rows, k))
    dw = bk.matmul_grouped_dw(DY, X, O, out=mark(len(lens), n, k))
    for t in (y, dx):
        assert (t[: o[0]] == 3.25).all() and (t[o[-1]:] == 3.25).all()
    y, dx, dw = y.cpu(), dx.cpu(), dw.cpu()
    for e, n_e in enumerate(lens):
        a, b = o[e], o[e + 1]
        xe, de, we = x[a:b].double(), dy[a:b].double(), w[e].double()
        if n_e:
            check_close(y[a:b], xe @ we.T, xe.abs() @ we.abs().T, k, 16, 256, f"y {e}")
            check_close(dx[a:b], de @ we, de.abs() @ we.abs(), n, 16, 256, f"dx {e}")
            check_close(dw[e], de.T @ xe, de.abs().T @ xe.abs(), n_e, 16, 256, f"dw {e}")
        else:
            assert (dw[e] == 0).all()


@pytest.mark.parametrize("rows,experts,n,k", [(1000, 3, 1024, 2048), (3000, 2, 520, 4096), (40, 8, 2048, 1024)])
def test_matmul_grouped_larger(bk, rows, experts, n, k):
    g = torch.Generator().manual_seed(rows)
    cuts = sorted(torch.randint(0, rows + 1, (experts - 1,), generator=g).tolist())
    o = [0] + cuts + [rows]
    x, dy, w = rand((rows, k), 1, BF16).cuda(), rand((rows, n), 2, BF16).cuda(), rand((experts, n, k), 3, BF16).cuda()
    O = bounds(o)
    y, dx = bk.matmul_grouped(x, w, O, out_dtype=F32), bk.matmul_grouped_dx(dy, w, O, out_dtype=F32)
    dw = bk.matmul_grouped_dw(dy, x, O, out_dtype=F32)
    for e in range(experts):
        a, b = o[e], o[e + 1]
        xe, de, we = x[a:b].double(), dy[a:b].double(), w[e].double()
        check_close(y[a:b], xe @ we.T, xe.abs() @ we.abs().T, k, 16, 256, f"y {e}")
        check_close(dx[a:b], de @ we, de.abs() @ we.abs(), n, 16, 256, f"dx {e}")
        check_close(dw[e], de.T @ xe, de.abs().T @ xe.abs(), b - a, 16, 256, f"dw {e}")


def test_gradients_are_those_of_the_product(bk):
    """Differences of L = sum(y * c) along random directions against <dx, .> and
    <dw, .>: L is linear in each operand, so the difference of two values is the
    derivative, up to the roundings of the three results (fp32 here)."""
    lens, n, k = [70, 0, 33, 200], 96, 160
    o = offsets_of(lens)
    rows = o[-1]
    x, w = rand((rows, k), 1, BF16).cuda(), rand((4, n, k), 2, BF16).cuda()
    c, O = rand((rows, n), 3, BF16).cuda(), bounds(o)
    dx = bk.matmul_grouped_dx(c, w, O, out_dtype=F32).double()
    dw = bk.matmul_grouped_dw(c, x, O, out_dtype=F32).double()
    loss = lambda x, w: (bk.matmul_grouped(x, w, O, out_dtype=F32).double() * c.double()).sum()  # noqa: E731
    vx, vw = rand((rows, k), 4, BF16).cuda(), rand((4, n, k), 5, BF16).cuda()
    x2, w2 = (x.float() + vx.float()).to(BF16), (w.float() + vw.float()).to(BF16)
    # the steps actually taken, in bf16, are exact differences in fp32
    hx, hw = x2.double() - x.double(), w2.double() - w.double()
    base = loss(x, w)
    size = (c.double().abs() * 40 * math.sqrt(k)).sum().item()
    tol = 30 * 2.0 ** -23 * size
    assert abs((loss(x2, w) - base - (dx * hx).sum()).item()) <= tol
    assert abs((loss(x, w2) - base - (dw * hw).sum()).item()) <= tol


@pytest.mark.parametrize("experts", [129, 1024])
def test_many_experts(bk, experts):
    """More experts than tiles are fitted to, most of them short or empty."""
    g = torch.Generator().manual_seed(experts)
    lens = torch.randint(0, 4, (experts,), generator=g).tolist()
    lens[experts // 2] = 150
    o = offsets_of(lens, 1)
    rows, n, k = o[-1] + 2, 40, 72
    x, dy = poison(rand((rows, k), 1, BF16), o).cuda(), poison(rand((rows, n), 2, BF16), o).cuda()
    w, O = rand((experts, n, k), 3, BF16).cuda(), bounds(o)
    e = torch.repeat_interleave(torch.arange(experts), torch.tensor(lens)).cuda()
    a, b = o[0], o[-1]
    xd, dd, wd = x[a:b].double(), dy[a:b].double(), w.double()[e]
    y, dx = bk.matmul_grouped(x, w, O), bk.matmul_grouped_dx(dy, w, O)
    check_close(y[a:b], torch.einsum("tk,tnk->tn", xd, wd), torch.einsum("tk,tnk->tn", xd.abs(), wd.abs()), k, 16, 256, "y")
    check_close(dx[a:b], torch.einsum("tn,tnk->tk", dd, wd), torch.einsum("tn,tnk->tk", dd.abs(), wd.abs()), n, 16, 256,
                "dx")
    outer = lambda p, q: torch.zeros((experts, p.shape[1], q.shape[1]), dtype=torch.float64, device="cuda").index_add_(  # noqa: E731
        0, e, p[:, :, None] * q[:, None])
    dw = bk.matmul_grouped_dw(dy, x, O, out_dtype=F32)
    check_close(dw, outer(dd, xd), outer(dd.abs(), xd.abs()), 150, 16, 256, "dw")
    count = torch.tensor(lens, dtype=torch.float64, device="cuda").clamp(min=1)[:, None, None]
    A = bk.gram_grouped(x, O)
    check_close(A, outer(xd, xd) / count, outer(xd.abs(), xd.abs()) / count, 150, 18, 128, "gram")


def test_results_beyond_32_bit_offsets(bk):
    """Operands and results of more than 2^31 elements, looked at behind there."""
    rows, n, k = 70001, 32768, 24
    x, w = rand((rows, k), 1, BF16).cuda(), rand((2, n, k), 2, BF16).cuda()
    y = bk.matmul_grouped(x, w, bounds([0, 69000, rows]))
    assert y.numel() > 2 ** 31
    for a, b, e in ((0, 70, 0), (68950, 69000, 0), (69000, 69050, 1), (rows - 60, rows, 1)):
        xe, we = x[a:b].double(), w[e].double()
        check_close(y[a:b], xe @ we.T, xe.abs() @ we.abs().T, k, 16, 256, f"y {a}")
    # y is now the operand: its last rows lie beyond 2^31 elements
    dx = bk.matmul_grouped_dx(y, w, bounds([0, 69000, rows]), out_dtype=F32)
    for a, b, e in ((0, 40, 0), (rows - 40, rows, 1)):
        de, we = y[a:b].double(), w[e].double()
        check_close(dx[a:b], de @ we, de.abs() @ we.abs(), n, 16, 512, f"dx {a}")
    q, s = bk.quantize_blocks(y)
    for a in (0, rows - 3):
        want_q, want_s = packed.quantize(y[a:a + 3].cpu(), 1)
        assert torch.equal(s[a:a + 3].double().cpu(), want_s)
        assert torch.equal(q[a:a + 3].float().double().cpu(), want_q)
    q128, s128 = bk.quantize_blocks(y, 128)
    last = rows // 128 * 128
    want_q, want_s = packed.quantize(y[last:, :256].cpu(), 128)
    assert torch.equal(s128[-1:, :2].double().cpu(), want_s)
    assert torch.equal(q128[last:, :256].float().double().cpu(), want_q)
    del q128, dx
    wq, ws = bk.quantize_blocks(rand((96, n), 5, F32).cuda(), 128)
    z = bk.matmul_blocks(q, s, wq, ws, out_dtype=F32)
    a = rows - 30
    xe = q[a:].float().double() * packed.spread(s[a:], n)
    we = wq.float().double() * packed.spread(ws, n)[:1]
    check_close(z[a:], xe @ we.T, xe.abs() @ we.abs().T, n, 4, 128, "blocks")
    del y, q, z
    experts, d = 33, 8192
    v = rand((2 * experts, d), 7, BF16).cuda()
    O = bounds(list(range(0, 2 * experts + 1, 2)))
    dw = bk.matmul_grouped_dw(v, v, O)
    assert dw.numel() > 2 ** 31
    last = v[-2:].double()
    check_close(dw[-1], last.T @ last, last.abs().T @ last.abs(), 2, 16, 256, "dw")
    del dw
    A = bk.gram_grouped(v, O, check_status=False)
    check_close(A[-1], last.T @ last / 2, last.abs().T @ last.abs() / 2, 2, 18, 128, "gram")


# --------------------------------------------------------------- Gram factors
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("d", [1, 9, 128, 130, 300, 520])
@pytest.mark.parametrize("lens,lead,tail", GROUPS)
def test_gram_grouped(bk, lens, lead, tail, d, dtype):
    o = offsets_of(lens, lead)
    rows = o[-1] + tail
    x = rand((rows, d), d)
    x *= torch.exp(rand((1, d), 8))
    x = poison(x.to(dtype), o)
    A = bk.gram_grouped(rows_of(x, 8), bounds(o), 0.01).cpu()
    assert torch.equal(A, A.transpose(1, 2))
    for e, n_e in enumerate(lens):
        if not n_e:
            assert (A[e] == 0).all()
            continue
        xe = x[o[e]:o[e + 1]].double()
        G = xe.T @ xe / n_e
        add = 0.01 * G.diagonal().mean()
        size = xe.abs().T @ xe.abs() / n_e
        # three bf16 parts: the dropped products are below 2^-24 of their own
        check_close(A[e], G + add * torch.eye(d, dtype=torch.float64), size + add * torch.eye(d), n_e, 18, 128,
                    f"gram {e}")


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("lens,lead,tail,n,k", [
    ([4099], 0, 0, 130, 72),             # one or a few tiles: eight CTAs share each
    ([1, 3001, 0, 79], 3, 5, 200, 131),  # ... with groups shorter than the parts
    ([5, 517, 1030], 0, 9, 1300, 257),   # fewer CTAs per tile
    ([700, 3, 1411, 260, 0, 517, 90, 333, 1601], 1, 7, 1003, 1130),  # tiles of CTA pairs
])
def test_contractions_over_rows(bk, lens, lead, tail, n, k, dtype):
    """dw and Gram factors by every tile shape and split, results with odd rows."""
    o = offsets_of(lens, lead)
    rows = o[-1] + tail
    x = poison((rand((rows, k), k) * torch.exp(rand((1, k), 8))).to(dtype), o)
    X, O = rows_of(x, 8), bounds(o)
    A = bk.gram_grouped(X, O)
    assert torch.equal(A, A.transpose(1, 2)) and torch.equal(A, bk.gram_grouped(X, O))
    if dtype != F32:
        dy = poison(rand((rows, n), n, dtype), o)
        D = rows_of(dy, 8)
        dw = {t: bk.matmul_grouped_dw(D, X, O, out_dtype=t) for t in (dtype, F32)}
        assert torch.equal(dw[F32], bk.matmul_grouped_dw(D, X, O, out_dtype=F32))
    for e, n_e in enumerate(lens):
        if not n_e:
            assert (A[e] == 0).all()
            continue
        xe = x[o[e]:o[e + 1]].cuda().double()
        check_close(A[e], xe.T @ xe / n_e, xe.abs().T @ xe.abs() / n_e, n_e, 18, 128, f"gram {e}")
        if dtype == F32:
            continue
        de = dy[o[e]:o[e + 1]].cuda().double()
        for t in dw:
            check_close(dw[t][e], de.T @ xe, de.abs().T @ xe.abs(), n_e, 16, 256, f"dw {e} {t}")


def test_gram_grouped_is_gram_for_one_group(bk):
    x = rand((1000, 300), 2).cuda()
    A, one = bk.gram_grouped(x, bounds([0, 1000]), 0.01)[0], bk.gram(x, 0.01)
    scale = one.diagonal().max()
    assert ((A - one).abs().max() / scale).item() < 2e-6  # both to fp32; gram's parts keep 21 bits


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_gram_grouped_nonfinite(bk, dtype):
    x = rand((60, 140), 3, dtype)
    O = bounds([0, 20, 50])
    for bad in (float("nan"), float("inf")):
        for row, col, hit in ((49, 139, True), (0, 0, True), (55, 3, False)):
            y = x.clone()
            y[row, col] = bad
            Y = rows_of(y, 8)
            if hit:
                with pytest.raises(bk.BakronError) as e:
                    bk.gram_grouped(Y, O)
                assert e.value.status == bk.Status.ERR_NONFINITE
            else:
                bk.gram_grouped(Y, O)


# ---------------------------------------------------- what all of them share
def calls(bk, rows=100, n=136, k=144, experts=3, dtype=BF16):
    """Every entry point on one packed problem: name -> function of offsets and out."""
    x, dy, w = rand((rows, k), 1, dtype).cuda(), rand((rows, n), 2, dtype).cuda(), rand((experts, n, k), 3, dtype).cuda()
    q, s = bk.quantize_blocks(x)
    wq, ws = bk.quantize_blocks(w, 128)
    return {
        "blocks": (lambda o, **kw: bk.matmul_blocks(q, s, wq, ws, o, **kw), (rows, n), BF16),
        "y": (lambda o, **kw: bk.matmul_grouped(x, w, o, **kw), (rows, n), dtype),
        "dx": (lambda o, **kw: bk.matmul_grouped_dx(dy, w, o, **kw), (rows, k), dtype),
        "dw": (lambda o, **kw: bk.matmul_grouped_dw(dy, x, o, **kw), (experts, n, k), dtype),
        "gram": (lambda o, **kw: bk.gram_grouped(x, o, **kw), (experts, k, k), F32),
        "gram fp32": (lambda o, **kw: bk.gram_grouped(x.float(), o, **kw), (experts, k, k), F32),
    }


@pytest.mark.parametrize("bad", [[0, 50, 40, 100], [0, 10, 20, 101], [-1, 10, 20, 30], [2 ** 31 - 1, 0, 5, 9],
                                 [0, 10, -(2 ** 31), 20]])
def test_bad_offsets_are_reported(bk, bad):
    for name, (f, _, _) in calls(bk).items():
        with pytest.raises(bk.BakronError) as e:
            f(bounds(bad))
        assert e.value.status == bk.Status.ERR_INVALID_ARG, name
        f(bounds([0, 10, 20, 100]))  # the next call starts clean


def test_no_rows(bk):
    x = torch.empty((0, 64), dtype=BF16, device="cuda")
    w, O = rand((2, 40, 64), 1, BF16).cuda(), bounds([0, 0, 0])
    assert bk.matmul_grouped(x, w, O).shape == (0, 40)
    dy = torch.empty((0, 40), dtype=BF16, device="cuda")
    assert bk.matmul_grouped_dx(dy, w, O).shape == (0, 64)
    assert (bk.matmul_grouped_dw(dy, x, O) == 0).all()
    for t in (F32, BF16):
        A = bk.gram_grouped(x.to(t), O, 0.01)
        assert A.shape == (2, 64, 64) and (A == 0).all()
    q, s = bk.quantize_blocks(x)
    wq, ws = bk.quantize_blocks(w, 128)
    assert bk.matmul_blocks(q, s, wq, ws, O).shape == (0, 40)
    assert bk.matmul_blocks(q, s, wq[0], ws[0]).shape == (0, 40)


def test_results_of_any_stride(bk):
    """Rows of the result at any element offset, neighbours untouched."""
    O = bounds([0, 30, 30, 97])
    for name, (f, shape, dtype) in calls(bk).items():
        if name in ("dw", "gram", "gram fp32"):
            continue
        plain = f(O, out=torch.full(shape, 5.0, dtype=dtype, device="cuda"))
        wide = torch.full((shape[0], shape[1] + 3), 5.0, dtype=dtype, device="cuda")
        got = f(O, out=wide[:, : shape[1]])
        assert torch.equal(got, plain), name
        assert (wide[:, shape[1]:] == 5.0).all(), name


def test_equal_calls_give_equal_bits_and_streams_are_followed(bk):
    O = bounds([0, 30, 30, 97])
    side = torch.cuda.Stream()
    for name, (f, shape, dtype) in calls(bk).items():
        fill = lambda: torch.full(shape, 5.0, dtype=dtype, device="cuda")  # noqa: E731
        first = f(O, out=fill())
        for _ in range(3):
            assert torch.equal(f(O, out=fill()), first), name
        out = fill()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            f(O, out=out)
        assert torch.equal(out, first), name
        out = fill()
        side.wait_stream(torch.cuda.current_stream())
        f(O, out=out, stream=side)
        assert torch.equal(out, first), name


def test_calls_on_two_streams_at_once(bk):
    """Split and whole contractions of two streams share the device."""
    a, b = calls(bk, rows=3000, n=200, k=264), calls(bk, rows=700, n=1104, k=1032)
    for p, x in ((a, rand((3000, 264), 4).cuda()), (b, rand((700, 1032), 5).cuda())):
        p["gram fp32"] = (lambda o, x=x, **kw: bk.gram_grouped(x, o, **kw), p["gram fp32"][1], F32)
    oa, ob = bounds([0, 1000, 1010, 3000]), bounds([0, 30, 400, 700])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for name in a:
        sides = [(p[name][0], o, p[name][1], p[name][2]) for p, o in ((a, oa), (b, ob))]
        want = [f(o) for f, o, _, _ in sides]
        outs = [[torch.zeros(shape, dtype=t, device="cuda") for _ in range(8)] for _, _, shape, t in sides]
        spaces = [bk.workspace(2 ** 25) for _ in sides]
        torch.cuda.synchronize()
        for i in range(8):
            for (f, o, _, _), out, ws, stream in zip(sides, outs, spaces, streams):
                f(o, out=out[i], ws=ws, stream=stream, check_status=False)
        for ws, stream in zip(spaces, streams):
            assert bk.get_status(ws, stream) == bk.Status.OK
        torch.cuda.synchronize()
        for out, w in zip(outs, want):
            assert all(torch.equal(y, w) for y in out), name


def test_what_a_call_allocates_belongs_to_its_stream(bk, monkeypatch):
    made, plain = [], bk.workspace
    monkeypatch.setattr(bk, "workspace", lambda *a: made.append(torch.cuda.current_stream()) or plain(*a))
    O, side = bounds([0, 30, 30, 97]), torch.cuda.Stream()
    problems = calls(bk, rows=1000, n=2056, k=2064)
    for name, (f, shape, dtype) in problems.items():
        made.clear()
        side.wait_stream(torch.cuda.current_stream())
        y = f(O, stream=side, check_status=False)
        assert made == [side], name
        side.synchronize()
        at = y.untyped_storage().data_ptr()
        del y
        assert torch.empty(shape, dtype=dtype, device="cuda").data_ptr() != at, name
    made.clear()
    bk.quantize_blocks(torch.ones((100, 100), device="cuda"), stream=side)
    assert made == [side]


def test_captured_calls_replay_with_other_offsets(bk):
    a, b = [0, 30, 30, 97], [2, 2, 60, 99]
    for name, (f, shape, dtype) in calls(bk).items():
        O, out = bounds(a), torch.full(shape, 5.0, dtype=dtype, device="cuda")
        want = {tuple(o): f(bounds(o), out=torch.full(shape, 5.0, dtype=dtype, device="cuda")) for o in (a, b)}
        ws = bk.workspace(1 << 20)
        f(O, out=out, ws=ws, check_status=False)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            f(O, out=out, ws=ws, check_status=False)
        for o in (b, a, b):
            O.copy_(bounds(o))
            out.fill_(5.0)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want[tuple(o)]), name
            assert bk.get_status(ws) == bk.Status.OK


def test_refusals(bk):
    x, w, O = rand((20, 64), 1, BF16).cuda(), rand((2, 40, 64), 2, BF16).cuda(), bounds([0, 5, 20])
    q, s = bk.quantize_blocks(x)
    wq, ws = bk.quantize_blocks(w, 128)
    with pytest.raises(TypeError):
        bk.matmul_grouped(x.float(), w.float(), O)
    with pytest.raises(TypeError):
        bk.matmul_grouped(x, w.half(), O)
    with pytest.raises(TypeError):
        bk.matmul_grouped(x, w, O.long())
    with pytest.raises(TypeError):
        bk.matmul_grouped(x, w, O.cpu())
    with pytest.raises(TypeError):
        bk.matmul_grouped(x, w, O, out_dtype=F16)
    with pytest.raises(ValueError):
        bk.matmul_grouped(x, w, bounds([0, 5, 20, 20]))
    with pytest.raises(ValueError):
        bk.matmul_grouped(x[:, :32], w, O)
    with pytest.raises(ValueError):
        bk.matmul_grouped(x.T.contiguous().T, w, O)
    with pytest.raises(ValueError):
        bk.matmul_grouped(x, w, O, out=torch.empty((20, 41), dtype=BF16, device="cuda"))
    with pytest.raises(ValueError):
        bk.matmul_grouped_dw(x, x[:10], O)
    with pytest.raises(ValueError):
        bk.matmul_blocks(q, s, wq, ws[:1], O)
    with pytest.raises(ValueError):
        bk.matmul_blocks(q, s, wq[0], ws[0].T.contiguous().T[:, :0])
    with pytest.raises(TypeError):
        bk.matmul_blocks(q, s, wq, ws)  # experts without offsets
    for f in (lambda: bk.matmul_grouped(x[:, 4:], w[:, :, 4:], O),  # rows off the 16-byte grid
              lambda: bk.matmul_grouped(rand((20, 61), 1, BF16).cuda(), rand((2, 40, 61), 1, BF16).cuda(), O),
              lambda: bk.gram_grouped(rand((20, 61), 1, BF16).cuda(), O)):
        with pytest.raises(bk.BakronError) as e:
            f()
        assert e.value.status == bk.Status.ERR_ALIGNMENT
    with pytest.raises(bk.BakronError) as e:
        bk.matmul_grouped(x[:1].expand(20, 64), w, O)  # a broadcast operand
    assert e.value.status == bk.Status.ERR_INVALID_ARG
    with pytest.raises(bk.BakronError) as e:
        bk.gram_grouped(x, O, -1.0)
    assert e.value.status == bk.Status.ERR_INVALID_ARG
    with pytest.raises(bk.BakronError) as e:
        bk.gram_grouped(x.float(), O, ws=bk.workspace(256))
    assert e.value.status == bk.Status.ERR_WORKSPACE
    with pytest.raises(bk.BakronError) as e:
        bk.quantize_blocks(x, 64)
    assert e.value.status == bk.Status.ERR_INVALID_ARG


# ------------------------------------------------------------ used together
def test_experts_from_samples_to_products(bk):
    """A layer of experts: packed samples -> factors per expert -> rounding ->
    products with the rounded experts, in 16 bits (V) and in 8 (codes)."""
    import oracle

    experts, n, k = 3, 136, 160
    lens = [700, 640, 900]
    o = offsets_of(lens)
    rows = o[-1]
    x, dy, w = rand((rows, k), 1, BF16), rand((rows, n), 2, BF16), rand((experts, n, k), 3, F32, 0.02)
    x = (x.float() * torch.exp(0.5 * rand((1, k), 4))).to(BF16)
    X, DY, O, W = x.cuda(), dy.cuda(), bounds(o), w.cuda()
    A, B = bk.gram_grouped(X, O, 0.01), bk.gram_grouped(DY, O, 0.01)
    problems = []
    for e in range(experts):
        LA, LB = bk.factor(A[e].contiguous(), B[e].contiguous())
        problems.append((W[e].contiguous(), LA, LB))
    solved = bk.solve_batch(problems, bits=4, streams=[torch.cuda.current_stream()])
    V = torch.stack([s[0] for s in solved])
    codes, steps = torch.stack([s[1] for s in solved]), torch.stack([s[2] for s in solved])
    for e in range(experts):
        loss = bk.proxy_loss(W[e].contiguous(), V[e].contiguous(), A[e].contiguous(), B[e].contiguous())
        near = torch.round(W[e] / steps[e][:, None]).clamp(-7, 7) * steps[e][:, None]
        E = (W[e] - near).double()
        rtn = torch.trace(E.T @ B[e].double() @ E @ A[e].double()).item()
        assert loss < rtn  # adaptive rounding beats the nearest codes on the same samples
    y16 = bk.matmul_grouped(X, V.to(BF16), O, out_dtype=F32)
    q, s = bk.quantize_blocks(X)
    y8 = bk.matmul_blocks(q, s, codes.float().to(E4M3), steps, O, out_dtype=F32)
    for e in range(experts):
        a, b = o[e], o[e + 1]
        v16 = V[e].to(BF16).double()
        xe = X[a:b].double()
        check_close(y16[a:b].cpu(), (xe @ v16.T).cpu(), (xe.abs() @ v16.abs().T).cpu(), k, 16, 256, f"16 bits {e}")
        xq = q[a:b].float().double() * packed.spread(s[a:b], k)
        v = codes[e].double() * steps[e].double()[:, None]
        check_close(y8[a:b].cpu(), (xq @ v.T).cpu(), (xq.abs() @ v.abs().T).cpu(), k, 4, 128, f"8 bits {e}")
        # an e4m3 code is off by at most 2^-4 of its value (2^-10 of its block's
        # largest below the smallest normal code), so the 8-bit product is that
        # close to the exact one
        most = packed.spread(s[a:b], k) * 448
        slack = (xe.abs() * 2.0 ** -4 + most * 2.0 ** -18) @ v.abs().T
        assert ((y8[a:b].double() - xe @ v.T).abs() <= slack * (1 + 2.0 ** -12)).all()
