"""What the packed-row products record about a call: the first error of the latest
call, in every call that has one."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def bk():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import two_sided_gptq_b200 as bk

    bk._lib()
    return bk


def rand(shape, seed, dtype=F32):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(dtype).cuda()


def bounds(o):
    return torch.tensor(o, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_the_first_error_is_reported(bk, dtype):
    """Bad bounds are found by the products, values that are not finite by the
    damping behind them."""
    x = rand((100, 72), 1, dtype)
    x[5, 7] = float("nan")
    ws = bk.workspace(1 << 20)
    for _ in range(2):
        bk.gram_grouped(x, bounds([0, 50, 40]), 0.01, ws=ws, check_status=False)
        assert bk.get_status(ws) == bk.Status.ERR_INVALID_ARG
        assert bk.get_status(ws) == bk.Status.OK  # reading clears all of it
        bk.gram_grouped(x, bounds([0, 50, 100]), 0.01, ws=ws, check_status=False)
        assert bk.get_status(ws) == bk.Status.ERR_NONFINITE
        bk.gram_grouped(x, bounds([10, 50, 100]), 0.01, ws=ws)


@pytest.mark.parametrize("name", ["blocks", "y", "dx", "dw", "gram"])
def test_no_report_of_bad_bounds_is_lost(bk, name):
    """Many calls of one or few blocks of threads, each with bad bounds, each on a
    status block of its own: the warp that reads the bounds and the thread that
    sets the block up do not wait for each other before."""
    calls = 3000
    x, dy, w = rand((10, 64), 1, BF16), rand((10, 40), 2, BF16), rand((2, 40, 64), 3, BF16)
    q, s = bk.quantize_blocks(x)
    wq, ws = bk.quantize_blocks(w, 128)
    O = bounds([0, 5, 11])
    f = {
        "blocks": lambda **kw: bk.matmul_blocks(q, s, wq, ws, O, **kw),
        "y": lambda **kw: bk.matmul_grouped(x, w, O, **kw),
        "dx": lambda **kw: bk.matmul_grouped_dx(dy, w, O, **kw),
        "dw": lambda **kw: bk.matmul_grouped_dw(dy, x, O, **kw),
        "gram": lambda **kw: bk.gram_grouped(x, O, **kw),
    }[name]
    spaces = torch.full((calls, 1024), 255, dtype=torch.uint8, device="cuda")
    out = f(ws=spaces[0], check_status=False)
    for i in range(calls):
        f(ws=spaces[i], out=out, check_status=False)
    torch.cuda.synchronize()
    blocks = spaces[:, :256].cpu()
    assert (blocks[:, :8] == 0).all()                       # no code, no place
    reports = blocks[:, 8:]
    assert ((reports == 0) | (reports == int(bk.Status.ERR_INVALID_ARG))).all()
    lost = (reports == 0).all(1).sum().item()
    assert lost == 0, f"{lost} of {calls}"
    # every CTA of a call reports it
    assert (reports == reports[0]).all()
