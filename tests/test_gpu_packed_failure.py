"""Failure detection of the packed-row products, without a fault: a wait that
counts as run out in one warp ends the call with BAKRON_ERR_DEVICE_TIMEOUT and
leaves the context usable."""
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


def bounds(o):
    return torch.tensor(o, dtype=torch.int32, device="cuda")


def check_product(bk, ws):
    """A product by CTA pairs on the same workspace: whole numbers below 2^24, so
    that any order of sums is exact."""
    g = torch.Generator().manual_seed(1)
    x = torch.randint(-8, 9, (700, 320), generator=g).to(BF16).cuda()
    w = torch.randint(-8, 9, (2, 264, 320), generator=g).to(BF16).cuda()
    y = bk.matmul_grouped(x, w, bounds([0, 300, 700]), out_dtype=F32, ws=ws)
    want = torch.cat([x[:300].float() @ w[0].float().T, x[300:].float() @ w[1].float().T])
    assert torch.equal(y, want)
    bk.matmul_grouped(x, w, bounds([0, 300, 700]), ws=ws)


@pytest.mark.parametrize("timeout_ms", [20, 5])
def test_one_warp_gives_up(bk, timeout_ms):
    """The four warps of a column half store together: when one has given up, none
    of them waits for it."""
    e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    ws = None
    for _ in range(3):
        e0.record()
        ws = bk.selftest_rows_abort(timeout_ms, ws)
        e1.record()
        assert bk.get_status(ws) == bk.Status.ERR_DEVICE_TIMEOUT
        assert bk.get_status(ws) == bk.Status.OK
        assert e0.elapsed_time(e1) < 500
        y = ws[1024: 1024 + 256 * 512 * 2].view(torch.int16).view(256, 512)
        assert (y[:128, :128] == -1).all()                # the half that gave up stored nothing
        assert ((y == -1) | (y == 0)).all()               # the others what they had
        assert (y[:, 128:256] == 0).all()                 # (the other CTA's first tile was complete)
        check_product(bk, ws)


def test_epilogue_gives_up_while_the_last_products_run(bk):
    """Tensor memory is released only once every issued matrix instruction has
    finished, also where nobody is left to read its result."""
    ws = None
    for _ in range(5):
        ws = bk.selftest_rows_abort(20, ws, way=2)
        torch.cuda.synchronize()
        assert ws[4:8].view(torch.int32).item() == 1
        assert bk.get_status(ws) == bk.Status.ERR_DEVICE_TIMEOUT
        y = ws[1024: 1024 + 256 * 512 * 2].view(torch.int16).view(256, 512)
        assert (y[:, :128] == -1).all() and (y[:, 128:256] == 0).all() and (y[:, 256:] == -1).all()
        check_product(bk, ws)
