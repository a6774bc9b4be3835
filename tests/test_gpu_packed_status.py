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
