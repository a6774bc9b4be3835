"""The time limit of the bounded waits is one of a pipeline step: a call that makes
progress ends well however long it takes.  The products whose contraction is the
packed rows, under a limit of one millisecond, with ragged groups that end several
milliseconds after the kernel begins.  Values are small whole numbers, so that sums
in any order are exact."""
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


def whole(shape, seed, dtype=BF16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-1, 2, shape, generator=g, device="cuda", dtype=torch.int8).to(dtype)


def bounds(lens):
    o = [0]
    for n in lens:
        o.append(o[-1] + n)
    return torch.tensor(o, dtype=torch.int32, device="cuda"), o


def product(a, b):
    """a^T b in fp32, exact (every partial sum is a whole number below 2^24), from
    pieces that keep the copies small."""
    return sum(a[i:i + 65536].float().T @ b[i:i + 65536].float() for i in range(0, len(a), 65536))


# the long group a multiple of 16 rows and the ragged one behind it; one long ragged
# group by tiles that several CTAs share
DW = [([131072, 33], 4096, 4096), ([4000007], 128, 128)]


@pytest.mark.parametrize("lens,n,k", DW)
def test_weight_gradients(bk, monkeypatch, lens, n, k):
    O, o = bounds(lens)
    dy, x = whole((o[-1], n), 1), whole((o[-1], k), 2)
    dw = bk.matmul_grouped_dw(dy, x, O, out_dtype=F32)
    for e in range(len(lens)):
        assert torch.equal(dw[e], product(dy[o[e]:o[e + 1]], x[o[e]:o[e + 1]]))
    monkeypatch.setenv("BAKRON_TIMEOUT_MS", "1")
    e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    e0.record()
    again = bk.matmul_grouped_dw(dy, x, O, out_dtype=F32, check_status=False)
    e1.record()
    torch.cuda.synchronize()
    assert e0.elapsed_time(e1) > 1.2  # long enough to say something
    assert torch.equal(again, dw)
    assert torch.equal(bk.matmul_grouped_dw(dy, x, O, out_dtype=F32), dw)


@pytest.mark.parametrize("dtype,lens,d", [(BF16, [196608, 33], 4096), (F32, [65536, 33], 4096), (BF16, [4000007], 128),
                                          (F32, [2000007], 128)])
def test_gram_factors(bk, monkeypatch, dtype, lens, d):
    O, o = bounds(lens)
    x = whole((o[-1], d), 3, dtype)
    A = bk.gram_grouped(x, O)
    for e, n in enumerate(lens):
        xe = x[o[e]:o[e + 1]]
        assert torch.equal(A[e], product(xe, xe) / torch.full((), n, dtype=F32, device="cuda"))
    monkeypatch.setenv("BAKRON_TIMEOUT_MS", "1")
    e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    e0.record()
    bk.gram_grouped(x, O, check_status=False)
    e1.record()
    torch.cuda.synchronize()
    assert e0.elapsed_time(e1) > 1.2
    assert torch.equal(bk.gram_grouped(x, O), A)
