"""Row bounds that go back, on the GPU: groups that would share rows with an
earlier one count as empty in every product, whatever tiles they would make, and
the error is recorded.  Each call is compared, bit for bit, with a call of the same
sizes (and so of the same launch) on bounds that do not go back."""
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


def calls(bk, rows, n, k, experts):
    """name -> (function of offsets and out, result's shape, type, rows in the result's first dimension)"""
    x, dy, w = rand((rows, k), 1, BF16), rand((rows, n), 2, BF16), rand((experts, n, k), 3, BF16)
    q, s = bk.quantize_blocks(x)
    wq, ws = bk.quantize_blocks(w, 128)
    samples = rand((rows, n), 4)
    return {
        "blocks": (lambda o, **kw: bk.matmul_blocks(q, s, wq, ws, o, **kw), (rows, n), BF16, True),
        "y": (lambda o, **kw: bk.matmul_grouped(x, w, o, **kw), (rows, n), BF16, True),
        "dx": (lambda o, **kw: bk.matmul_grouped_dx(dy, w, o, **kw), (rows, k), BF16, True),
        "dw": (lambda o, **kw: bk.matmul_grouped_dw(dy, x, o, **kw), (experts, n, k), BF16, False),
        "gram": (lambda o, **kw: bk.gram_grouped(dy, o, 0.01, **kw), (experts, n, n), F32, False),
        "gram fp32": (lambda o, **kw: bk.gram_grouped(samples, o, 0.01, **kw), (experts, n, n), F32, False),
    }


def check(bk, rows, n, k, bad, good, lost):
    """`good`: bounds without the step back; `lost`: the groups that count as empty
    in `bad` but not in `good`."""
    for name, (f, shape, dtype, by_row) in calls(bk, rows, n, k, len(bad) - 1).items():
        ws, out = bk.workspace(1 << 24), torch.full(shape, 5.0, dtype=dtype, device="cuda")
        want = f(bounds(good), out=torch.full(shape, 5.0, dtype=dtype, device="cuda"))
        for e in lost:
            if by_row:
                want[good[e]:good[e + 1]] = 5.0
            else:
                want[e] = 0.0
        f(bounds(bad), out=out, ws=ws, check_status=False)
        assert bk.get_status(ws) == bk.Status.ERR_INVALID_ARG, name
        assert torch.equal(out, want), name
        f(bounds(good), out=out, ws=ws)  # the next call starts clean


def test_few_groups(bk):
    check(bk, 100, 136, 144, [0, 50, 40, 100], [0, 50, 50, 100], [2])
    check(bk, 100, 136, 144, [0, 50, 40, 45, 60, 100], [0, 50, 50, 50, 60, 100], [3])


@pytest.mark.parametrize("at", [1, 31, 32, 33, 60])
def test_many_groups(bk, at):
    """A step back at either side of the 32 groups that are numbered at a time."""
    good = list(range(0, 4 * 70 + 1, 4))
    bad = good[:at + 1] + [good[at] - 3] + good[at + 2:]
    good[at + 1] = good[at]
    check(bk, 285, 72, 136, bad, good, [at + 1])


# rows, n, k, bounds: calls with few tiles, whose contraction is shared by the CTAs
# of a cluster (8-bit and 16-bit operands), where each group's bounds alone would
# make more tiles than there are clusters
@pytest.mark.parametrize("rows,n,k,bad", [
    (300, 128, 4096, [0, 300, 0, 300]),
    (190, 128, 4096, [0, 190, 0, 190, 0, 190]),
    (190, 256, 128, [0, 190, 0, 190, 0, 190]),
    (1000, 128, 512, [0, 1000] * 11),
])
def test_more_tiles_than_launched(bk, rows, n, k, bad):
    check(bk, rows, n, k, bad, [0] + [rows] * (len(bad) - 1), [])
