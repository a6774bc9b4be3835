"""Products over packed rows and the 8-bit quantiser: argument checks that
need no GPU (the C ABI refuses before it enqueues anything; the binding refuses
tensors it cannot pass on)."""
import pytest

FAKE = 1 << 20  # 16-byte aligned, never dereferenced: validation fails first
F32, BF16, F16 = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    from two_sided_gptq_b200 import _native, build

    build.build()
    return _native.load()


@pytest.fixture(scope="module")
def status():
    from two_sided_gptq_b200._native import Status

    return Status


def changed(args, **by_name):
    d = dict(args)
    assert set(by_name) <= set(d), by_name
    d.update(by_name)
    return list(d.values())


QUANTIZE = dict(x=FAKE, x_type=F32, batch=1, rows=4, cols=130, x_batch=0, ldx=130, block_rows=1, q=FAKE, ldq=144,
                scales=FAKE, ws=FAKE, ws_bytes=256, stream=None)
BLOCKS = dict(x=FAKE, ldx=144, xs=FAKE, w=FAKE, ldw=144, w_stride=144 * 8, ws_=FAKE, scale_rows=128, offsets=FAKE,
              experts=3, y=FAKE, y_type=BF16, ldy=8, rows=5, n=8, k=130, ws=FAKE, ws_bytes=256, stream=None)
GROUPED = dict(x=FAKE, type=BF16, ldx=136, w=FAKE, ldw=136, w_stride=136 * 136, offsets=FAKE, experts=3, y=FAKE,
               y_type=BF16, ldy=136, rows=5, n=136, k=130, ws=FAKE, ws_bytes=256, stream=None)
DW = dict(dy=FAKE, type=F16, ldy=8, x=FAKE, ldx=136, offsets=FAKE, experts=3, dw=FAKE, dw_type=F16, rows=5, n=8, k=130,
          ws=FAKE, ws_bytes=256, stream=None)
GRAM = dict(x=FAKE, type=F16, ldx=136, offsets=FAKE, experts=3, damping=0.01, A=FAKE, rows=5, d=130, ws=FAKE,
            ws_bytes=1 << 20, stream=None)

INVALID = {
    "bakron_quantize_blocks": (QUANTIZE, [
        dict(x=None), dict(q=None), dict(scales=None), dict(x_type=3), dict(x_type=-1), dict(batch=-1), dict(rows=-1),
        dict(cols=0), dict(cols=(1 << 30) + 1, ldx=1 << 31, ldq=1 << 31), dict(ldx=129), dict(ldq=128),
        dict(block_rows=2), dict(block_rows=0), dict(x_batch=-1), dict(rows=1 << 30, batch=2)]),
    "bakron_matmul_blocks": (BLOCKS, [
        dict(x=None), dict(xs=None), dict(w=None), dict(ws_=None), dict(y=None), dict(offsets=None), dict(experts=0),
        dict(experts=1025), dict(offsets=FAKE + 2), dict(y_type=3), dict(scale_rows=64), dict(ldx=128), dict(ldw=128),
        dict(w_stride=144 * 8 - 16), dict(ldy=7), dict(rows=-1), dict(n=0), dict(k=0), dict(rows=(1 << 30) + 1),
        dict(rows=1 << 30, n=1 << 30, w_stride=144 << 30, ldy=1 << 30)]),
    "bakron_matmul_grouped": (GROUPED, [
        dict(x=None), dict(w=None), dict(y=None), dict(offsets=None), dict(experts=0), dict(experts=1025),
        dict(type=F32), dict(type=3), dict(y_type=F16), dict(ldx=128), dict(ldw=128), dict(w_stride=136 * 135),
        dict(ldy=135), dict(rows=-1), dict(n=0), dict(k=0), dict(offsets=FAKE + 1)]),
    "bakron_matmul_grouped_dx": (GROUPED, [
        dict(x=None), dict(w=None), dict(y=None), dict(offsets=None), dict(type=F32), dict(y_type=F16), dict(ldx=128),
        dict(ldw=128), dict(ldy=129), dict(experts=0)]),
    "bakron_matmul_grouped_dw": (DW, [
        dict(dy=None), dict(x=None), dict(dw=None), dict(offsets=None), dict(type=F32), dict(dw_type=BF16),
        dict(ldy=0), dict(ldx=128), dict(experts=0), dict(experts=1025), dict(rows=-1), dict(n=0), dict(k=0)]),
    "bakron_gram_grouped": (GRAM, [
        dict(x=None), dict(A=None), dict(offsets=None), dict(type=3), dict(ldx=128), dict(experts=0),
        dict(experts=1025), dict(damping=-0.5), dict(damping=float("nan")), dict(damping=float("inf")), dict(rows=-1),
        dict(d=0), dict(d=1 << 22, ldx=1 << 22)]),
}
MISALIGNED = {
    "bakron_quantize_blocks": (QUANTIZE, [dict(x=FAKE + 4), dict(q=FAKE + 8), dict(scales=FAKE + 4), dict(ldq=136),
                                          dict(ws=FAKE + 8)]),
    "bakron_matmul_blocks": (BLOCKS, [dict(x=FAKE + 8), dict(w=FAKE + 8), dict(ldx=136), dict(ldw=136),
                                      dict(y=FAKE + 2), dict(xs=FAKE + 4), dict(ws_=FAKE + 4),
                                      dict(w_stride=144 * 8 + 8)]),
    "bakron_matmul_grouped": (GROUPED, [dict(x=FAKE + 2), dict(w=FAKE + 2), dict(ldx=131), dict(ldw=132),
                                        dict(y=FAKE + 2), dict(w_stride=136 * 136 + 4)]),
    "bakron_matmul_grouped_dw": (DW, [dict(dy=FAKE + 2), dict(x=FAKE + 2), dict(ldy=9), dict(ldx=131),
                                      dict(dw=FAKE + 4)]),
    "bakron_gram_grouped": (GRAM, [dict(x=FAKE + 2), dict(ldx=131), dict(A=FAKE + 4)]),
}


@pytest.mark.parametrize("name", sorted(INVALID))
def test_invalid_arguments_are_refused(lib, status, name):
    args, bad = INVALID[name]
    for b in bad:
        assert getattr(lib, name)(*changed(args, **b)) == status.ERR_INVALID_ARG, b


@pytest.mark.parametrize("name", sorted(MISALIGNED))
def test_misaligned_operands_are_refused(lib, status, name):
    args, bad = MISALIGNED[name]
    for b in bad:
        got = getattr(lib, name)(*changed(args, **b))
        # the workspace is looked at last, where a machine without a GPU has
        # already failed to set the device up
        assert got == status.ERR_ALIGNMENT, b


def test_workspace_is_checked(lib, status):
    assert lib.bakron_quantize_blocks(*changed(QUANTIZE, ws=None)) == status.ERR_WORKSPACE
    assert lib.bakron_quantize_blocks(*changed(QUANTIZE, ws_bytes=255)) == status.ERR_WORKSPACE
    size = lib.bakron_gram_grouped_workspace_size
    assert size(F16, 100, 40) == 1024 and size(BF16, 0, 40) == 1024
    assert size(F32, 100, 41) == 1024 + -(-3 * 100 * 48 * 2 // 1024) * 1024
    assert size(3, 100, 40) == 0 and size(F32, -1, 40) == 0 and size(F32, 100, 0) == 0


def test_timeout_variable_is_checked(lib, status, monkeypatch):
    monkeypatch.setenv("BAKRON_TIMEOUT_MS", "soon")
    assert lib.bakron_quantize_blocks(*changed(QUANTIZE)) == status.ERR_INVALID_ARG


def test_binding_refuses_what_it_cannot_pass_on():
    import torch

    import two_sided_gptq_b200 as bk

    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    w = torch.zeros((2, 8, 64), dtype=torch.bfloat16)
    o = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(TypeError, match="x must be a CUDA tensor"):
        bk.quantize_blocks(x)
    with pytest.raises(TypeError, match="x must be a CUDA tensor"):
        bk.matmul_grouped(x, w, o)
    with pytest.raises(TypeError, match="dy must be a CUDA tensor"):
        bk.matmul_grouped_dx(x, w, o)
    with pytest.raises(TypeError, match="dy must be a CUDA tensor"):
        bk.matmul_grouped_dw(x, x, o)
    with pytest.raises(TypeError, match="X must be a CUDA tensor"):
        bk.gram_grouped(x, o)
    with pytest.raises(TypeError, match="x must be a CUDA tensor"):
        bk.matmul_blocks(x, x, x, x)
