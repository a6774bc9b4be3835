"""Argument checks of the packed-row products' self-test that need no GPU."""
import pytest


@pytest.fixture(scope="module")
def lib():
    from two_sided_gptq_b200 import _native, build

    build.build()
    return _native.load()


def test_rows_abort_refuses(lib):
    from two_sided_gptq_b200._native import Status

    fake = 1 << 20  # never dereferenced: validation fails first
    need = lib.bakron_selftest_rows_abort_workspace_size()
    assert need == 1024 + 2 * (256 * 512 + 256 * 2048 + 512 * 2048)
    call = lib.bakron_selftest_rows_abort
    assert call(0, 1, fake, need, None) == Status.ERR_INVALID_ARG
    assert call(10001, 1, fake, need, None) == Status.ERR_INVALID_ARG
    assert call(5, 0, fake, need, None) == Status.ERR_INVALID_ARG
    assert call(5, 3, fake, need, None) == Status.ERR_INVALID_ARG
    assert call(5, 1, None, need, None) == Status.ERR_WORKSPACE
    assert call(5, 1, fake, need - 1, None) == Status.ERR_WORKSPACE
    assert call(5, 2, fake + 8, need, None) == Status.ERR_ALIGNMENT
