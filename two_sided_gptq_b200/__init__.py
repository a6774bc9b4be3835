"""B200-native BaKron two-sided adaptive-rounding solver (Python binding).

Thin marshalling layer over the C ABI in ``include/bakron.h``: every step of
the computation runs in the library's CUDA kernels.  PyTorch supplies device
memory and streams only.

    LA, LB = factor(A, B)                       # chol(A^-1), chol(B^-1), FP64 inside
    V, codes, scales = solve(W, LA, LB, bits=4) # BaKron (Algorithm 6)
    loss = proxy_loss(W, V, A, B)               # tr((W-V)^T B (W-V) A)

Method: "BaKron: Efficient Quantization with Kronecker-Factored Hessians"
(arXiv 2608.06291).
"""
from __future__ import annotations

import ctypes
import functools

from . import _native
from ._native import BakronError, BatchItem, Config, PlanStats, Profile, ProfileLaunch, Quantizer, Status, check

__all__ = ["factor", "solve", "solve_host", "proxy_loss", "plan_stats", "last_profile",
           "last_profile_launches", "tune_leaf", "tune_cache_key", "tune_cache_get", "tune_cache_put",
           "solve_batch", "gram", "gram_grouped", "quantize_blocks", "matmul_blocks", "matmul_grouped",
           "matmul_grouped_dx", "matmul_grouped_dw", "selftest_wait_timeout", "selftest_band_abort",
           "selftest_rows_abort", "workspace", "get_status", "BakronError", "Status", "version", "library_path"]


# bakron_config_t.leaf values bakron_tune_leaf times (one ms_out entry each)
LEAF_STRUCTURES = (1, 2, 3, 4, 5, 6, 7, 8)


def _lib():
    return _native.load()


def library_path() -> str:
    return _native.LIB_PATH


def version() -> str:
    return _lib().bakron_version().decode()


def _torch():
    import torch

    return torch


def _ptr(t) -> int:
    return t.data_ptr() if t is not None else 0


def _stream(stream):
    torch = _torch()
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _dev_f32(x, name):
    torch = _torch()
    if not isinstance(x, torch.Tensor) or not x.is_cuda or x.dtype != torch.float32 or not x.is_contiguous():
        raise TypeError(f"{name} must be a contiguous float32 CUDA tensor")
    return x


def _config(gemm=0, timeout_ms=0, wt_out=None, profile=False, leaf=0, b_identity=False, graph=False, fuse_width=0,
            self_test_omit=0):
    return Config(0, int(gemm), 1 if graph else 0, int(timeout_ms), _ptr(wt_out), 1 if profile else 0, int(leaf),
                  1 if b_identity else 0, int(fuse_width), int(self_test_omit))


def workspace(nbytes: int, device=None):
    """A device byte buffer usable as a workspace (torch owns the memory)."""
    torch = _torch()
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device or "cuda")


def get_status(ws, stream=None) -> Status:
    """Synchronise and return (and clear) the device status recorded in ``ws``."""
    return Status(_lib().bakron_get_status(_ptr(ws), ws.numel(), _stream(stream)))


def selftest_wait_timeout(timeout_ms: int, ws, stream=None) -> None:
    """Launch the bounded-wait self-test (``bakron_selftest_wait_timeout``): a
    device wait that nothing completes gives up after ``timeout_ms`` and records
    ``Status.ERR_DEVICE_TIMEOUT`` in ``ws``; read it with :func:`get_status`."""
    check(_lib().bakron_selftest_wait_timeout(int(timeout_ms), _ptr(ws), ws.numel(), _stream(stream)),
          "bakron_selftest_wait_timeout")


def selftest_band_abort(timeout_ms: int, ws=None, stream=None):
    """Launch the band kernel's abort-path self-test (``bakron_selftest_band_abort``):
    the stage-1 band kernel with no copies issued, whose bounded waits run out
    after ``timeout_ms``.  Returns the workspace; its status word then reads
    ``Status.ERR_DEVICE_TIMEOUT`` (read it with :func:`get_status`)."""
    need = _lib().bakron_selftest_band_abort_workspace_size()
    if ws is None:
        ws = workspace(need)
    check(_lib().bakron_selftest_band_abort(int(timeout_ms), _ptr(ws), ws.numel(), _stream(stream)),
          "bakron_selftest_band_abort")
    return ws


def selftest_rows_abort(timeout_ms: int, ws=None, *, way=1, stream=None):
    """Launch the packed-row products' abort-path self-test
    (``bakron_selftest_rows_abort``): a product in which one epilogue warp's wait
    counts as run out and its neighbours' do not (``way`` 1), or in which the
    epilogue gives up while the last matrix instructions run (2).  Returns the
    workspace; its status then reads ``Status.ERR_DEVICE_TIMEOUT`` (read it with
    :func:`get_status`)."""
    need = _lib().bakron_selftest_rows_abort_workspace_size()
    if ws is None:
        ws = workspace(need)
    check(_lib().bakron_selftest_rows_abort(int(timeout_ms), int(way), _ptr(ws), ws.numel(), _stream(stream)),
          "bakron_selftest_rows_abort")
    return ws


def factor(A, B=None, *, stream=None, ws=None, check_status=True):
    """``(LA, LB)`` with ``LA LA^T = A^{-1}``, ``LB LB^T = B^{-1}`` (lower, fp32)."""
    torch = _torch()
    lib = _lib()
    n = 0 if A is None else A.shape[0]
    m = 0 if B is None else B.shape[0]
    if A is not None:
        _dev_f32(A, "A")
    if B is not None:
        _dev_f32(B, "B")
    dev = (A if A is not None else B).device
    LA = torch.empty((n, n), dtype=torch.float32, device=dev) if n else None
    LB = torch.empty((m, m), dtype=torch.float32, device=dev) if m else None
    need = lib.bakron_factor_workspace_size(n, m)
    if ws is None:
        ws = workspace(need, dev)
    st = _stream(stream)
    check(lib.bakron_factor(_ptr(A), n, _ptr(B), m, _ptr(LA), _ptr(LB), _ptr(ws), ws.numel(), st), "bakron_factor")
    if check_status:
        check(lib.bakron_get_status(_ptr(ws), ws.numel(), st), "bakron_factor (device)")
    return LA, LB


def solve_workspace_size(m: int, n: int, gemm: int = 0) -> int:
    return int(_lib().bakron_solve_workspace_size(m, n, ctypes.byref(_config(gemm))))


def solve(W, LA, LB, bits=4, *, qmin=0, qmax=0, row_scale=None, gemm=0, ws=None, out=None, stream=None,
          wt_out=None, check_status=True, timeout_ms=0, profile=False, leaf=0, shrink_grid=0, graph=False,
          fuse_width=0, self_test_omit=0):
    """BaKron solve on device tensors.  Returns ``(V, codes, scales)``.

    ``LB=None`` selects the one-sided path (B = I: GPTQ with Hessian A, over
    128-column blocks).

    ``gemm=0`` uses the tcgen05 3xTF32 band products, ``gemm=1`` the FP32
    CUDA-core ones; ``shrink_grid`` > 1 searches each row's step for the least
    round-to-nearest error over that many shrink factors in [1/2, 1]; ``leaf``
    selects the leaf sweep structure (0 default (6),
    1 two-level CTA-wide, 2 single-level, 3 three warps per 32 x 32
    sub-tile, 4 six warps per 64 x 64 sub-tile, 5 as 3 with each tile on a
    cluster of four CTAs, 6 as 5 with the older product terms formed during
    the sweeps, 7 as 6 with two tile diagonals per launch (device flags, the
    width-2 nodes' updates inside the leaf), 8 continuous strip sweeps, one
    per CTA, staggered by 48 steps; :func:`tune_leaf` picks one by
    measurement).  ``self_test_omit`` is a self-test hook of structure 7.  ``fuse_width`` (0 default, 1 never) runs the two band
    products of recursion nodes at most that many tile diagonals wide as one
    launch per target tile.  ``graph=True`` captures the solve's launches for this
    argument set into a CUDA graph on the first call and replays it on later
    calls with the same buffers.  ``out`` may supply ``(V, codes, scales)`` buffers and
    ``ws`` a workspace; ``check_status=False`` skips the synchronising status
    read (for timing).
    """
    torch = _torch()
    lib = _lib()
    one_sided = LB is None
    _dev_f32(W, "W"), _dev_f32(LA, "LA")
    if not one_sided:
        _dev_f32(LB, "LB")
    m, n = W.shape
    if LA.shape != (n, n) or (not one_sided and LB.shape != (m, m)):
        raise ValueError("LA must be n x n and LB m x m")
    cfg = _config(gemm, timeout_ms, wt_out, profile, leaf, one_sided, graph, fuse_width, self_test_omit)
    if out is None:
        V = torch.empty((m, n), dtype=torch.float32, device=W.device)
        codes = torch.empty((m, n), dtype=torch.int8, device=W.device)
        scales = torch.empty((m,), dtype=torch.float32, device=W.device)
    else:
        V, codes, scales = out
    if ws is None:
        ws = workspace(lib.bakron_solve_workspace_size(m, n, ctypes.byref(cfg)), W.device)
    q = Quantizer(int(bits), int(qmin), int(qmax), _ptr(row_scale), int(shrink_grid))
    st = _stream(stream)
    check(lib.bakron_solve(_ptr(W), m, n, _ptr(LA), _ptr(LB), ctypes.byref(q), _ptr(V), _ptr(codes), _ptr(scales),
                           _ptr(ws), ws.numel(), ctypes.byref(cfg), st), "bakron_solve")
    if check_status:
        check(lib.bakron_get_status(_ptr(ws), ws.numel(), st), "bakron_solve (device)")
    return V, codes, scales


def tune_cache_key(m: int, n: int, bits: int, device_name: str) -> str:
    """Key of a leaf-structure measurement in the autotune cache (the library
    version is part of it: a new build re-measures)."""
    return f"{int(m)}x{int(n)}/int{int(bits)}/{device_name}/{version()}"


def tune_cache_get(path: str, key: str):
    """``(leaf, ms_list)`` stored under ``key`` in the JSON file ``path``, or None."""
    import json
    import os

    if not path or not os.path.exists(path):
        return None
    try:
        with open(path) as f:
            entry = json.load(f).get(key)
    except (OSError, ValueError):
        return None
    if not isinstance(entry, dict) or entry.get("leaf") not in LEAF_STRUCTURES:
        return None
    return int(entry["leaf"]), [float(x) for x in entry.get("ms", [])]


def tune_cache_put(path: str, key: str, leaf: int, ms) -> None:
    """Store a measurement under ``key`` in the JSON file ``path`` (written to a
    temporary file and renamed, so readers never see a partial file)."""
    import json
    import os
    import tempfile

    data = {}
    if os.path.exists(path):
        try:
            with open(path) as f:
                data = json.load(f)
        except (OSError, ValueError):
            data = {}
    data[key] = {"leaf": int(leaf), "ms": [float(x) for x in ms]}
    d = os.path.dirname(os.path.abspath(path))
    fd, tmp = tempfile.mkstemp(dir=d, prefix=".bakron_tune_")
    with os.fdopen(fd, "w") as f:
        json.dump(data, f, indent=1, sort_keys=True)
    os.replace(tmp, path)


def tune_leaf(W, LA, LB, bits=4, *, ws=None, out=None, stream=None, gemm=0, timeout_ms=0, cache=None):
    """Leaf structure chosen by measurement (``bakron_tune_leaf``): one timed
    solve per structure on this problem.  Returns ``(leaf, [ms_leaf1, ...,
    ms_leaf8])``; pass ``leaf`` to :func:`solve`.

    ``cache`` (or the ``BAKRON_TUNE_CACHE`` environment variable) names a JSON
    file keyed by (m, n, bits, GPU name): a stored measurement is returned
    without timing, a new one is stored."""
    import os

    torch = _torch()
    lib = _lib()
    _dev_f32(W, "W"), _dev_f32(LA, "LA"), _dev_f32(LB, "LB")
    m, n = W.shape
    cache = cache or os.environ.get("BAKRON_TUNE_CACHE")
    key = tune_cache_key(m, n, bits, torch.cuda.get_device_name(W.device)) if cache else None
    if cache:
        hit = tune_cache_get(cache, key)
        if hit is not None:
            return hit
    cfg = _config(gemm, timeout_ms)
    if out is None:
        out = (torch.empty((m, n), dtype=torch.float32, device=W.device),
               torch.empty((m, n), dtype=torch.int8, device=W.device),
               torch.empty((m,), dtype=torch.float32, device=W.device))
    V, codes, scales = out
    if ws is None:
        ws = workspace(lib.bakron_solve_workspace_size(m, n, ctypes.byref(cfg)), W.device)
    q = Quantizer(int(bits), 0, 0, None)
    leaf = ctypes.c_int32(0)
    ms = (ctypes.c_double * len(LEAF_STRUCTURES))()
    st = _stream(stream)
    check(lib.bakron_tune_leaf(_ptr(W), m, n, _ptr(LA), _ptr(LB), ctypes.byref(q), _ptr(V), _ptr(codes),
                               _ptr(scales), _ptr(ws), ws.numel(), ctypes.byref(cfg), st, ctypes.byref(leaf), ms),
          "bakron_tune_leaf")
    check(lib.bakron_get_status(_ptr(ws), ws.numel(), st), "bakron_tune_leaf (device)")
    result = int(leaf.value), [float(x) for x in ms]
    if cache:
        tune_cache_put(cache, key, *result)
    return result


def solve_batch(problems, bits=4, *, streams, outs=None, workspaces=None, gemm=0, leaf=0, shrink_grid=0,
                check_status=True, fuse_width=0):
    """Independent solves through ``bakron_solve_batch``: ``problems`` is a list
    of ``(W, LA, LB)`` device tensors, solve i runs on ``streams[i %
    len(streams)]`` (torch streams).  ``outs`` / ``workspaces`` may supply the
    ``(V, codes, scales)`` buffers and workspaces.  Returns the list of
    ``(V, codes, scales)``."""
    torch = _torch()
    lib = _lib()
    cfg = _config(gemm, leaf=leaf, fuse_width=fuse_width)
    items = (BatchItem * max(1, len(problems)))()
    res, wss = [], []
    for i, (W, LA, LB) in enumerate(problems):
        _dev_f32(W, "W"), _dev_f32(LA, "LA"), _dev_f32(LB, "LB")
        m, n = W.shape
        if outs is None:
            o = (torch.empty((m, n), dtype=torch.float32, device=W.device),
                 torch.empty((m, n), dtype=torch.int8, device=W.device),
                 torch.empty((m,), dtype=torch.float32, device=W.device))
        else:
            o = outs[i]
        ws = workspaces[i] if workspaces is not None else workspace(
            lib.bakron_solve_workspace_size(m, n, ctypes.byref(cfg)), W.device)
        items[i] = BatchItem(_ptr(W), m, n, _ptr(LA), _ptr(LB), _ptr(o[0]), _ptr(o[1]), _ptr(o[2]), _ptr(ws),
                             ws.numel())
        res.append(o)
        wss.append(ws)
    st = (ctypes.c_void_p * len(streams))(*[s.cuda_stream for s in streams])
    q = Quantizer(int(bits), 0, 0, None, int(shrink_grid))
    check(lib.bakron_solve_batch(items, len(problems), ctypes.byref(q), ctypes.byref(cfg), st, len(streams)),
          "bakron_solve_batch")
    if check_status:
        for i, ws in enumerate(wss):
            check(lib.bakron_get_status(_ptr(ws), ws.numel(), _stream(streams[i % len(streams)])),
                  f"bakron_solve_batch item {i} (device)")
    return res


def gram(X, damping=0.0, *, ws=None, out=None, stream=None, check_status=True):
    """Kronecker factor ``X^T X / N + damping * mean(diag) * I`` from samples
    ``X`` (N x d device tensor) on the tensor cores (``bakron_gram``)."""
    torch = _torch()
    lib = _lib()
    _dev_f32(X, "X")
    N, d = X.shape
    A = torch.empty((d, d), dtype=torch.float32, device=X.device) if out is None else out
    if ws is None:
        ws = workspace(lib.bakron_gram_workspace_size(N, d), X.device)
    st = _stream(stream)
    check(lib.bakron_gram(_ptr(X), N, d, float(damping), _ptr(A), _ptr(ws), ws.numel(), st), "bakron_gram")
    if check_status:
        check(lib.bakron_get_status(_ptr(ws), ws.numel(), st), "bakron_gram (device)")
    return A


# ------------------------------------------------- products over packed rows
STATUS_BYTES = 256  # workspace of the calls below that need no more than the status block

# set by the first _device(): torch dtype -> bakron_type_t, the types that the
# calls take, torch's binding module
_type_ids = _eight = _single = _half = _bytes = _offset = _raw_module = None


def _device():
    """The current device's index (asked once per call, through torch's binding
    module: the checks of a small product would otherwise cost more than it)."""
    global _type_ids, _eight, _single, _half, _bytes, _offset, _raw_module
    if _raw_module is None:
        torch = _torch()
        _type_ids = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
        _eight, _single, _half = (torch.float8_e4m3fn,), (torch.float32,), (torch.bfloat16, torch.float16)
        _bytes, _offset = torch.uint8, (torch.int32,)
        if not torch.cuda.is_available():
            return None  # no tensor is on it
        _raw_module = torch._C
    return _raw_module._cuda_getDevice()


def _on_stream(call):
    """Takes the call's ``stream``, which is the current one during it: what the call
    allocates then belongs to that stream, and the next user of a freed
    workspace's memory comes after the call's kernels."""
    @functools.wraps(call)
    def run(*args, stream=None, **kw):
        if stream is None:
            return call(*args, **kw)
        with _torch().cuda.stream(stream):
            return call(*args, **kw)
    return run


def _here(t, name, dims, dtypes, dev):
    """A CUDA tensor on device ``dev`` with unit stride along its last dimension."""
    try:
        stride = t.stride()
        if (t.dtype in dtypes and len(stride) in dims and t.get_device() == dev
                and (stride[-1] == 1 or t.shape[-1] <= 1)):
            return
    except AttributeError:
        pass
    torch = _torch()
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype not in dtypes or t.dim() not in dims:
        raise TypeError(f"{name} must be a CUDA tensor of {' or '.join(map(str, dims))} dimensions and type "
                        f"{', '.join(str(d) for d in dtypes)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, not on the current device")
    raise ValueError(f"{name} must have unit stride along its last dimension")


def _ld(t, dim, least, align):
    """Row (or matrix) stride of a dimension; any will do where it has one entry."""
    return t.stride(dim) if t.shape[dim] > 1 else -(-least // align) * align


def _groups(offsets, dev, experts=None):
    _here(offsets, "offsets", (1,), _offset, dev)
    n = offsets.shape[0]
    if n < 2 or (experts is not None and n != experts + 1):
        raise ValueError("offsets must hold one bound more than there are experts")
    return n - 1


def _result(out, shape, dtype, allowed, dev):
    """The result tensor: ``out``, or a new one of ``dtype``."""
    if out is None:
        if dtype not in allowed:
            raise TypeError(f"out_dtype must be one of {', '.join(str(d) for d in allowed)}")
        torch = _torch()
        return torch.empty(shape, dtype=dtype, device=torch.device("cuda", dev))
    _here(out, "out", (len(shape),), allowed, dev)
    if out.shape != shape or (dtype is not None and out.dtype != dtype):
        raise ValueError(f"out must have shape {shape}" + (f" and type {dtype}" if dtype is not None else ""))
    return out


def _call(name, args, ws, check_status, dev, need=STATUS_BYTES):
    """One library call on a workspace: ``ws``, or a new one."""
    if ws is None:
        ws = workspace(need, dev)
    elif ws.get_device() != dev or ws.dtype != _bytes or not ws.is_contiguous():
        raise ValueError("ws must be a contiguous uint8 tensor on the current device")
    lib, at, size = _native._lib or _lib(), ws.data_ptr(), ws.numel()
    st = _raw_module._cuda_getCurrentRawStream(dev)
    status = getattr(lib, name)(*args, at, size, st)
    if status:
        check(status, name)
    if check_status:
        check(lib.bakron_get_status(at, size, st), name + " (device)")


@_on_stream
def quantize_blocks(x, block_rows=1, *, out=None, ws=None, stream=None, check_status=True):
    """8-bit floating point codes of ``x`` (rows x cols, or batch x rows x cols;
    float32, bfloat16 or float16) with one float32 step per block of
    ``block_rows`` x 128 values, ``block_rows`` 1 or 128
    (``bakron_quantize_blocks``): ``x ~= codes * step``.

    Returns ``(codes, scales)``: ``codes`` float8_e4m3fn of x's shape, with rows
    that start on 16-byte boundaries as :func:`matmul_blocks` wants them (a view
    of a wider buffer for odd widths), ``scales`` of shape ``[..., ceil(rows /
    block_rows), ceil(cols / 128)]``.  ``out`` may supply both."""
    torch = _torch()
    dev = _device()
    _here(x, "x", (2, 3), _type_ids, dev)
    rows, cols = x.shape[-2:]
    batch = x.shape[0] if x.dim() == 3 else 1
    lead = tuple(x.shape[:-2])
    steps = lead + (-(-rows // block_rows) if block_rows in (1, 128) else rows, -(-cols // 128))
    if out is None:
        wide = -(-cols // 16) * 16
        strides = (wide, 1) if not lead else (rows * wide, wide, 1)
        q = torch.empty_strided(x.shape, strides, dtype=torch.float8_e4m3fn, device=x.device)
        scales = torch.empty(steps, dtype=torch.float32, device=x.device)
    else:
        q, scales = out
        _here(q, "codes", (x.dim(),), (torch.float8_e4m3fn,), dev)
        _here(scales, "scales", (x.dim(),), (torch.float32,), dev)
        if q.shape != x.shape or scales.shape != steps or not scales.is_contiguous():
            raise ValueError(f"codes must have shape {tuple(x.shape)}, scales {steps} (contiguous)")
    ldq = _ld(q, -2, cols, 16)
    if x.dim() == 3 and batch > 1 and rows and q.stride(0) != rows * ldq:
        raise ValueError("codes must hold its matrices one directly after another")
    ldx = _ld(x, -2, cols, 1)
    _call("bakron_quantize_blocks",
          (x.data_ptr(), _type_ids[x.dtype], batch, rows, cols, x.stride(0) if batch > 1 else 0, ldx, block_rows,
           q.data_ptr(), ldq, scales.data_ptr()), ws, check_status, dev)
    return q, scales


@_on_stream
def matmul_blocks(x, x_scales, w, w_scales, offsets=None, *, out_dtype=None, out=None, ws=None, stream=None,
                  check_status=True):
    """``y = (x * steps) (w * steps)^T`` of 8-bit (float8_e4m3fn) operands
    (``bakron_matmul_blocks``), accumulated in float32.

    ``x`` rows x k with ``x_scales`` rows x ceil(k/128), as
    :func:`quantize_blocks` gives them; ``w`` n x k with ``w_scales`` either
    ceil(n/128) x ceil(k/128), or of shape (n,): one step per row, as
    :func:`solve` returns them (its codes of up to 5 bits are e4m3 values:
    ``codes.float().to(torch.float8_e4m3fn)``).  With ``offsets`` (int32,
    experts + 1 row bounds on the device) ``w`` is experts x n x k, the steps
    have the same leading dimension, and rows ``offsets[e] .. offsets[e+1] - 1``
    are multiplied by ``w[e]``; rows outside every group keep what ``out`` holds
    (unspecified in a new result).  Result: rows x n, bfloat16 unless
    ``out_dtype`` or ``out`` says float16 or float32."""
    dev = _device()
    lead = 0 if offsets is None else 1
    f8, f32 = _eight, _single
    _here(x, "x", (2,), f8, dev), _here(x_scales, "x_scales", (2,), f32, dev)
    _here(w, "w", (2 + lead,), f8, dev), _here(w_scales, "w_scales", (1 + lead, 2 + lead), f32, dev)
    rows, k = x.shape
    kblocks = (k + 127) // 128
    if lead:
        experts, n, kw = w.shape
        _groups(offsets, dev, experts)
        stride, at = w.stride(), offsets.data_ptr()
    else:
        n, kw = w.shape
        experts, stride, at = 1, (0,) + w.stride(), 0
    given = w_scales.shape
    per_row = len(given) == 1 + lead
    if (kw != k or x_scales.shape != (rows, kblocks) or given[lead:] != ((n,) if per_row else ((n + 127) // 128, kblocks))
            or (lead and given[0] != experts)):
        raise ValueError("x is rows x k with steps rows x ceil(k/128); w is n x k with steps ceil(n/128) x "
                         "ceil(k/128) or (n,), under one leading dimension when offsets are given")
    if not x_scales.is_contiguous() or not w_scales.is_contiguous():
        raise ValueError("x_scales and w_scales must be contiguous")
    types = _type_ids
    y = _result(out, (rows, n), out_dtype if out is not None or out_dtype is not None else _torch().bfloat16, types, dev)
    wide = (k + 15) // 16 * 16  # a stride that will do where there is one row
    ldw = stride[1] if n > 1 else wide
    _call("bakron_matmul_blocks",
          (x.data_ptr(), x.stride(0) if rows > 1 else wide, x_scales.data_ptr(), w.data_ptr(), ldw,
           stride[0] if experts > 1 else (n * ldw + 15) // 16 * 16, w_scales.data_ptr(), 1 if per_row else 128, at,
           experts, y.data_ptr(), types[y.dtype], y.stride(0) if rows > 1 else n, rows, n, k), ws, check_status,
          dev)
    return y


def _grouped(name, x, w, offsets, across, out_dtype, out, ws, check_status):
    dev = _device()
    _here(x, "x" if across == 2 else "dy", (2,), _half, dev)
    dtype = x.dtype
    _here(w, "w", (3,), (dtype,), dev)
    experts, n, k = w.shape
    _groups(offsets, dev, experts)
    rows, into = x.shape
    if into != (k if across == 2 else n):
        raise ValueError(f"{'x' if across == 2 else 'dy'} must have {k if across == 2 else n} columns")
    width = n if across == 2 else k
    if out is None and out_dtype is None:
        out_dtype = dtype
    y = _result(out, (rows, width), out_dtype, (dtype,) + _single, dev)
    ldw = _ld(w, 1, k, 8)
    _call(name, (x.data_ptr(), _type_ids[dtype], _ld(x, 0, into, 8), w.data_ptr(), ldw,
                 w.stride(0) if experts > 1 else n * ldw, offsets.data_ptr(), experts, y.data_ptr(),
                 _type_ids[y.dtype], _ld(y, 0, width, 1), rows, n, k), ws, check_status, dev)
    return y


@_on_stream
def matmul_grouped(x, w, offsets, *, out_dtype=None, out=None, ws=None, stream=None, check_status=True):
    """``y[t] = x[t] w[e]^T`` for the packed rows ``t`` of every expert e
    (``bakron_matmul_grouped``): ``x`` rows x k, ``w`` experts x n x k, both
    bfloat16 or float16, ``offsets`` int32 with experts + 1 row bounds on the
    device.  Sums in float32; ``y`` rows x n of x's type or float32.  Rows
    outside every group keep what ``out`` holds (unspecified in a new result)."""
    return _grouped("bakron_matmul_grouped", x, w, offsets, 2, out_dtype, out, ws, check_status)


@_on_stream
def matmul_grouped_dx(dy, w, offsets, *, out_dtype=None, out=None, ws=None, stream=None, check_status=True):
    """Gradient of :func:`matmul_grouped` for its rows: ``dx[t] = dy[t] w[e]``
    (``bakron_matmul_grouped_dx``)."""
    return _grouped("bakron_matmul_grouped_dx", dy, w, offsets, 1, out_dtype, out, ws, check_status)


@_on_stream
def matmul_grouped_dw(dy, x, offsets, *, out_dtype=None, out=None, ws=None, stream=None, check_status=True):
    """Gradient of :func:`matmul_grouped` for its weights: ``dw[e] = sum_t
    dy[t]^T x[t]`` over expert e's rows, experts x n x k, zeros for an expert
    without rows (``bakron_matmul_grouped_dw``)."""
    torch = _torch()
    dev = _device()
    _here(dy, "dy", (2,), (torch.bfloat16, torch.float16), dev)
    _here(x, "x", (2,), (dy.dtype,), dev)
    experts = _groups(offsets, dev)
    rows, n = dy.shape
    if x.shape[0] != rows:
        raise ValueError("dy and x must have the same rows")
    k = x.shape[1]
    if out is None and out_dtype is None:
        out_dtype = x.dtype
    dw = _result(out, (experts, n, k), out_dtype, (x.dtype, torch.float32), dev)
    if not dw.is_contiguous():
        raise ValueError("out must be contiguous")
    _call("bakron_matmul_grouped_dw",
          (dy.data_ptr(), _type_ids[x.dtype], _ld(dy, 0, n, 8), x.data_ptr(), _ld(x, 0, k, 8), offsets.data_ptr(),
           experts, dw.data_ptr(), _type_ids[dw.dtype], rows, n, k), ws, check_status, dev)
    return dw


@_on_stream
def gram_grouped(X, offsets, damping=0.0, *, ws=None, out=None, stream=None, check_status=True):
    """:func:`gram` for every expert of a layer: ``A[e] = X_e^T X_e / N_e +
    damping * mean(diag) * I`` from packed samples ``X`` (rows x d, float32,
    bfloat16 or float16) whose experts' row bounds are ``offsets`` (int32,
    experts + 1, on the device); experts x d x d float32, zeros for an expert
    without rows (``bakron_gram_grouped``)."""
    torch = _torch()
    dev = _device()
    _here(X, "X", (2,), _type_ids, dev)
    experts = _groups(offsets, dev)
    rows, d = X.shape
    A = _result(out, (experts, d, d), torch.float32, (torch.float32,), dev)
    if not A.is_contiguous():
        raise ValueError("out must be contiguous")
    t = _type_ids[X.dtype]
    need = _lib().bakron_gram_grouped_workspace_size(t, rows, d) if ws is None else 0
    _call("bakron_gram_grouped", (X.data_ptr(), t, _ld(X, 0, d, 8), offsets.data_ptr(), experts, float(damping),
                                  A.data_ptr(), rows, d), ws, check_status, dev, need)
    return A


def solve_host_workspace_size(m: int, n: int, gemm: int = 0) -> int:
    return int(_lib().bakron_solve_host_workspace_size(m, n, ctypes.byref(_config(gemm))))


def solve_host(W, LA, LB, bits=4, *, V=None, codes=None, scales=None, gemm=0, ws=None, stream=None,
               synchronize=True, leaf=0, fuse_width=0):
    """BaKron solve on HOST buffers (torch CPU tensors, ideally pinned): the
    library stages them through ``ws`` on the device and copies the results
    back.  Returns ``(V, codes, scales)`` host tensors."""
    torch = _torch()
    lib = _lib()
    m, n = W.shape
    for t, name in ((W, "W"), (LA, "LA"), (LB, "LB")):
        if t is None and name == "LB":
            continue  # B = I: the one-sided path
        if t.is_cuda or t.dtype != torch.float32 or not t.is_contiguous():
            raise TypeError(f"{name} must be a contiguous float32 CPU tensor")
    V = torch.empty((m, n), dtype=torch.float32, pin_memory=True) if V is None else V
    codes = torch.empty((m, n), dtype=torch.int8, pin_memory=True) if codes is None else codes
    scales = torch.empty((m,), dtype=torch.float32, pin_memory=True) if scales is None else scales
    cfg = _config(gemm, leaf=leaf, b_identity=int(LB is None), fuse_width=fuse_width)
    if ws is None:
        ws = workspace(lib.bakron_solve_host_workspace_size(m, n, ctypes.byref(cfg)))
    q = Quantizer(int(bits), 0, 0, 0)
    st = _stream(stream)
    check(lib.bakron_solve_host(_ptr(W), m, n, _ptr(LA), _ptr(LB), ctypes.byref(q), _ptr(V), _ptr(codes),
                                _ptr(scales), _ptr(ws), ws.numel(), ctypes.byref(cfg), st), "bakron_solve_host")
    if synchronize:
        check(lib.bakron_get_status(_ptr(ws), ws.numel(), st), "bakron_solve_host (device)")
    return V, codes, scales


def proxy_loss(W, V, A, B, *, stream=None) -> float:
    """``tr((W-V)^T B (W-V) A)`` computed on the device (both products on the
    tensor cores in 3xTF32, the elementwise dot in FP64 in a fixed order)."""
    torch = _torch()
    lib = _lib()
    m, n = W.shape
    out = torch.zeros((1,), dtype=torch.float64, device=W.device)
    ws = workspace(lib.bakron_proxy_loss_workspace_size(m, n), W.device)
    host = ctypes.c_double(0.0)
    check(lib.bakron_proxy_loss(_ptr(W), _ptr(V), _ptr(A), _ptr(B), m, n, _ptr(out), ctypes.byref(host), _ptr(ws),
                                ws.numel(), _stream(stream)), "bakron_proxy_loss")
    return float(host.value)


def last_profile() -> dict:
    """Per-kernel-class device times (ms) of the latest ``solve(..., profile=True)``
    on this thread."""
    pr = Profile()
    check(_lib().bakron_get_profile(ctypes.byref(pr)), "bakron_get_profile")
    return {f: getattr(pr, f) for f, _ in Profile._fields_}


def last_profile_launches() -> list:
    """Every launch of the latest ``solve(..., profile=True)`` on this thread, in
    launch order: dicts with kind ("prep", "leaf", "stage1", "stage2", "fused":
    both band products of a node in one launch), the recursion node (k, h, l)
    in tile diagonals, ms, FLOPs (tile-dense) and structural FLOPs (without
    the zero upper triangles of the diagonal factor tiles)."""
    lib = _lib()
    n = lib.bakron_get_profile_launches(None, 0)
    buf = (ProfileLaunch * max(1, n))()
    lib.bakron_get_profile_launches(buf, n)
    kinds = ("prep", "leaf", "stage1", "stage2", "fused")
    return [{"kind": kinds[r.kind], "k": r.k, "h": r.h, "l": r.l, "ms": r.ms, "flops": r.flops,
             "structural_flops": r.structural_flops} for r in buf[:n]]


def plan_stats(m: int, n: int, one_sided: bool = False, leaf: int = 0) -> dict:
    """Schedule statistics of an m x n solve (host only); ``one_sided`` for
    the B = I schedule over column blocks; ``leaf`` the leaf structure (7
    moves the width-2 nodes' products into the leaf launches)."""
    s = PlanStats()
    cfg = _config(b_identity=int(one_sided), leaf=leaf)
    check(_lib().bakron_plan_stats(m, n, ctypes.byref(cfg), ctypes.byref(s)), "bakron_plan_stats")
    return {f: getattr(s, f) for f, _ in PlanStats._fields_}
