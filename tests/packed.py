"""Plain 64-bit forms of the products over packed rows and of the 8-bit
quantiser, and the error bounds the GPU tests hold the kernels to.

Bounds.  An output is a sum of products p_i of exactly represented operands
(a product of two 16-bit or 8-bit floating values is exact in fp32).  The
tensor cores add a step of 16 or 32 products at a time to an fp32 accumulator;
every such addition may truncate, that is, lose up to one unit of the last of
24 bits of a partial sum (2^-23, relative to at most S = sum |p_i|).  An output
goes through at most `steps` of those in one accumulator and `chunks` fp32
additions of accumulators, so its error is at most (steps + chunks + c) 2^-23 S
with a small c for scaling and division, plus half a unit of the result's type.
The tests count 16-bit products at 16 steps and 256 products an accumulator; the
kernels sum 512 (fp32 results) or 1024 (16-bit ones) in one, so up to 8192 terms
the tests hold them to less than that worst case.
"""
import torch

EPS = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}


def offsets_of(lens, lead=0):
    b = [lead]
    for n in lens:
        b.append(b[-1] + n)
    return b


def check_close(got, want, size, terms, steps, per_chunk, what):
    """`got` against the 64-bit `want`; `size` the sum of the products' absolute
    values, `terms` the contraction's length."""
    assert got.shape == want.shape, what
    chunks = -(-max(terms, 1) // per_chunk)
    bound = (steps + chunks + 4) * 2.0 ** -23 * size + EPS[got.dtype] * want.abs() * (1 + 2.0 ** -8) + TINY[got.dtype]
    off = (got.double() - want).abs()
    worst = (off / bound).max().item() if off.numel() else 0.0
    print(f"[{what}] worst error / bound {worst:.3f}")
    assert torch.isfinite(got).all(), what
    assert (off <= bound).all(), (what, worst)


def quantize(x, block_rows):
    """(codes as float64, steps as float64) of x [rows, cols] by the definition."""
    x = x.double()
    rows, cols = x.shape
    codes, steps = torch.zeros_like(x), []
    for r in range(0, rows, block_rows):
        row = []
        for c in range(0, cols, 128):
            b = x[r:r + block_rows, c:c + 128]
            s = (b.abs().max() / 448).float().double()
            s = torch.ones_like(s) if s == 0 else s
            v = (b / s).float().double().clamp(-448, 448)
            e = torch.frexp(v)[1] - 1
            ulp = torch.ldexp(torch.ones_like(v), e.clamp(min=-6) - 3)
            codes[r:r + block_rows, c:c + 128] = torch.round(v / ulp) * ulp
            row.append(s)
        steps.append(torch.stack(row))
    return codes, torch.stack(steps) if steps else torch.zeros((0, -(-cols // 128)), dtype=torch.float64)


def spread(x, cols):
    """Steps [.., blocks] over columns: one value per column."""
    return x.double().repeat_interleave(128, -1)[..., :cols]
