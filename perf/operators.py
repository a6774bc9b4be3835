"""Operators around the solver, for measurement: what a program does with
quantised weights and with experts.

Each operator in its plain form (elementary torch operations in 32 bits,
rounded once at the end), the call a user makes of this package for it, and
its definition in 64 bits.

    quantize       8-bit floating point (e4m3) codes with one fp32 step for
                   each block of 1 x 128 or 128 x 128 values
    blocks         product of two such operands, dense or grouped by expert;
                   the weight's steps per 128 x 128 block or per row
    grouped        products grouped by expert over packed rows: forward and
                   the two gradients
    gram           one damped Gram factor per expert from packed samples
"""
import random

import torch

own = False

_TYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}
_SIZE = {"float32": 4, "bfloat16": 2, "float16": 2}
_E4M3_MAX = 448.0


# ------------------------------------------------------------------- cases
def listed():
    return [
        # activations of a whole prompt, cast once per layer before its 8-bit products
        {"name": "quantize rows 16384x4096 bf16", "op": "quantize", "rows": 16384, "cols": 4096, "block_rows": 1,
         "dtype": "bfloat16", "batch": 1},
        # a weight matrix laid out in 8 bits as it is loaded
        {"name": "quantize tiles 14336x4096 fp32", "op": "quantize", "rows": 14336, "cols": 4096, "block_rows": 128,
         "dtype": "float32", "batch": 1},
        # one token through a projection: the latency of a decoding step
        {"name": "blocks 1x4096x4096", "op": "blocks", "rows": 1, "n": 4096, "k": 4096, "experts": 0, "tail": 0,
         "per_row": False, "out": "bfloat16", "skew": 0.0},
        # a short prompt through an up projection rounded to 4-bit codes with one step per row
        {"name": "blocks 777x11008x4096 per row", "op": "blocks", "rows": 777, "n": 11008, "k": 4096, "experts": 0,
         "tail": 0, "per_row": True, "out": "bfloat16", "skew": 0.0},
        # a long prompt through the widest projection
        {"name": "blocks 8192x14336x4096", "op": "blocks", "rows": 8192, "n": 14336, "k": 4096, "experts": 0, "tail": 0,
         "per_row": False, "out": "bfloat16", "skew": 0.0},
        # a batch routed to experts, uneven loads, a padded end
        {"name": "blocks 4100 rows 16 experts", "op": "blocks", "rows": 4100, "n": 4096, "k": 2048, "experts": 16,
         "tail": 60, "per_row": False, "out": "bfloat16", "skew": 1.0},
        # a decoding step of many sequences over many small experts, some without a row
        {"name": "grouped 96 rows 64 experts", "op": "grouped", "what": "y", "rows": 96, "n": 1024, "k": 2048,
         "experts": 64, "tail": 0, "dtype": "bfloat16", "out": "bfloat16", "skew": 1.0},
        # a calibration batch forward through large experts
        {"name": "grouped 16384 rows 8 experts", "op": "grouped", "what": "y", "rows": 16384, "n": 4096, "k": 4096,
         "experts": 8, "tail": 0, "dtype": "bfloat16", "out": "bfloat16", "skew": 0.5},
        # gradients flowing back to the experts' inputs, half precision, odd sizes
        {"name": "grouped dx 5001 rows 16 experts", "op": "grouped", "what": "dx", "rows": 5001, "n": 2760, "k": 1023,
         "experts": 16, "tail": 7, "dtype": "float16", "out": "float16", "skew": 1.0},
        # the experts' weight gradients, accumulated in 32 bits
        {"name": "grouped dw 16384 rows 8 experts", "op": "grouped", "what": "dw", "rows": 16384, "n": 4096, "k": 1024,
         "experts": 8, "tail": 0, "dtype": "bfloat16", "out": "float32", "skew": 0.5},
        # input factors of small experts from 32-bit samples
        {"name": "gram fp32 8192x1024 8 experts", "op": "gram", "rows": 8192, "d": 1024, "experts": 8, "tail": 5,
         "dtype": "float32", "skew": 0.5},
        # input factors of large experts from 16-bit activations
        {"name": "gram bf16 16384x4096 4 experts", "op": "gram", "rows": 16384, "d": 4096, "experts": 4, "tail": 0,
         "dtype": "bfloat16", "skew": 0.5},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


_MOST_FLOPS = 2.0 * 8192 * 14336 * 4096  # the largest listed product


def draw(rng):
    op = rng.choice(["quantize", "blocks", "blocks", "grouped", "grouped", "grouped", "gram"])
    if op == "quantize":
        return {"op": op, "rows": _log(rng, 1, 11000), "cols": _log(rng, 60, 4096), "block_rows": rng.choice([1, 128]),
                "dtype": rng.choice(["float32", "bfloat16", "float16"]), "batch": rng.choice([1, 1, 3])}
    if op == "blocks":
        grouped = rng.random() < 0.5
        c = {"op": op, "rows": _log(rng, 1, 8192), "n": _log(rng, 100, 8192), "k": _log(rng, 100, 4096),
             "experts": _log(rng, 2, 24) if grouped else 0, "tail": rng.choice([0, 33]) if grouped else 0,
             "per_row": rng.random() < 0.5, "out": rng.choice(["bfloat16", "float16", "float32"]),
             "skew": rng.choice([0.0, 1.0])}
        if grouped:
            c["n"] = min(c["n"], 4096)
        return c
    if op == "grouped":
        t = rng.choice(["bfloat16", "float16"])
        c = {"op": op, "what": rng.choice(["y", "dx", "dw"]), "rows": _log(rng, 1, 16384), "n": _log(rng, 64, 4096),
             "k": _log(rng, 64, 4096), "experts": _log(rng, 1, 48), "tail": rng.choice([0, 19]), "dtype": t,
             "out": rng.choice([t, "float32"]), "skew": rng.choice([0.0, 0.5, 1.0])}
        # the padded products and the exact sums stay in seconds: many experts are small ones
        while c["experts"] * c["n"] * c["k"] > 8 * 4096 * 4096:
            c["n"], c["k"] = (c["n"] + 1) // 2, (c["k"] + 1) // 2
        return c
    c = {"op": op, "rows": _log(rng, 16, 16384), "d": _log(rng, 64, 2048), "experts": _log(rng, 1, 16),
         "tail": rng.choice([0, 11]), "dtype": rng.choice(["float32", "bfloat16", "float16"]),
         "skew": rng.choice([0.0, 0.5])}
    while c["experts"] * c["d"] * c["d"] > 8 * 2048 * 2048:
        c["d"] = (c["d"] + 1) // 2
    return c


def _counts(case):
    """Rows of each expert, largest first: a fixed function of the case, so
    that what a pass has to read does not depend on the seed."""
    e, t = case["experts"], case["rows"]
    r = random.Random("%d/%d/%s" % (t, e, case["skew"]))
    share = [r.expovariate(1.0) ** case["skew"] for _ in range(e)]
    got = [0] * e
    for i in r.choices(range(e), share, k=t):
        got[i] += 1
    return sorted(got, reverse=True)


def work(case):
    if case["op"] == "quantize":
        n = case["batch"] * case["rows"] * case["cols"]
        blocks = case["batch"] * -(-case["rows"] // case["block_rows"]) * -(-case["cols"] // 128)
        return {"bytes": n * (_SIZE[case["dtype"]] + 1) + 4 * blocks, "flops": 3 * n}
    if case["op"] == "blocks":
        t, n, k = case["rows"], case["n"], case["k"]
        live = sum(c > 0 for c in _counts(case)) if case["experts"] else 1
        steps = n if case["per_row"] else -(-n // 128) * -(-k // 128)
        return {"bytes": t * k + 4 * t * -(-k // 128) + live * (n * k + 4 * steps) + t * n * _SIZE[case["out"]],
                "flops": 2 * t * n * k}
    t, e, s = case["rows"], case["experts"], _SIZE[case["dtype"]]
    live = sum(c > 0 for c in _counts(case))
    if case["op"] == "grouped":
        n, k, o = case["n"], case["k"], _SIZE[case["out"]]
        b = {"y": t * k * s + live * n * k * s + t * n * o, "dx": t * n * s + live * n * k * s + t * k * o,
             "dw": t * (n + k) * s + e * n * k * o}
        return {"bytes": b[case["what"]], "flops": 2 * t * n * k}
    d = case["d"]
    return {"bytes": t * d * s + 4 * e * d * d, "flops": t * d * (d + 1)}


# ------------------------------------------------------------------ inputs
def _randn(shape, gen, scale=1.0):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * scale


def _activations(rows, cols, gen):
    """Rows with a few outlier channels and uneven token norms, as
    activations of a language model have."""
    x = _randn((rows, cols), gen)
    x *= torch.where(torch.rand(cols, generator=gen, device="cuda") < 0.01, 20.0, 1.0)
    x *= torch.exp(0.3 * _randn((rows, 1), gen))
    return x


def _aligned(x, multiple):
    """The same values with rows that start on 16-byte boundaries, the layout
    in which a program keeps an odd width."""
    pad = -x.shape[-1] % multiple
    if not pad:
        return x.contiguous()
    wide = torch.zeros(x.shape[:-1] + (x.shape[-1] + pad,), dtype=x.dtype, device=x.device)
    wide[..., : x.shape[-1]] = x
    return wide[..., : x.shape[-1]]


def _offsets(case, gen):
    order = torch.randperm(case["experts"], generator=gen, device="cuda").tolist()
    counts = _counts(case)
    bounds = [0]
    for e in order:
        bounds.append(bounds[-1] + counts[e])
    return torch.tensor(bounds, dtype=torch.int32, device="cuda"), max(counts)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    # the few bytes in which the package records errors found on the device
    state = {"case": case, "status": torch.empty(1024, dtype=torch.uint8, device="cuda")}
    if case["op"] == "quantize":
        x = _activations(case["batch"] * case["rows"], case["cols"], gen) * 0.7
        if case["block_rows"] == 128:
            x = x * 0.02
        x = x.to(_TYPES[case["dtype"]])
        state["x"] = x if case["batch"] == 1 else x.view(case["batch"], case["rows"], case["cols"])
        return state
    rows = case["rows"] + case["tail"]
    if case["experts"]:
        state["offsets"], state["longest"] = _offsets(case, gen)
    if case["op"] == "blocks":
        n, k, e = case["n"], case["k"], max(1, case["experts"])
        q, s = _quantize(_activations(rows, k, gen), 1)
        state["x"], state["x_scales"] = _aligned(q.view(torch.uint8), 16).view(torch.float8_e4m3fn), s
        w = _randn((e, n, k), gen, 0.02)
        if case["per_row"]:  # 4-bit codes with one step per row, as the solver returns them
            s = w.abs().amax(2) / 7.0
            q = torch.round(w / s[..., None]).clamp(-7, 7).to(torch.float8_e4m3fn)
        else:
            q, s = _quantize(w, 128)
        q = _aligned(q.view(torch.uint8), 16).view(torch.float8_e4m3fn)
        state["w"], state["w_scales"] = (q, s) if case["experts"] else (q[0], s[0])
        state["out"] = torch.zeros((rows, n), dtype=_TYPES[case["out"]], device="cuda")
        return state
    t = _TYPES[case["dtype"]]
    if case["op"] == "gram":
        state["x"] = _aligned((_activations(rows, case["d"], gen)).to(t), 8)
        return state
    n, k, e = case["n"], case["k"], case["experts"]
    x, dy = _activations(rows, k, gen), _randn((rows, n), gen, 0.1)
    if case["what"] in ("y", "dw"):
        state["x"] = _aligned(x.to(t), 8)
    if case["what"] in ("dx", "dw"):
        state["dy"] = _aligned(dy.to(t), 8)
    if case["what"] in ("y", "dx"):
        state["w"] = _aligned(_randn((e, n, k), gen, 0.02).to(t), 8)
    shape = {"y": (rows, n), "dx": (rows, k), "dw": (e, n, k)}[case["what"]]
    state["out"] = torch.zeros(shape, dtype=_TYPES[case["out"]], device="cuda")
    return state


# ------------------------------------------------------------- plain forms
def _quantize(x, block_rows):
    """(codes, steps) of x [.., R, C]: steps over blocks of block_rows x 128."""
    r, c = x.shape[-2:]
    pr, pc = -r % block_rows, -c % 128
    x = torch.nn.functional.pad(x.float(), (0, pc, 0, pr))
    b = x.reshape(x.shape[:-2] + ((r + pr) // block_rows, block_rows, (c + pc) // 128, 128))
    # a block whose step is zero (all zeros, or underflow) gets 1
    s = b.abs().amax(dim=(-3, -1))
    # a quotient of tensors: by a number, torch multiplies with its reciprocal
    s = s / torch.full_like(s, _E4M3_MAX)
    s = torch.where(s == 0, 1.0, s)
    v = (b / s[..., :, None, :, None]).clamp(-_E4M3_MAX, _E4M3_MAX).reshape(x.shape)[..., :r, :c]
    return v.to(torch.float8_e4m3fn), s


def _expert_of(offsets, rows):
    """(expert, place within it) of each packed row that belongs to one; the
    rows behind the last sequence come with expert = number of experts."""
    t = torch.arange(rows, device=offsets.device, dtype=torch.int64)
    o = offsets.to(torch.int64)
    e = torch.searchsorted(o[1:], t, right=True)
    return e, t - o[e]


def _padded(x, e, at, experts, longest):
    """Packed rows as [experts, longest, width], zeros behind each sequence."""
    p = torch.zeros((experts + 1, longest, x.shape[1]), dtype=torch.float32, device=x.device)
    inside = e < experts
    p[torch.where(inside, e, experts), torch.where(inside, at, 0)] = torch.where(inside[:, None], x.float(), 0.0)
    return p[:experts]


def _packed(p, e, at, out):
    """The rows of [experts, longest, width] back in their packed places; the
    rows behind the last sequence stay what `out` has."""
    experts = p.shape[0]
    inside = (e < experts)[:, None]
    got = p[e.clamp(max=experts - 1), torch.where(e < experts, at, 0)]
    return torch.where(inside, got.to(out.dtype), out)


def _plain(state):
    case = state["case"]
    if case["op"] == "quantize":
        return _quantize(state["x"], case["block_rows"])
    if case["op"] == "blocks":
        k, n = case["k"], case["n"]
        x = state["x"].float() * state["x_scales"].repeat_interleave(128, 1)[:, :k]
        w, s = state["w"].float(), state["w_scales"]
        w = w * (s[..., None] if case["per_row"] else
                 s.repeat_interleave(128, -1).repeat_interleave(128, -2)[..., :n, :k])
        if not case["experts"]:
            return (x @ w.T).to(state["out"].dtype)
        e, at = _expert_of(state["offsets"], x.shape[0])
        y = torch.bmm(_padded(x, e, at, case["experts"], state["longest"]), w.transpose(1, 2))
        return _packed(y, e, at, state["out"])
    rows = case["rows"] + case["tail"]
    e, at = _expert_of(state["offsets"], rows)
    pad = lambda v: _padded(v, e, at, case["experts"], state["longest"])  # noqa: E731
    if case["op"] == "gram":
        x = pad(state["x"])
        count = (state["offsets"][1:] - state["offsets"][:-1]).clamp(min=1).float()
        a = torch.bmm(x.transpose(1, 2), x) / count[:, None, None]
        mean = a.diagonal(dim1=1, dim2=2).mean(1)
        return a + torch.diag_embed((0.01 * mean)[:, None].expand(-1, case["d"]))
    if case["what"] == "y":
        return _packed(torch.bmm(pad(state["x"]), state["w"].float().transpose(1, 2)), e, at, state["out"])
    if case["what"] == "dx":
        return _packed(torch.bmm(pad(state["dy"]), state["w"].float()), e, at, state["out"])
    return torch.bmm(pad(state["dy"]).transpose(1, 2), pad(state["x"])).to(state["out"].dtype)


def _calls(state):
    import two_sided_gptq_b200 as bk

    case = state["case"]
    kept = {"ws": state["status"], "check_status": False}
    if case["op"] == "quantize":
        return bk.quantize_blocks(state["x"], case["block_rows"], **kept)
    if case["op"] == "blocks":
        return bk.matmul_blocks(state["x"], state["x_scales"], state["w"], state["w_scales"], state.get("offsets"),
                                out=state["out"], **kept)
    if case["op"] == "gram":
        return bk.gram_grouped(state["x"], state["offsets"], 0.01, check_status=False)
    if case["what"] == "y":
        return bk.matmul_grouped(state["x"], state["w"], state["offsets"], out=state["out"], **kept)
    if case["what"] == "dx":
        return bk.matmul_grouped_dx(state["dy"], state["w"], state["offsets"], out=state["out"], **kept)
    return bk.matmul_grouped_dw(state["dy"], state["x"], state["offsets"], out=state["out"], **kept)


def run(state):
    if own:
        return _calls(state)
    return _plain(state)


# ------------------------------------------------------------- definitions
def _e4m3(v):
    """The nearest e4m3 value of each |v| <= 448, ties to the even code."""
    exponent = torch.frexp(v)[1] - 1
    step = torch.ldexp(torch.ones_like(v), exponent.clamp(min=-6) - 3)
    return torch.round(v / step) * step


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "quantize":
        x = state["x"].double()
        x = x if x.dim() == 3 else x[None]
        rows, cols, high = case["rows"], case["cols"], case["block_rows"]
        codes, steps = torch.zeros_like(x), []
        for c in range(0, cols, 128):
            part = x[:, :, c:c + 128]
            most = part.abs().amax(2)
            if high > 1:
                most = torch.stack([most[:, r:r + high].amax(1) for r in range(0, rows, high)], 1)
            s = (most / 448).float().double()
            s[s == 0] = 1
            steps.append(s)
            each = s.repeat_interleave(high, 1)[:, :rows, None]
            # the decision is taken on the quotient rounded to 32 bits
            codes[:, :, c:c + 128] = _e4m3((part / each).float().double().clamp(-448, 448))
        steps = torch.stack(steps, 2)
        return (codes, steps) if case["batch"] > 1 else (codes[0], steps[0])
    if case["op"] == "blocks":
        k, n = case["k"], case["n"]
        column = torch.arange(k, device="cuda") // 128
        x = state["x"].double() * state["x_scales"].double()[:, column]

        def weight(w, s):
            if case["per_row"]:
                return w.double() * s.double()[:, None]
            return w.double() * s.double()[torch.arange(n, device="cuda") // 128][:, column]

        if not case["experts"]:
            return x @ weight(state["w"], state["w_scales"]).T
        bounds = state["offsets"].tolist()
        y = state["out"].double()
        for e, (a, b) in enumerate(zip(bounds, bounds[1:])):
            y[a:b] = x[a:b] @ weight(state["w"][e], state["w_scales"][e]).T
        return y
    bounds = state["offsets"].tolist()
    if case["op"] == "gram":
        a = torch.zeros((case["experts"], case["d"], case["d"]), dtype=torch.float64, device="cuda")
        for e, (lo, hi) in enumerate(zip(bounds, bounds[1:])):
            if hi > lo:
                x = state["x"][lo:hi].double()
                a[e] = x.T @ x / (hi - lo)
                a[e] += 0.01 * (a[e].trace() / case["d"]) * torch.eye(case["d"], dtype=torch.float64, device="cuda")
        return a
    out = state["out"].double()
    for e, (lo, hi) in enumerate(zip(bounds, bounds[1:])):
        if case["what"] == "y":
            out[lo:hi] = state["x"][lo:hi].double() @ state["w"][e].double().T
        elif case["what"] == "dx":
            out[lo:hi] = state["dy"][lo:hi].double() @ state["w"][e].double()
        else:
            out[e] = state["dy"][lo:hi].double().T @ state["x"][lo:hi].double()
    return out
