"""The MXFP4 and mixture-of-experts operators: measured cases, plain forms and exact values.

A case names one operator path and its sizes:

    quantize   activations or weights to MXFP4 and back to the values they stand for
    linear     16-bit activations times MXFP4 weights (decode, small batch, prefill)
    matmul     activations quantised to MXFP4 in the call, times MXFP4 weights
    route      top-k routing of tokens to experts and the expert-ordered plan
    gate_up    per-expert product over ragged row groups, gathered, with silu(gate) * up
    down       per-expert product over ragged row groups, then the weighted sum per token

MXFP4 here is the OCP microscaling format: e2m1 codes, two to a byte (even column in the
low nibble), one power-of-two scale byte (exponent + 127) per 32 consecutive columns.
"""
from __future__ import annotations

import math

import torch

own = False          # False: the plain forms; True: this package's operators

DEVICE = "cuda"
BLOCK = 32
_DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # A few decode tokens' activations on their way into a 4-bit product: launch latency.
        dict(name="quantize-7-tokens", op="quantize", M=7, K=4096, dtype="bf16"),
        # A whole 70B-class FFN matrix quantised at load time: bandwidth.
        dict(name="quantize-weights", op="quantize", M=28672, K=8192, dtype="fp16"),
        # One decode token through the gate (or up) projection of an 8B-class layer.
        dict(name="linear-1", op="linear", M=1, N=14336, K=4096, dtype="bf16"),
        # A small odd serving batch through the long-K down projection.
        dict(name="linear-50", op="linear", M=50, N=4096, K=14336, dtype="fp16"),
        # Prefill of a prompt whose length is no multiple of any tile.
        dict(name="linear-2000", op="linear", M=2000, N=14336, K=4096, dtype="fp16"),
        # A short prompt with 4-bit activations, long K, few output tiles.
        dict(name="matmul-200", op="matmul", M=200, N=4096, K=14336, dtype="bf16"),
        # A long prefill through a 70B-class FFN matrix with 4-bit activations.
        dict(name="matmul-4096", op="matmul", M=4096, N=28672, K=8192, dtype="bf16"),
        # Routing of a few decode tokens: launch latency.
        dict(name="route-3", op="route", T=3, E=64, k=6, dtype="fp32", renormalize=True,
             masked=False),
        # Routing of a long prefill over many experts; padding tokens take no expert, and
        # each token may use only some of the expert groups.
        dict(name="route-8191", op="route", T=8191, E=128, k=8, dtype="bf16", renormalize=False,
             masked=True),
        # Four decode tokens through the experts' gate and up projections: most of the
        # chosen experts have one row, the other experts' weights are not read.
        dict(name="gate-up-4", op="gate_up", T=4, E=64, k=8, K=4096, N=1792, dtype="bf16"),
        # A mid-sized serving batch through the experts' down projections: tens of rows each.
        dict(name="down-300", op="down", T=300, E=64, k=8, K=1792, N=4096, dtype="fp16"),
        # A long prefill through the experts' gate and up projections.
        dict(name="gate-up-8192", op="gate_up", T=8192, E=64, k=4, K=4096, N=1792, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case: sizes over the listed ranges, M, N and T odd as they fall, K any
    multiple of the 32-column block."""
    op = rng.choice(["quantize", "linear", "linear", "matmul", "route", "gate_up", "down"])
    dtype = rng.choice(["fp16", "bf16"])
    if op == "quantize":
        return dict(op=op, M=_log_int(rng, 1, 16384), K=32 * _log_int(rng, 1, 448),
                    dtype=rng.choice(["fp16", "bf16", "fp32"]))
    if op in ("linear", "matmul"):
        return dict(op=op, M=_log_int(rng, 1, 4096), N=_log_int(rng, 64, 16384),
                    K=32 * _log_int(rng, 4, 448), dtype=dtype)
    E = rng.choice([4, 8, 16, 32, 60, 64, 128])
    k = rng.randint(1, min(E, 8))
    if op == "route":
        return dict(op=op, T=_log_int(rng, 1, 16384), E=E, k=k,
                    dtype=rng.choice(["fp16", "bf16", "fp32"]),
                    renormalize=rng.random() < 0.5, masked=rng.random() < 0.5)
    E = min(E, 64)
    return dict(op=op, T=_log_int(rng, 1, 4096), E=E, k=min(k, E),
                K=32 * _log_int(rng, 8, 128), N=_log_int(rng, 64, 2048), dtype=dtype)


# ----------------------------------------------------------------- the inputs

def _generator(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed))
    return g


def _normal(shape, g, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device=DEVICE) * scale).to(dtype)


def _weight(rows, K, g, outlier=1e-3):
    """A layer's weight: normal, sigma 0.02, one entry in a thousand an outlier."""
    w = torch.randn((rows, K), generator=g, device=DEVICE) * 0.02
    big = torch.rand((rows, K), generator=g, device=DEVICE) < outlier
    return torch.where(big, w * 25.0, w)


def _weight_codes(rows, K, g):
    """A weight in MXFP4 as a checkpoint holds it, made in slices of rows."""
    codes = torch.empty((rows, K // 2), dtype=torch.uint8, device=DEVICE)
    scales = torch.empty((rows, K // BLOCK), dtype=torch.uint8, device=DEVICE)
    step = max(1, (1 << 26) // K)
    for r in range(0, rows, step):
        n = min(step, rows - r)
        codes[r:r + n], scales[r:r + n] = _plain_quantize(_weight(n, K, g))
    return codes, scales


def _logits(T, E, g, dtype):
    """Router logits: some experts are more popular than others, and one token in
    eight repeats a value across experts (16-bit logits tie in earnest)."""
    popular = torch.randn((1, E), generator=g, device=DEVICE) * 0.5
    x = torch.randn((T, E), generator=g, device=DEVICE) + popular
    coarse = (x * 2).round() / 2
    ties = torch.arange(T, device=DEVICE)[:, None] % 8 == 7
    return torch.where(ties, coarse, x).to(dtype)


def _mask(logits, g):
    """Every 16th token is padding (no expert allowed), and of each four neighbouring
    experts a token may use none or all, three times in four all."""
    T, E = logits.shape
    group = torch.rand((T, (E + 3) // 4), generator=g, device=DEVICE) < 0.25
    logits[group.repeat_interleave(4, dim=1)[:, :E]] = -math.inf
    logits[15::16] = -math.inf


def prepare(case, seed):
    g = _generator(seed)
    op, dtype = case["op"], _DTYPES[case["dtype"]]
    state = {"case": case}
    if op == "quantize":
        if case["M"] > 1000:                       # a weight
            state["x"] = _weight(case["M"], case["K"], g).to(dtype)
        else:
            state["x"] = _normal((case["M"], case["K"]), g, dtype)
    elif op in ("linear", "matmul"):
        state["x"] = _normal((case["M"], case["K"]), g, dtype)
        state["codes"], state["scales"] = _weight_codes(case["N"], case["K"], g)
    elif op == "route":
        state["logits"] = _logits(case["T"], case["E"], g, dtype)
        if case["masked"]:
            _mask(state["logits"], g)
    else:
        T, E, k, K, N = (case[n] for n in ("T", "E", "k", "K", "N"))
        logits = _logits(T, E, g, torch.float32)
        ids, weights = _plain_route(logits, k, True)
        state["offsets"], state["tokens"], state["positions"] = _plain_plan(ids, E)
        state["weights"] = weights
        rows = T if op == "gate_up" else T * k
        out = 2 * N if op == "gate_up" else N
        state["x"] = _normal((rows, K), g, dtype)
        codes, scales = _weight_codes(E * out, K, g)
        state["codes"] = codes.view(E, out, K // 2)
        state["scales"] = scales.view(E, out, K // BLOCK)
    return state


# ------------------------------------------------------------ the plain forms

def _power(e):
    """2^e in 32 bits for whole -126 <= e <= 127, exact."""
    return ((e + 127) << 23).view(torch.float32)


def _plain_quantize(x):
    M, K = x.shape
    b = x.float().view(M, K // BLOCK, BLOCK)
    a = b.abs()
    peak = a.amax(dim=2)
    e = torch.frexp(peak)[1].to(torch.int32) - 3          # floor(log2 peak) - 2
    e = torch.where(peak > 0, e, torch.zeros_like(e)).clamp(-127, 127)
    v = a * _power(-e)[:, :, None]
    c = ((v > 0.25).to(torch.uint8) + (v >= 0.75).to(torch.uint8) + (v > 1.25).to(torch.uint8)
         + (v >= 1.75).to(torch.uint8) + (v > 2.5).to(torch.uint8) + (v >= 3.5).to(torch.uint8)
         + (v > 5.0).to(torch.uint8))
    c = torch.where(torch.signbit(b), c + 8, c).view(M, K // 2, 2)
    return c[:, :, 0] | (c[:, :, 1] << 4), (e + 127).to(torch.uint8)


def _plain_values(codes, scales):
    """The values MXFP4 codes and scales stand for, in 32 bits."""
    table = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), device=codes.device)
    c = torch.stack((codes & 15, codes >> 4), dim=-1).to(torch.int32)
    v = table[c].view(scales.shape + (BLOCK,))
    return (v * _power(scales.to(torch.int32) - 127)[..., None]).view(
        codes.shape[:-1] + (2 * codes.shape[-1],))


def _plain_product(x, codes, scales):
    return x.float() @ _plain_values(codes, scales).t()


def _plain_route(logits, k, renormalize):
    """An expert whose logit is -inf is not chosen: its slot has id -1 and weight 0."""
    x = logits.float()
    top, ids = torch.sort(x, dim=1, descending=True, stable=True)
    peak = top[:, :1].clamp(min=torch.finfo(torch.float32).min)
    top, ids = top[:, :k], ids[:, :k].to(torch.int32)
    p = torch.exp(top - peak)
    total = (p if renormalize else torch.exp(x - peak)).sum(dim=1, keepdim=True)
    left = top > -math.inf
    return torch.where(left, ids, -1), torch.where(left, p / total, 0.0)


def _plain_plan(ids, E):
    """Rows ordered by expert, then by token; choices of no expert come last, as token
    and position -1."""
    T, k = ids.shape
    flat = torch.where((ids >= 0) & (ids < E), ids, E).reshape(-1).long()
    order = torch.argsort(flat, stable=True)
    counts = (flat[:, None] == torch.arange(E, device=ids.device)).sum(0)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=ids.device)
    offsets[1:] = counts.cumsum(0)
    rows = torch.arange(T * k, dtype=torch.int32, device=ids.device)
    used = rows < offsets[E]
    positions = torch.empty(T * k, dtype=torch.int32, device=ids.device)
    positions[order] = torch.where(used, rows, -1)
    tokens = torch.where(used, (order // k).to(torch.int32), -1)
    return offsets, tokens, positions.view(T, k)


def _plain_grouped(x, state):
    bounds = state["offsets"].tolist()
    out = torch.empty((bounds[-1], state["codes"].shape[1]), device=x.device)
    for e, (lo, hi) in enumerate(zip(bounds, bounds[1:])):
        if hi > lo:
            out[lo:hi] = _plain_product(x[lo:hi], state["codes"][e], state["scales"][e])
    return out


def _run_plain(state):
    case = state["case"]
    op, dtype = case["op"], _DTYPES[case["dtype"]]
    if op == "quantize":
        return _plain_values(*_plain_quantize(state["x"])).to(dtype)
    if op == "linear":
        return _plain_product(state["x"], state["codes"], state["scales"]).to(dtype)
    if op == "matmul":
        x = _plain_values(*_plain_quantize(state["x"]))
        return _plain_product(x, state["codes"], state["scales"]).to(dtype)
    if op == "route":
        ids, weights = _plain_route(state["logits"], case["k"], case["renormalize"])
        return (ids, weights) + _plain_plan(ids, case["E"])
    if op == "gate_up":
        h = _plain_grouped(state["x"][state["tokens"].long()], state)
        gate, up = h[:, :case["N"]], h[:, case["N"]:]
        return (gate / (1 + torch.exp(-gate)) * up).to(dtype)
    y = _plain_grouped(state["x"], state)
    rows = y[state["positions"].long()]                   # [T, k, N]
    return (rows * state["weights"][:, :, None]).sum(dim=1).to(dtype)


# ------------------------------------------------------- this package's calls

def _run_own(state):
    from weight_only_int4_gemv_amd import mxfp4

    case = state["case"]
    op = case["op"]
    if op == "quantize":
        codes, scales = mxfp4.quantize(state["x"])
        return mxfp4.dequantize(codes, scales, dtype=state["x"].dtype)
    if op == "linear":
        return mxfp4.linear(state["x"], state["codes"], state["scales"])
    if op == "matmul":
        codes, scales = mxfp4.quantize(state["x"])
        return mxfp4.matmul(codes, scales, state["codes"], state["scales"],
                            dtype=state["x"].dtype)
    if op == "route":
        ids, weights = mxfp4.route(state["logits"], case["k"], renormalize=case["renormalize"])
        return (ids, weights) + tuple(mxfp4.plan(ids, case["E"]))
    if op == "gate_up":
        return mxfp4.grouped_linear(state["x"], state["codes"], state["scales"],
                                    state["offsets"], tokens=state["tokens"], swiglu=True)
    y = mxfp4.grouped_linear(state["x"], state["codes"], state["scales"], state["offsets"])
    return mxfp4.combine(y, state["positions"], state["weights"])


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------- the work

def work(case):
    """Bytes and operations one pass cannot do without.  The experts' weights count
    for the experts that some token chooses, their number taken at its mean for
    independent, equally likely choices."""
    op = case["op"]
    size = 4 if case["dtype"] == "fp32" else 2
    if op == "quantize":
        n = case["M"] * case["K"]
        # in, the codes and scales out and in again, the values out
        return {"bytes": 2 * size * n + 2 * (n // 2 + n // BLOCK), "flops": 4 * n}
    if op in ("linear", "matmul"):
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": 2 * M * K + N * (K // 2 + K // BLOCK) + 2 * M * N,
                "flops": 2 * M * N * K}
    T, E, k = case["T"], case["E"], case["k"]
    if op == "route":
        return {"bytes": T * E * size + 8 * T * k + 4 * (E + 1) + 8 * T * k,
                "flops": 4 * T * E}
    K, N = case["K"], case["N"]
    touched = E * (1 - (1 - k / E) ** T)
    if op == "gate_up":
        return {"bytes": int(touched * 2 * N * (K // 2 + K // BLOCK)) + 2 * T * K
                + 4 * T * k + 2 * T * k * N, "flops": 4 * T * k * N * K}
    return {"bytes": int(touched * N * (K // 2 + K // BLOCK)) + 2 * T * k * K + 8 * T * k
            + 2 * T * N, "flops": 2 * T * k * N * K + 2 * T * k * N}


# ----------------------------------------------------------- the exact values

def _exact_weights(codes, scales):
    """MXFP4 values in 64 bits from the format's fields: sign, exponent, mantissa."""
    nib = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2).to(torch.int16)
    s, ex, m = nib >> 3, (nib >> 1) & 3, (nib & 1).double()
    mag = torch.where(ex == 0, m * 0.5, (1 + m * 0.5) * (2.0 ** (ex - 1).double()))
    v = torch.where(s == 1, -mag, mag)
    e = scales.long() - 127
    return v * ((e + 1023) << 52).view(torch.float64).repeat_interleave(BLOCK, dim=-1)


def _exact_rounded(x):
    """x in 64 bits, each block of 32 rounded to its MXFP4 values: the scale from the
    exponent field of the block's peak, the element to the nearest multiple of its binade's
    step (half to even)."""
    shape = x.shape
    b = x.double().reshape(-1, BLOCK)
    e = ((b.abs().amax(dim=1).view(torch.int64) >> 52) - 1023 - 2).clamp(-127, 127)
    power = ((e + 1023) << 52).view(torch.float64)[:, None]
    a = b.abs() / power
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).double()
    q = (torch.round(a / step) * step).clamp(max=6.0)
    return (torch.copysign(q, b) * power).reshape(shape)


def _exact_routing(rows, case):
    E, k = case["E"], case["k"]
    ids, weights = [], []
    for row in rows:
        usable = [i for i in range(E) if row[i] > -math.inf]
        chosen = sorted(usable, key=lambda i: (-row[i], i))[:k]
        peak = max((row[i] for i in usable), default=0.0)
        total = math.fsum(math.exp(row[i] - peak)
                          for i in (chosen if case["renormalize"] else usable))
        spare = k - len(chosen)
        ids.append(chosen + [-1] * spare)
        weights.append([math.exp(row[i] - peak) / total for i in chosen] + [0.0] * spare)
    lists = [[] for _ in range(E)]
    for t, chosen in enumerate(ids):
        for j, e in enumerate(chosen):
            if e >= 0:
                lists[e].append((t, j))
    offsets, tokens = [0], []
    positions = [[-1] * k for _ in ids]
    for members in lists:
        for t, j in members:
            positions[t][j] = len(tokens)
            tokens.append(t)
        offsets.append(len(tokens))
    tokens += [-1] * (len(ids) * k - len(tokens))
    return (torch.tensor(ids, dtype=torch.int32), torch.tensor(weights, dtype=torch.float64),
            torch.tensor(offsets, dtype=torch.int32), torch.tensor(tokens, dtype=torch.int32),
            torch.tensor(positions, dtype=torch.int32))


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        x = state["x"]
        step = max(1, (1 << 26) // case["K"])             # bounds the 64-bit copies
        return torch.cat([_exact_rounded(x[r:r + step]).float()
                          for r in range(0, case["M"], step)]).double()
    if op in ("linear", "matmul"):
        x = state["x"].double() if op == "linear" else _exact_rounded(state["x"])
        return x @ _exact_weights(state["codes"], state["scales"]).t()
    if op == "route":
        return _exact_routing(state["logits"].double().cpu().tolist(), case)
    N, k = case["N"], case["k"]
    x, offsets = state["x"].double(), state["offsets"].cpu()
    tokens = state["tokens"].long()
    chunks = []
    for e in range(case["E"]):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if hi == lo:
            continue
        a = x[tokens[lo:hi]] if op == "gate_up" else x[lo:hi]
        h = a @ _exact_weights(state["codes"][e], state["scales"][e]).t()
        if op == "gate_up":
            h = torch.nn.functional.silu(h[:, :N]) * h[:, N:]
        chunks.append(h)
    h = torch.cat(chunks)
    if op == "gate_up":
        return h
    out = torch.zeros((case["T"], N), dtype=torch.float64, device=h.device)
    for j in range(k):
        out += state["weights"][:, j:j + 1].double() * h[state["positions"][:, j].long()]
    return out
