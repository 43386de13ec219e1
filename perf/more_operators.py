"""Products with an epilogue and the backward pass of the expert layer: measured cases,
plain forms and exact values.

A case names one operator path and its sizes:

    linear        16-bit rows times MXFP4 weights with bias, activation and residual in the
                  epilogue, the values before the activation kept where a backward pass follows
    experts       the same by expert over ragged row groups, gathered, every expert with its bias
    act_grad      gradient through the activation, and the bias's gradient
    grad          gradient through the product: rows times the MXFP4 weights, untransposed
    expert_grad   the same by expert over ragged row groups
    balance       balance loss and per-expert counts of a routing, and the gradient of the loss
                  and of the routing weights with respect to the router's logits
    combine_grad  gradient of the weighted sum over a token's expert rows

MXFP4 is the OCP microscaling format: e2m1 codes, two to a byte (even column in the low
nibble), one power-of-two scale byte (exponent + 127) per 32 consecutive columns.
"""
from __future__ import annotations

import math

import torch

own = False          # False: the plain forms; True: this package's operators

DEVICE = "cuda"
BLOCK = 32
_DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
_ACTIVATIONS = ("none", "relu", "silu", "gelu", "gelu_tanh", "swiglu")
_MOST = 1 << 39      # products of a drawn case: those of the largest listed one


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # One decode token through a biased down projection that adds to the residual
        # stream: latency of a small, memory-bound launch.
        dict(name="linear-1", op="linear", M=1, N=4096, K=14336, dtype="bf16", activation="none",
             bias=True, residual=True, save=False),
        # A training or prefill chunk of odd length through a biased up projection with GELU,
        # the values before it kept for the backward pass.
        dict(name="linear-701", op="linear", M=701, N=14336, K=4096, dtype="fp16",
             activation="gelu_tanh", bias=True, residual=False, save=True),
        # A mid-sized serving batch through biased experts: tens of rows each.
        dict(name="experts-300", op="experts", T=300, E=64, k=8, K=4096, N=3584, dtype="bf16",
             activation="swiglu", bias=True, save=False),
        # A few tokens' gradients through an activation: launch latency.
        dict(name="act-grad-6", op="act_grad", M=6, N=4096, dtype="fp16", activation="gelu",
             bias=True),
        # A long chunk's gradients through silu(gate) * up of a whole layer: bandwidth.
        dict(name="act-grad-4095", op="act_grad", M=4095, N=28672, dtype="bf16",
             activation="swiglu", bias=True),
        # The gradient of a few tokens (an adapter's or a prompt's tuning): weights read once.
        dict(name="grad-17", op="grad", M=17, N=4096, K=14336, dtype="bf16"),
        # A training chunk's gradient through a gate or up projection.
        dict(name="grad-3001", op="grad", M=3001, N=14336, K=4096, dtype="fp16"),
        # A long chunk's gradient through the experts' gate and up projections; one token in
        # sixteen is padding, whose rows belong to no expert.
        dict(name="expert-grad-8192", op="expert_grad", T=8192, E=64, k=4, N=3584, K=4096,
             dtype="bf16", fp32_rows=False),
        # The loss and the router's gradient of a few tokens: launch latency.
        dict(name="balance-5", op="balance", T=5, E=64, k=6, dtype="fp32", renormalize=True,
             masked=False),
        # A whole batch's router with padding tokens and experts that some tokens may not use.
        dict(name="balance-65521", op="balance", T=65521, E=128, k=8, dtype="bf16",
             renormalize=False, masked=True),
        # The weighted sum's gradient for a few tokens, and for a long chunk with padding.
        dict(name="combine-grad-9", op="combine_grad", T=9, E=16, k=4, N=1792, dtype="fp16",
             fp32_rows=False),
        dict(name="combine-grad-6000", op="combine_grad", T=6000, E=64, k=8, N=4096, dtype="bf16",
             fp32_rows=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case: sizes over the listed ranges, M, N and T odd as they fall, K any
    multiple of the 32-column block."""
    op = rng.choice(["linear", "linear", "experts", "act_grad", "grad", "grad", "expert_grad",
                     "balance", "combine_grad"])
    dtype = rng.choice(["fp16", "bf16"])
    activation = rng.choice(_ACTIVATIONS)
    bias, save = rng.random() < 0.7, rng.random() < 0.4
    if op in ("linear", "grad"):
        N, K = _log_int(rng, 64, 16384), BLOCK * _log_int(rng, 4, 448)
        M = _log_int(rng, 1, max(1, min(4096, _MOST // (N * K))))
        if op == "grad":
            return dict(op=op, M=M, N=N, K=K, dtype=dtype)
        if activation == "swiglu":
            N += N % 2
        return dict(op=op, M=M, N=N, K=K, dtype=dtype, activation=activation, bias=bias,
                    residual=rng.random() < 0.5, save=save)
    if op == "act_grad":
        N = _log_int(rng, 64, 28672)
        return dict(op=op, M=_log_int(rng, 1, 4096), N=N + N % 2, dtype=dtype,
                    activation=activation, bias=bias)
    E = rng.choice([4, 8, 16, 32, 60, 64])
    k = rng.randint(1, min(E, 8))
    if op == "balance":
        return dict(op=op, T=_log_int(rng, 1, 65536), E=rng.choice([E, 2 * E]), k=k,
                    dtype=rng.choice(["fp16", "bf16", "fp32"]), renormalize=rng.random() < 0.5,
                    masked=rng.random() < 0.5)
    if op == "combine_grad":
        return dict(op=op, T=_log_int(rng, 1, 6000), E=E, k=k, N=_log_int(rng, 64, 4096),
                    dtype=dtype, fp32_rows=rng.random() < 0.3)
    T, K, N = _log_int(rng, 1, 4096), BLOCK * _log_int(rng, 8, 128), 2 * _log_int(rng, 64, 1792)
    if op == "expert_grad":
        return dict(op=op, T=T, E=E, k=k, N=N - rng.randint(0, 1), K=K, dtype=dtype,
                    fp32_rows=rng.random() < 0.3)
    return dict(op=op, T=T, E=E, k=k, K=K, N=N, dtype=dtype, activation=activation, bias=bias,
                save=save)


# ----------------------------------------------------------------- the inputs

def _generator(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed))
    return g


def _normal(shape, g, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device=DEVICE) * scale).to(dtype)


def _weight_codes(rows, K, g):
    """A layer's weight in MXFP4 as a checkpoint holds it (normal, sigma 0.02, one entry in
    a thousand an outlier), made in slices of rows."""
    codes = torch.empty((rows, K // 2), dtype=torch.uint8, device=DEVICE)
    scales = torch.empty((rows, K // BLOCK), dtype=torch.uint8, device=DEVICE)
    step = max(1, (1 << 26) // K)
    for r in range(0, rows, step):
        n = min(step, rows - r)
        w = torch.randn((n, K), generator=g, device=DEVICE) * 0.02
        big = torch.rand((n, K), generator=g, device=DEVICE) < 1e-3
        codes[r:r + n], scales[r:r + n] = _quantized(torch.where(big, w * 25.0, w))
    return codes, scales


def _quantized(x):
    M, K = x.shape
    b = x.view(M, K // BLOCK, BLOCK)
    peak = b.abs().amax(dim=2)
    e = torch.frexp(peak)[1].to(torch.int32) - 3          # floor(log2 peak) - 2
    e = torch.where(peak > 0, e, torch.zeros_like(e)).clamp(-127, 127)
    v = b.abs() * _power(-e)[:, :, None]
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=x.device)
    c = torch.bucketize(v, edges, out_int32=True).to(torch.uint8)
    c = torch.where(torch.signbit(b), c + 8, c).view(M, K // 2, 2)
    return c[:, :, 0] | (c[:, :, 1] << 4), (e + 127).to(torch.uint8)


def _logits(T, E, g, dtype, masked):
    """Router logits: some experts are more popular than others.  Masked: every 16th token is
    padding (no expert allowed), and of each four neighbouring experts a token may use none
    or all, three times in four all."""
    popular = torch.randn((1, E), generator=g, device=DEVICE) * 0.5
    x = (torch.randn((T, E), generator=g, device=DEVICE) + popular).to(dtype)
    if masked:
        group = torch.rand((T, (E + 3) // 4), generator=g, device=DEVICE) < 0.25
        x[group.repeat_interleave(4, dim=1)[:, :E]] = -math.inf
        x[15::16] = -math.inf
    return x


def _choices(logits, k, renormalize):
    """The k largest logits, ties to the lowest expert (-1: none left), and their weights."""
    x = logits.float()
    top, ids = torch.sort(x, dim=1, descending=True, stable=True)
    left = top > -math.inf
    p = torch.where(left, torch.exp(top - top[:, :1].clamp(min=-1e30)), 0.0)
    total = (p[:, :k] if renormalize else p).sum(dim=1, keepdim=True)
    w = torch.where(left, p / total, 0.0)[:, :k].contiguous()
    return torch.where(left, ids, -1)[:, :k].to(torch.int32).contiguous(), w


def _ordered(ids, E):
    """Rows ordered by expert, then by token; choices of no expert come last, as token and
    position -1."""
    T, k = ids.shape
    flat = torch.where((ids >= 0) & (ids < E), ids, E).reshape(-1).long()
    order = torch.argsort(flat, stable=True)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=ids.device)
    offsets[1:] = torch.bincount(flat, minlength=E + 1)[:E].cumsum(0)
    rows = torch.arange(T * k, dtype=torch.int32, device=ids.device)
    used = rows < offsets[E]
    positions = torch.empty(T * k, dtype=torch.int32, device=ids.device)
    positions[order] = torch.where(used, rows, -1)
    tokens = torch.where(used, (order // k).to(torch.int32), -1)
    return offsets, tokens, positions.view(T, k)


def prepare(case, seed):
    g = _generator(seed)
    op, dtype = case["op"], _DTYPES[case["dtype"]]
    # Gradients are small numbers; fp16 training scales its loss for them.
    grad = 0.05 if dtype == torch.float16 else 1e-3
    state = {"case": case}
    if op in ("linear", "experts"):
        N, K, swiglu = case["N"], case["K"], case["activation"] == "swiglu"
        state["bias"] = None
    if op == "linear":
        M, F = case["M"], N // 2 if swiglu else N
        state["x"] = _normal((M, K), g, dtype)
        state["codes"], state["scales"] = _weight_codes(N, K, g)
        state["residual"] = _normal((M, F), g, dtype) if case["residual"] else None
        if case["bias"]:
            state["bias"] = _normal((N,), g, dtype, 0.3)
    elif op == "act_grad":
        M, N = case["M"], case["N"]
        F = N // 2 if case["activation"] == "swiglu" else N
        state["dy"] = _normal((M, F), g, dtype, grad)
        state["z"] = _normal((M, N), g, dtype, 1.5)
    elif op == "grad":
        state["dy"] = _normal((case["M"], case["N"]), g, dtype, grad)
        state["codes"], state["scales"] = _weight_codes(case["N"], case["K"], g)
    elif op == "balance":
        T, k = case["T"], case["k"]
        state["logits"] = _logits(T, case["E"], g, dtype, case["masked"])
        state["ids"], _ = _choices(state["logits"], k, case["renormalize"])
        # The coefficient of the loss, and what comes back from the experts.
        state["dloss"] = torch.full((), 1024.0 * 0.01 if dtype == torch.float16 else 0.01,
                                    device=DEVICE)
        state["dweights"] = _normal((T, k), g, torch.float32, grad)
    else:
        T, E, k = case["T"], case["E"], case["k"]
        logits = _logits(T, E, g, torch.float32, masked=op != "experts")
        ids, weights = _choices(logits, k, True)
        state["offsets"], state["tokens"], state["positions"] = _ordered(ids, E)
        state["weights"] = weights
        if op == "combine_grad":
            state["dout"] = _normal((T, case["N"]), g, dtype, grad)
            state["y"] = _normal((T * k, case["N"]), g,
                                 torch.float32 if case["fp32_rows"] else dtype)
            return state
        N, K = case["N"], case["K"]
        codes, scales = _weight_codes(E * N, K, g)
        state["codes"] = codes.view(E, N, K // 2)
        state["scales"] = scales.view(E, N, K // BLOCK)
        if op == "experts":
            state["x"] = _normal((T, K), g, dtype)
            if case["bias"]:
                state["bias"] = _normal((E, N), g, dtype, 0.3)
        else:
            state["dy"] = _normal((T * k, N), g, dtype, grad)
    return state


# ------------------------------------------------------------ the plain forms

def _power(e):
    """2^e in 32 bits for whole -126 <= e <= 127, exact."""
    return ((e + 127) << 23).view(torch.float32)


def _plain_values(codes, scales):
    """The values MXFP4 codes and scales stand for, in 32 bits."""
    table = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), device=codes.device)
    c = torch.stack((codes & 15, codes >> 4), dim=-1).to(torch.int32)
    v = table[c].view(scales.shape + (BLOCK,))
    return (v * _power(scales.to(torch.int32) - 127)[..., None]).view(
        codes.shape[:-1] + (2 * codes.shape[-1],))


def _halves(z):
    return z[:, :z.shape[1] // 2], z[:, z.shape[1] // 2:]


def _sigmoid(v):
    return 1 / (1 + torch.exp(-v))


def _plain_act(z, activation):
    if activation == "none":
        return z
    if activation == "relu":
        return torch.where(z > 0, z, 0.0)
    if activation == "silu":
        return z * _sigmoid(z)
    if activation == "gelu":
        return 0.5 * z * torch.erfc(-math.sqrt(0.5) * z)
    if activation == "gelu_tanh":
        return z * _sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z))
    gate, up = _halves(z)
    return gate * _sigmoid(gate) * up


def _plain_slope(z, activation):
    if activation == "none":
        return torch.ones_like(z)
    if activation == "relu":
        return (z > 0).float()
    if activation == "silu":
        s = _sigmoid(z)
        return s * (1 + z * (1 - s))
    if activation == "gelu":
        return (0.5 * torch.erfc(-math.sqrt(0.5) * z)
                + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi)))
    c = 2 * math.sqrt(2 / math.pi)
    s = _sigmoid(c * (z + 0.044715 * z * z * z))
    return s + z * s * (1 - s) * c * (1 + 3 * 0.044715 * z * z)


def _plain_act_grad(dy, z, activation):
    if activation != "swiglu":
        return dy * _plain_slope(z, activation)
    gate, up = _halves(z)
    return torch.cat((dy * up * _plain_slope(gate, "silu"), dy * gate * _sigmoid(gate)), dim=1)


def _plain_experts(x, state, rows, transposed):
    """Each expert's rows times its weights, in 32 bits; rows of no expert stay 0."""
    codes, scales, bias = state["codes"], state["scales"], state.get("bias")
    bounds = state["offsets"].tolist()
    columns = codes.shape[1] if transposed else 2 * codes.shape[2]
    out = torch.zeros((rows, columns), device=x.device)
    for e, (lo, hi) in enumerate(zip(bounds, bounds[1:])):
        if hi > lo:
            w = _plain_values(codes[e], scales[e])
            out[lo:hi] = x[lo:hi].float() @ (w.t() if transposed else w)
            if bias is not None:
                out[lo:hi] += bias[e].float()
    return out


def _plain_softmax(logits):
    """Over the usable experts; a row without one is 0."""
    x = logits.float()
    peak = x.amax(dim=1, keepdim=True)
    p = torch.exp(x - torch.where(peak > -math.inf, peak, 0.0))
    total = p.sum(dim=1, keepdim=True)
    return torch.where(total > 0, p / total, 0.0)


def _plain_balance(state):
    case, ids = state["case"], state["ids"].long()
    logits, dw = state["logits"], state["dweights"]
    E = case["E"]
    p = _plain_softmax(logits)
    chosen = ids >= 0
    slot = torch.where(chosen, ids, 0)
    counts = torch.zeros(E + 1, dtype=torch.int32, device=ids.device)
    counts[:E] = torch.bincount(ids[chosen], minlength=E)
    counts[E] = (logits > -math.inf).any(dim=1).sum()
    c = counts[:E].float()
    scale = E / (c.sum() * counts[E]).clamp(min=1)
    loss = scale * (c * p.double().sum(dim=0)).sum()
    dl = state["dloss"] * scale * p * (c - (p * c).sum(dim=1, keepdim=True))
    w = torch.where(chosen, p.gather(1, slot), 0.0)
    if case["renormalize"]:
        w = torch.where(chosen, w / w.sum(dim=1, keepdim=True), 0.0)
        part = w * (dw - (w * dw).sum(dim=1, keepdim=True))
    else:
        dl = dl - p * (w * dw).sum(dim=1, keepdim=True)
        part = w * dw
    dl.scatter_add_(1, slot, torch.where(chosen, part, 0.0))
    return loss.float(), counts, dl.to(logits.dtype)


def _plain_combine_grad(state):
    dout, y, positions = state["dout"].float(), state["y"], state["positions"].long()
    dy = torch.zeros(y.shape, dtype=state["dout"].dtype, device=y.device)
    dw = torch.zeros(positions.shape, device=y.device)
    for j in range(positions.shape[1]):
        used = positions[:, j] >= 0
        rows, d = positions[used, j], dout[used]
        dy[rows] = (state["weights"][used, j:j + 1] * d).to(dy.dtype)
        dw[used, j] = (d * y[rows].float()).sum(dim=1)
    return dy, dw


def _run_plain(state):
    case = state["case"]
    op, dtype = case["op"], _DTYPES[case["dtype"]]
    if op in ("linear", "experts"):
        if op == "linear":
            z = state["x"].float() @ _plain_values(state["codes"], state["scales"]).t()
            if state["bias"] is not None:
                z = z + state["bias"].float()
        else:
            z = _plain_experts(state["x"][state["tokens"].long()], state, len(state["tokens"]),
                               True)
        y = _plain_act(z, case["activation"])
        if op == "linear" and state["residual"] is not None:
            y = y + state["residual"].float()
        return (y.to(dtype), z.to(dtype)) if case["save"] else y.to(dtype)
    if op == "act_grad":
        dz = _plain_act_grad(state["dy"].float(), state["z"].float(), case["activation"])
        return (dz.to(dtype), dz.sum(dim=0)) if case["bias"] else dz.to(dtype)
    if op == "grad":
        return (state["dy"].float() @ _plain_values(state["codes"], state["scales"])).to(dtype)
    if op == "expert_grad":
        dx = _plain_experts(state["dy"], state, len(state["dy"]), False)
        return dx if case["fp32_rows"] else dx.to(dtype)
    return _plain_balance(state) if op == "balance" else _plain_combine_grad(state)


# ------------------------------------------------------- this package's calls

def _run_own(state):
    from weight_only_int4_gemv_amd import mxfp4

    case = state["case"]
    op = case["op"]
    if op == "linear":
        return mxfp4.linear_act(state["x"], state["codes"], state["scales"], bias=state["bias"],
                                activation=case["activation"], residual=state["residual"],
                                save=case["save"])
    if op == "experts":
        return mxfp4.grouped_linear_act(state["x"], state["codes"], state["scales"],
                                        state["offsets"], tokens=state["tokens"],
                                        bias=state["bias"], activation=case["activation"],
                                        save=case["save"])
    if op == "act_grad":
        return mxfp4.activation_grad(state["dy"], state["z"], case["activation"],
                                     bias=case["bias"])
    if op == "grad":
        return mxfp4.linear_grad(state["dy"], state["codes"], state["scales"])
    if op == "expert_grad":
        return mxfp4.grouped_linear_grad(state["dy"], state["codes"], state["scales"],
                                         state["offsets"],
                                         dtype=torch.float32 if case["fp32_rows"] else None)
    if op == "balance":
        loss, counts = mxfp4.balance(state["logits"], state["ids"])
        dlogits = mxfp4.route_grad(state["logits"], state["ids"], dweights=state["dweights"],
                                   renormalize=case["renormalize"], counts=counts,
                                   dloss=state["dloss"])
        return loss, counts, dlogits
    return mxfp4.combine_grad(state["dout"], state["y"], state["tokens"], state["positions"],
                              state["weights"])


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------- the work

def work(case):
    """Bytes and operations one pass cannot do without.  The experts' weights count for the
    experts that some token chooses, their number taken at its mean for independent, equally
    likely choices."""
    op = case["op"]
    size = 4 if case["dtype"] == "fp32" else 2
    if op in ("linear", "grad"):
        M, N, K = case["M"], case["N"], case["K"]
        moved = 2 * M * K + N * (K // 2 + K // BLOCK)
        if op == "grad":
            return {"bytes": moved + 2 * M * N, "flops": 2 * M * N * K}
        F = N // 2 if case["activation"] == "swiglu" else N
        return {"bytes": moved + 2 * M * F * (1 + case["residual"]) + 2 * M * N * case["save"]
                + 2 * N * case["bias"], "flops": 2 * M * N * K}
    if op == "act_grad":
        M, N = case["M"], case["N"]
        F = N // 2 if case["activation"] == "swiglu" else N
        return {"bytes": 2 * M * F + 4 * M * N + 4 * N * case["bias"], "flops": 8 * M * N}
    T, E, k = case["T"], case["E"], case["k"]
    if op == "balance":
        return {"bytes": 2 * T * E * size + 8 * T * k + 4 * (E + 2), "flops": 10 * T * E}
    N = case["N"]
    if op == "combine_grad":
        return {"bytes": 2 * T * N + T * k * N * (6 if case["fp32_rows"] else 4) + 16 * T * k,
                "flops": 3 * T * k * N}
    K = case["K"]
    touched = E * (1 - (1 - k / E) ** T)
    weights = int(touched * N * (K // 2 + K // BLOCK))
    if op == "expert_grad":
        return {"bytes": weights + 2 * T * k * N + T * k * K * (4 if case["fp32_rows"] else 2),
                "flops": 2 * T * k * N * K}
    F = N // 2 if case["activation"] == "swiglu" else N
    return {"bytes": weights + 2 * T * K + 4 * T * k + 2 * T * k * (F + N * case["save"])
            + int(touched * 2 * N) * case["bias"], "flops": 2 * T * k * N * K}


# ----------------------------------------------------------- the exact values

def _exact_weights(codes, scales):
    """MXFP4 values in 64 bits from the format's fields: sign, exponent, mantissa."""
    nib = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2).to(torch.int16)
    s, ex, m = nib >> 3, (nib >> 1) & 3, (nib & 1).double()
    mag = torch.where(ex == 0, m * 0.5, (1 + m * 0.5) * (2.0 ** (ex - 1).double()))
    e = scales.long() - 127
    return (torch.where(s == 1, -mag, mag)
            * ((e + 1023) << 52).view(torch.float64).repeat_interleave(BLOCK, dim=-1))


def _exact_act(z, activation):
    nn = torch.nn.functional
    if activation == "swiglu":
        gate, up = z.chunk(2, dim=1)
        return nn.silu(gate) * up
    return {"none": lambda v: v, "relu": nn.relu, "silu": nn.silu, "gelu": nn.gelu,
            "gelu_tanh": lambda v: nn.gelu(v, approximate="tanh")}[activation](z)


def _exact_experts(state, case):
    """The experts' products in 64 bits, expert by expert."""
    offsets = state["offsets"].cpu()
    forward = case["op"] == "experts"
    rows = state["tokens"].shape[0]
    out = torch.zeros((rows, case["N"] if forward else case["K"]), dtype=torch.float64,
                      device=DEVICE)
    for e in range(case["E"]):
        mine = slice(int(offsets[e]), int(offsets[e + 1]))
        if mine.start == mine.stop:
            continue
        w = _exact_weights(state["codes"][e], state["scales"][e])
        if forward:
            out[mine] = state["x"][state["tokens"][mine].long()].double() @ w.t()
            if state["bias"] is not None:
                out[mine] += state["bias"][e].double()
        else:
            out[mine] = state["dy"][mine].double() @ w
    return out


def _exact_balance(state, case):
    """The loss as a function of the logits of the tokens that may use an expert, and the
    gradient of dloss * loss + sum(dweights * weights) from differentiating it."""
    E, ids = case["E"], state["ids"].long()
    live = (state["logits"] > -math.inf).any(dim=1)
    grad = torch.zeros(state["logits"].shape, dtype=torch.float64, device=DEVICE)
    ids, dw = ids[live], state["dweights"][live].double()
    counts = torch.stack([(ids == e).sum() for e in range(E)]).double()
    total = torch.cat((counts, live.sum()[None])).to(torch.int32)
    if not bool(live.any()):
        return torch.zeros((), dtype=torch.float64, device=DEVICE), total, grad
    x = state["logits"][live].double().requires_grad_()
    p = torch.softmax(x, dim=1)
    loss = E * ((counts / counts.sum()) * p.mean(dim=0)).sum()
    there = ids >= 0
    if case["renormalize"]:
        picked = torch.where(there, x.gather(1, ids.clamp(min=0)), -math.inf)
        w = torch.softmax(picked, dim=1)
    else:
        w = torch.where(there, p.gather(1, ids.clamp(min=0)), 0.0)
    (state["dloss"].double() * loss + (w * dw).sum()).backward()
    grad[live] = torch.where(state["logits"][live] > -math.inf, x.grad, 0.0)
    return loss.detach(), total, grad


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op in ("linear", "experts"):
        if op == "linear":
            z = state["x"].double() @ _exact_weights(state["codes"], state["scales"]).t()
            if state["bias"] is not None:
                z += state["bias"].double()
        else:
            z = _exact_experts(state, case)
        y = _exact_act(z, case["activation"])
        if op == "linear" and state["residual"] is not None:
            y = y + state["residual"].double()
        return (y, z) if case["save"] else y
    if op == "act_grad":
        z = state["z"].double().requires_grad_()
        _exact_act(z, case["activation"]).backward(state["dy"].double())
        return (z.grad, z.grad.sum(dim=0)) if case["bias"] else z.grad
    if op == "grad":
        return state["dy"].double() @ _exact_weights(state["codes"], state["scales"])
    if op == "expert_grad":
        return _exact_experts(state, case)
    if op == "balance":
        return _exact_balance(state, case)
    # combine_grad: row by row, from the row's token and the slot that names it.
    tokens = state["tokens"].long()
    used = tokens >= 0
    rows = torch.arange(len(tokens), device=DEVICE)[used]
    mine = state["positions"][tokens[used]] == rows[:, None]
    slots = mine.long().argmax(dim=1)
    dw = torch.zeros(state["weights"].shape, dtype=torch.float64, device=DEVICE)
    dy = torch.zeros(state["y"].shape, dtype=torch.float64, device=DEVICE)
    for lo in range(0, len(rows), 8192):
        r, s = rows[lo:lo + 8192], slots[lo:lo + 8192]
        t = tokens[r]
        d = state["dout"][t].double()
        dy[r] = state["weights"][t, s].double()[:, None] * d
        dw[t, s] = torch.linalg.vecdot(d, state["y"][r].double())
    return dy, dw
