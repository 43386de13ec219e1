"""One mixture-of-experts feed-forward layer with MXFP4 experts, as a serving
loop runs it: the experts' weights quantized once (the router keeps its own, a
small matrix whose rounding would change which experts run), then per step the
router's product, routing, the expert-ordered plan, the gathered gate-up product
with silu(gate) * up, the down product and the weighted sum, replayed from one
graph.

TrainingLayer is the same layer as training runs it: the experts' weights stay
codes, their biases, the router and what lies before the layer learn, and a
balance loss keeps the experts in use.

    python -m weight_only_int4_gemv_amd.moe_example [tokens]
"""
from __future__ import annotations

import sys
import time

import torch

from . import mxfp4


class Layer:
    """E experts of `inner` gate and up rows over `hidden` columns; router [E, hidden]."""

    def __init__(self, gate_up: torch.Tensor, down: torch.Tensor, router: torch.Tensor, choices: int):
        self.gate_up = mxfp4.quantize(gate_up)       # [E, 2 inner, hidden]
        self.down = mxfp4.quantize(down)             # [E, hidden, inner]
        self.router = router.float()
        self.experts, self.choices = gate_up.shape[0], choices

    def logits(self, x: torch.Tensor) -> torch.Tensor:
        return torch.nn.functional.linear(x.float(), self.router)

    def __call__(self, x: torch.Tensor) -> torch.Tensor:
        ids, weights = mxfp4.route(self.logits(x), self.choices)
        p = mxfp4.plan(ids, self.experts)
        h = mxfp4.grouped_linear(x, *self.gate_up, p.offsets, tokens=p.tokens, swiglu=True)
        y = mxfp4.grouped_linear(h, *self.down, p.offsets, dtype=torch.float32)
        return mxfp4.combine(y, p.positions, weights, dtype=x.dtype)


def reference(layer: Layer, x: torch.Tensor) -> torch.Tensor:
    """The layer in 64 bits, its router too, on the values the experts' codes stand
    for."""
    value = [mxfp4.dequantize(c, s, dtype=torch.float32).double().cpu()
             for c, s in (layer.gate_up, layer.down)]
    logits = x.double().cpu() @ layer.router.double().cpu().t()
    top, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    weights = torch.softmax(top[:, :layer.choices], dim=1)
    out = torch.zeros(x.shape, dtype=torch.float64)
    rows = x.double().cpu()
    inner = value[1].shape[2]
    for t in range(len(rows)):
        for j in range(layer.choices):
            e = int(ids[t, j])
            h = value[0][e] @ rows[t]
            out[t] += weights[t, j] * (value[1][e] @ (torch.nn.functional.silu(h[:inner]) * h[inner:]))
    return out


def run(tokens: int, experts: int, choices: int, hidden: int, inner: int, seed: int = 0) -> float:
    """Builds a layer, captures a step, replays it on new inputs; the largest
    error against the 64-bit layer, relative to the largest output."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    layer = Layer(normal(experts, 2 * inner, hidden) / hidden ** 0.5,
                  normal(experts, hidden, inner) / inner ** 0.5,
                  normal(experts, hidden) / hidden ** 0.5, choices)
    x = normal(tokens, hidden).bfloat16()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer(x)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer(x)
    worst = 0.0
    for _ in range(3):
        x.copy_(normal(tokens, hidden))
        graph.replay()
        want = reference(layer, x)
        worst = max(worst, float((out.double().cpu() - want).abs().max() / want.abs().max()))
    return worst


class TrainingLayer(Layer):
    """Layer with a bias for every expert's gate-up [E, 2 inner] and down [E, hidden] product,
    and its backward pass.  balance: the loss's coefficient, fp32 on the GPU."""

    def __init__(self, gate_up, down, router, choices, gate_up_bias, down_bias, balance):
        super().__init__(gate_up, down, router, choices)
        self.gate_up_bias, self.down_bias, self.balance = gate_up_bias, down_bias, balance

    def forward(self, x: torch.Tensor):
        """(output, balance loss, what backward() needs)."""
        logits = self.logits(x)
        ids, weights = mxfp4.route(logits, self.choices)
        loss, counts = mxfp4.balance(logits, ids)
        p = mxfp4.plan(ids, self.experts)
        h, z = mxfp4.grouped_linear_act(x, *self.gate_up, p.offsets, tokens=p.tokens,
                                        bias=self.gate_up_bias, activation="swiglu", save=True)
        y = mxfp4.grouped_linear_act(h, *self.down, p.offsets, bias=self.down_bias,
                                     dtype=torch.float32)
        out = mxfp4.combine(y, p.positions, weights, dtype=x.dtype)
        return out, loss, (x, logits, ids, weights, counts, p, z, y)

    def backward(self, dout: torch.Tensor, saved):
        """Gradients of <output, dout> + balance * loss: x [T, hidden], router [E, hidden] and
        the two biases, the last three in fp32."""
        x, logits, ids, weights, counts, p, z, y = saved
        rows, dweights = mxfp4.combine_grad(dout, y, p.tokens, p.positions, weights)
        _, ddown_bias = mxfp4.activation_grad(rows, rows, "none", offsets=p.offsets)
        dh = mxfp4.grouped_linear_grad(rows, *self.down, p.offsets)
        dz, dgate_up_bias = mxfp4.activation_grad(dh, z, "swiglu", offsets=p.offsets)
        dx = mxfp4.grouped_linear_grad(dz, *self.gate_up, p.offsets, dtype=torch.float32)
        dx = mxfp4.combine(dx, p.positions, torch.ones_like(weights), dtype=x.dtype)
        dlogits = mxfp4.route_grad(logits, ids, dweights, counts=counts, dloss=self.balance)
        dx += (dlogits @ self.router).to(x.dtype)
        return dx, dlogits.t().contiguous() @ x.float(), dgate_up_bias, ddown_bias


def gradient_reference(layer: TrainingLayer, x: torch.Tensor, dout: torch.Tensor):
    """The same gradients by differentiating the layer in 64 bits, on the values the experts'
    codes stand for, the choices being what they are."""
    value = [mxfp4.dequantize(c, s, dtype=torch.float32).double().cpu()
             for c, s in (layer.gate_up, layer.down)]
    leaves = [t.detach().double().cpu().requires_grad_()
              for t in (x, layer.router, layer.gate_up_bias, layer.down_bias)]
    rows, router, bias1, bias2 = leaves
    logits = rows @ router.t()
    top, ids = torch.sort(logits.detach(), dim=1, descending=True, stable=True)
    ids = ids[:, :layer.choices]
    weights = torch.softmax(logits.gather(1, ids), dim=1)
    share = torch.bincount(ids.flatten(), minlength=layer.experts).double() / ids.numel()
    loss = layer.experts * (share * torch.softmax(logits, dim=1).mean(dim=0)).sum()
    inner = value[1].shape[2]
    out = []
    for t in range(len(rows)):
        total = 0
        for j in range(layer.choices):
            e = int(ids[t, j])
            h = value[0][e] @ rows[t] + bias1[e]
            y = value[1][e] @ (torch.nn.functional.silu(h[:inner]) * h[inner:]) + bias2[e]
            total = total + weights[t, j] * y
        out.append(total)
    total = (torch.stack(out) * dout.double().cpu()).sum() + float(layer.balance) * loss
    return torch.autograd.grad(total, leaves)


def train(tokens: int, experts: int, choices: int, hidden: int, inner: int, seed: int = 0):
    """A training step captured in a graph and replayed on new inputs; the error of each
    gradient's norm against the 64-bit layer, relative to that norm, the largest of three."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    layer = TrainingLayer(normal(experts, 2 * inner, hidden) / hidden ** 0.5,
                          normal(experts, hidden, inner) / inner ** 0.5,
                          normal(experts, hidden) / hidden ** 0.5, choices,
                          (normal(experts, 2 * inner) * 0.3).bfloat16(),
                          (normal(experts, hidden) * 0.3).bfloat16(),
                          torch.full((), 0.5, device="cuda"))
    x, dout = normal(tokens, hidden).bfloat16(), normal(tokens, hidden).bfloat16()

    def step():
        _, _, saved = layer.forward(x)
        return layer.backward(dout, saved)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        grads = step()
    worst = [0.0] * len(grads)
    for _ in range(3):
        x.copy_(normal(tokens, hidden))
        dout.copy_(normal(tokens, hidden))
        graph.replay()
        for i, (got, want) in enumerate(zip(grads, gradient_reference(layer, x, dout))):
            worst[i] = max(worst[i], float((got.double().cpu() - want).norm() / want.norm()))
    return worst


def main() -> None:
    tokens = int(sys.argv[1]) if len(sys.argv) > 1 else 16
    print("error against the 64-bit layer: %.2e of the largest output"
          % run(tokens=tokens, experts=8, choices=2, hidden=512, inner=256))
    print("errors of the gradients (x, router, biases): %s of their norms"
          % ", ".join("%.2e" % e for e in train(tokens=tokens, experts=8, choices=2, hidden=512,
                                                inner=256)))
    g = torch.Generator(device="cuda").manual_seed(1)
    layer = Layer(*(torch.randn(s, generator=g, device="cuda").mul_(0.02).bfloat16()
                    for s in ((64, 2 * 1792, 4096), (64, 4096, 1792), (64, 4096))), choices=8)
    x = torch.randn((tokens, 4096), generator=g, device="cuda").bfloat16()
    for _ in range(3):
        layer(x)
    torch.cuda.synchronize()
    start = time.perf_counter()
    for _ in range(20):
        layer(x)
    torch.cuda.synchronize()
    print("%d tokens, 8 of 64 experts of 3584 x 4096: %.0f us a layer"
          % (tokens, (time.perf_counter() - start) / 20 * 1e6))


if __name__ == "__main__":
    main()
