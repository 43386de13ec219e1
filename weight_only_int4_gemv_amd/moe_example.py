"""One mixture-of-experts feed-forward layer with MXFP4 experts, as a serving
loop runs it: the experts' weights quantized once (the router keeps its own, a
small matrix whose rounding would change which experts run), then per step the
router's product, routing, the expert-ordered plan, the gathered gate-up product
with silu(gate) * up, the down product and the weighted sum, replayed from one
graph.

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


def main() -> None:
    tokens = int(sys.argv[1]) if len(sys.argv) > 1 else 16
    print("error against the 64-bit layer: %.2e of the largest output"
          % run(tokens=tokens, experts=8, choices=2, hidden=512, inner=256))
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
