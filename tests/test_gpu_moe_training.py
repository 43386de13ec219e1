"""A run of the backward operators together, as a training step uses them: gradients of a whole
expert layer against its differentiation in 64 bits, in a graph and on other streams."""
import numpy as np
import pytest

from test_gpu_linear_act import HALVES, gpu, mx, say, weights  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("tokens,experts,choices,hidden,inner", [(1, 4, 1, 64, 32), (9, 4, 2, 128, 96),
                                                                 (200, 8, 3, 256, 160), (40, 70, 6, 96, 64)])
def test_example_gradients(mx, tokens, experts, choices, hidden, inner):  # noqa: F811
    """Between the inputs and a gradient lie at most six roundings to bf16 (activations kept,
    expert rows, their gradients, the result), each with an error of at most 2^-8 of its value,
    independent of the others and spread evenly: together at most sqrt(6 / 3) 2^-8 of the norm,
    and the gradient passes through factors (silu, softmax) that move with the rounded values."""
    from weight_only_int4_gemv_amd import moe_example
    say("training step T=%d E=%d k=%d %dx%d" % (tokens, experts, choices, hidden, inner))
    errors = moe_example.train(tokens, experts, choices, hidden, inner, seed=tokens)
    assert max(errors) <= 4 * 2.0 ** -8, errors


def step(mx, state, act, dtype):  # noqa: F811
    """Every operator of this kind once, on the tensors in state."""
    logits, ids, dw, x, c, s, b, r, dout, y, tokens, positions, w, offsets, ce, se, be = state
    out = list(mx.balance(logits, ids))
    out.append(mx.route_grad(logits, ids, dw, counts=out[1], dloss=dw.new_ones(())))
    Y, Z = mx.linear_act(x, c, s, bias=b, activation=act, residual=r, save=True)
    out += [Y, Z, *mx.activation_grad(r, Z, act), mx.linear_grad(Z, c, s)]
    H, G = mx.grouped_linear_act(x, ce, se, offsets, tokens=tokens, bias=be, activation=act, save=True)
    rows, dweights = mx.combine_grad(dout, y, tokens, positions, w)
    dz, db = mx.activation_grad(H, G, act, offsets=offsets)
    out += [H, G, rows, dweights, dz, db, mx.grouped_linear_grad(dz, ce, se, offsets, dtype=torch.float32)]
    return out


def make(mx, rng, T, dtype, act):  # noqa: F811
    E, k, N, K = 6, 2, 192, 160
    F = N // 2 if act == "swiglu" else N
    logits = gpu(rng.standard_normal((T, E)), dtype)
    if T > 2:
        logits[1] = float("-inf")
    ids, w = mx.route(logits, k)
    p = mx.plan(ids, E)
    c, s = weights(rng, (N, K))
    ce, se = weights(rng, (E, N, K))

    def n(*shape):
        return gpu(rng.standard_normal(shape), dtype)
    return (logits, ids, gpu(rng.standard_normal((T, k)), torch.float32), n(T, K), gpu(c), gpu(s), n(N),
            n(T, F), n(T, F), n(T * k, F), p.tokens, p.positions, w, p.offsets, gpu(ce), gpu(se), n(E, N))


def same(a, b):
    return all(torch.equal(u.nan_to_num(7), v.nan_to_num(7)) for u, v in zip(a, b))


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("act", ["gelu", "swiglu"])
@pytest.mark.parametrize("T", [1, 24, 300])
def test_all_in_a_graph(mx, dtype, act, T):  # noqa: F811
    """Captured once and replayed on new inputs with eager work between: every replay gives what
    the eager calls give, bit for bit; two graphs replayed in turn do not disturb each other."""
    say("graph %s %s T=%d" % (dtype, act, T))
    rng = np.random.default_rng(T)
    states = [make(mx, rng, T, dtype, act) for _ in range(2)]
    for state in states:
        step(mx, state, act, dtype)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for state in states:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(step(mx, state, act, dtype))
        graphs.append(graph)
    for turn in range(3):
        for state in states:
            for t, fresh in zip(state, make(mx, rng, T, dtype, act)):
                t.copy_(fresh)
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for state, out in zip(states, outs):
            assert same(out, step(mx, state, act, dtype)), turn


@pytest.mark.parametrize("act", ["gelu_tanh", "swiglu"])
def test_all_on_two_streams_at_once(mx, act):  # noqa: F811
    say("two streams %s" % act)
    rng = np.random.default_rng(5)
    states = [make(mx, rng, 260, torch.bfloat16, act) for _ in range(2)]
    want = [step(mx, state, act, torch.bfloat16) for state in states]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in states]
    got = [None, None]
    for _ in range(4):
        for i, stream in enumerate(streams):
            with torch.cuda.stream(stream):
                got[i] = step(mx, states[i], act, torch.bfloat16)
    torch.cuda.synchronize()
    assert same(got[0], want[0]) and same(got[1], want[1])


def test_gradients_are_differences(mx):  # noqa: F811
    """Central differences of the fp32 rows of a layer with GELU against its gradients: products of
    small powers of two, so that the sums are exact and the differences those of the activation."""
    rng = np.random.default_rng(3)
    M, N, K, h = 20, 64, 64, 2.0 ** -6
    c, s = weights(rng, (1, N, K), 122, 123)
    c, s, o = gpu(c), gpu(s), gpu(np.array([0, M], dtype=np.int32))
    x = rng.choice([-0.5, 0.5, 1.0], (M, K))
    b = gpu(rng.choice([-0.25, 0.5], (1, N)), torch.bfloat16)
    d = rng.choice([-1.0, 1.0], (M, N))

    def value(v):
        y = mx.grouped_linear_act(gpu(v, torch.bfloat16), c, s, o, bias=b, activation="gelu",
                                  dtype=torch.float32)
        return (y.double().cpu().numpy() * d).sum(axis=1)
    _, z = mx.grouped_linear_act(gpu(x, torch.bfloat16), c, s, o, bias=b, activation="gelu", save=True)
    dz, _ = mx.activation_grad(gpu(d, torch.bfloat16), z, "gelu")
    dx = mx.grouped_linear_grad(dz, c, s, o, dtype=torch.float32).double().cpu().numpy()
    col = 17
    step_ = np.zeros((M, K))
    step_[:, col] = h
    diff = (value(x + step_) - value(x - step_)) / (2 * h)
    w = mx.dequantize(c[0], s[0], dtype=torch.float32).double().cpu().numpy()[:, col]
    # dz rounded to bf16 (slopes below 1.13), z to bf16 (curvature below 0.8, |z| < 16), the third
    # derivative below 1.6, fp32 values of at most 16 over 2 h
    bound = np.abs(w).sum() * (1.13 * 2.0 ** -8 + 0.8 * 16 * 2.0 ** -8) + \
        1.6 / 6 * h * h * (np.abs(w) ** 3).sum() + N * 16 * 2.0 ** -20 / (2 * h)
    assert np.abs(dx[:, col] - diff).max() <= bound
