"""The gradient through an activation where a lane takes eight columns (2^18 elements and more, rows
on 16 bytes), on the GPU against the plain 64-bit form: every activation, dense and by expert, with
and without the bias's gradient."""
import numpy as np
import pytest

import mxfp4_grad_reference as gref
from test_gpu_linear_act import HALVES, RAGGED, check_activation_grad, gpu, mx, say  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

# Rows end inside a block of 64, inside the sixteen that a block has in hand, or one past a block;
# columns end eight into a block of 512 or fill an eighth of one.
SIZES = [(701, 520), (65, 4104), (4099, 64)]


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("act", gref.ACTIVATIONS)
@pytest.mark.parametrize("M,F", SIZES)
def test_eight_columns(mx, dtype, act, M, F):  # noqa: F811
    assert M * F >= 1 << 18 and F % 8 == 0
    N = 2 * F if act == "swiglu" else F
    say("eight columns %s %s M=%d N=%d" % (dtype, act, M, N))
    rng = np.random.default_rng([M, F])
    dy, z = gpu(rng.standard_normal((M, F)), dtype), gpu(rng.standard_normal((M, N)) * 3, dtype)
    first = check_activation_grad(mx, dy, z, act)
    again = mx.activation_grad(dy, z, act)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("act", gref.ACTIVATIONS)
def test_eight_columns_of_rows_further_apart(mx, dtype, act):  # noqa: F811
    """What lies between the rows is not read (NaN there), and what lies around dZ not written."""
    M, F = 701, 520
    N = 2 * F if act == "swiglu" else F
    say("eight columns, rows apart %s %s" % (dtype, act))
    rng = np.random.default_rng(2)
    dy = torch.full((M, F + 16), float("nan"), dtype=dtype, device="cuda")
    z = torch.full((M, N + 24), float("nan"), dtype=dtype, device="cuda")
    dy[:, 8:F + 8], z[:, 16:N + 16] = gpu(rng.standard_normal((M, F)), dtype), gpu(rng.standard_normal((M, N)) * 3, dtype)
    dy, z = dy[:, 8:F + 8], z[:, 16:N + 16]
    room = torch.full((M + 2, N), 7.0, dtype=dtype, device="cuda")
    got, _ = check_activation_grad(mx, dy, z, act, dZ=room[1:-1])
    assert got.data_ptr() == room[1:-1].data_ptr() and (room[0] == 7).all() and (room[-1] == 7).all()


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("act", gref.ACTIVATIONS[:-1])
def test_eight_columns_of_far_values(mx, dtype, act):  # noqa: F811
    """Infinities, zeros and the type's ends among the values before the activation."""
    M, F = 701, 520
    say("eight columns, far values %s %s" % (dtype, act))
    rng = np.random.default_rng(3)
    z = gpu(rng.standard_normal((M, F)) * 3, dtype)
    far = [float("inf"), -float("inf"), 0.0, torch.finfo(dtype).max, torch.finfo(dtype).min, 45.0, -45.0]
    for i, v in enumerate(far):
        z.view(-1)[i * 11::97] = v
    got, _ = check_activation_grad(mx, gpu(rng.standard_normal((M, F)), dtype), z, act)
    assert got.isfinite().all()


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("name", list(RAGGED))
@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "gelu_tanh"])
def test_eight_columns_by_expert(mx, dtype, name, act):  # noqa: F811
    R, F = 720, 520
    say("eight columns by expert %s %s %s" % (dtype, name, act))
    rng = np.random.default_rng(4)
    offsets = gpu((np.array(RAGGED[name]) * 9).astype(np.int32))
    check_activation_grad(mx, gpu(rng.standard_normal((R, F)), dtype),
                          gpu(rng.standard_normal((R, F)) * 2, dtype), act, offsets=offsets)
