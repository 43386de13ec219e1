"""Products with an epilogue and the backward operators on the host: refusals of the C ABI
(no kernel is launched: without a device a call that passes the checks reports DEVICE), of
the binding, and the 64-bit reference against differences."""
import numpy as np
import pytest
import torch

import mxfp4_grad_reference as gref
from test_mxfp4_host import A, B, C, D, DEVICE, F, FAKE, INVALID, MISALIGNED, OK, SHAPE, lib  # noqa: F401
from weight_only_int4_gemv_amd import mxfp4

ROWS = 16                            # MXFP4_FP32_ROWS
G, H, I, J = (FAKE * i for i in range(6, 10))
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are not real")
NONE, RELU, SWIGLU = 0, 1, 5


def linear_act(lib, X=A, dt=0, M=4, xs=64, c=B, s=C, N=8, K=64, b=G, act=RELU, r=H, rs=8, Y=D, Z=F,  # noqa: F811
               ws=None, wb=0):
    return lib.mxfp4_linear_act(X, dt, M, xs, c, s, N, K, b, act, r, rs, Y, Z, ws, wb, None)


def test_linear_act_refusals(lib):  # noqa: F811
    def call(**kw):
        return linear_act(lib, **kw)
    assert call(dt=2) == INVALID and call(dt=ROWS) == INVALID and call(dt=-1) == INVALID
    assert call(act=-1) == INVALID and call(act=6) == INVALID
    assert call(N=7, act=SWIGLU) == SHAPE and call(K=80) == SHAPE
    assert call(M=-1) == INVALID and call(N=1 << 25) == INVALID and call(K=-32) == INVALID
    assert call(xs=32) == INVALID and call(xs=68) == MISALIGNED
    assert call(rs=7) == INVALID and call(rs=3, act=SWIGLU) == INVALID and call(rs=1 << 40) == INVALID
    for name in ("X", "c", "s", "Y"):
        assert call(**{name: None}) == INVALID
    for name in ("b", "r", "Y", "Z"):
        assert call(**{name: I + 1}) == MISALIGNED
    assert call(X=A + 8) == MISALIGNED and call(c=B + 8) == MISALIGNED
    for other in (A, B, C, G, H):                                # inputs under an output
        assert call(Y=other) == INVALID and call(Z=other) == INVALID
    assert call(Y=F) == INVALID and call(Y=F + 62) == INVALID
    assert call(wb=16) == INVALID and call(ws=I + 8, wb=64) == MISALIGNED
    assert call(M=0, X=None, Y=None) == OK and call(N=0, c=None, s=None, Y=None) == OK


@no_gpu
def test_linear_act_valid_calls(lib):  # noqa: F811
    def call(**kw):
        return linear_act(lib, **kw)
    assert call() == DEVICE and call(dt=1, act=SWIGLU, rs=4) == DEVICE
    assert call(b=None, r=None, Z=None, rs=0, act=NONE) == DEVICE
    assert call(K=0, xs=0, X=None, c=None, s=None) == DEVICE
    assert call(Y=D + 2, Z=F + 2, b=G + 2, r=H + 2, rs=9) == DEVICE
    assert call(Y=F + 64) == DEVICE                              # right behind Z
    # with SwiGLU Y is half of Z's width
    assert call(act=SWIGLU, rs=4, Y=F - 32) == DEVICE and call(Y=F - 32) == INVALID
    M, N, K = 50, 512, 8192
    need = lib.mxfp4_linear_act_workspace_bytes(M, N, K)
    assert need > 0
    far = 16 * FAKE

    def sliced(ws, wb):
        return linear_act(lib, M=M, N=N, K=K, xs=K, rs=N, ws=ws, wb=wb)
    assert sliced(far, need) == DEVICE and sliced(None, 0) == DEVICE
    assert sliced(far, need - 1) == INVALID
    for other in (A, B, C, G, H, D, F):
        assert sliced(other - need + 16, need) == INVALID


def test_grouped_linear_act_refusals(lib):  # noqa: F811
    def call(X=A, dt=0, xr=4, xs=64, tok=None, R=4, c=B, s=C, off=D, E=2, N=8, K=64, b=G, act=RELU, Y=F,
             Z=H):
        return lib.mxfp4_grouped_linear_act(X, dt, xr, xs, tok, R, c, s, off, E, N, K, b, act, Y, Z, None)
    assert call(dt=2) == INVALID and call(dt=ROWS + 2) == INVALID and call(act=9) == INVALID
    assert call(E=0) == INVALID and call(E=1025) == INVALID and call(R=-1) == INVALID
    assert call(K=63) == SHAPE and call(N=7, act=SWIGLU) == SHAPE
    assert call(R=5) == INVALID and call(xs=32) == INVALID and call(xs=68) == MISALIGNED
    for name in ("X", "c", "s", "off", "Y"):
        assert call(**{name: None}) == INVALID
    assert call(b=G + 1) == MISALIGNED and call(Z=H + 1) == MISALIGNED and call(off=D + 2) == MISALIGNED
    assert call(dt=ROWS, Y=F + 2) == MISALIGNED
    for other in (A, B, C, D, G):
        assert call(Y=other) == INVALID and call(Z=other) == INVALID
    assert call(b=F + 60) == INVALID and call(Z=F) == INVALID
    assert call(dt=ROWS, Z=F + 64) == INVALID                    # fp32 rows are twice as long
    assert call(R=0, Y=None) == OK and call(N=0, Y=None) == OK
    if not torch.cuda.is_available():
        assert call() == DEVICE and call(b=None, Z=None) == DEVICE and call(Z=F + 64) == DEVICE
        assert call(dt=ROWS + 1, act=SWIGLU) == DEVICE and call(b=F + 64) == DEVICE


def test_activation_grad_refusals(lib):  # noqa: F811
    def call(dY=A, dt=0, R=4, ys=8, Z=B, zs=8, N=8, act=RELU, off=None, E=0, dZ=C, db=D, ws=None, wb=0):
        return lib.mxfp4_activation_grad(dY, dt, R, ys, Z, zs, N, act, off, E, dZ, db, ws, wb, None)
    assert call(dt=2) == INVALID and call(R=-1) == INVALID and call(N=-1) == INVALID
    assert call(act=6) == INVALID and call(act=SWIGLU, N=9, zs=9) == SHAPE
    assert call(ys=7) == INVALID and call(zs=7) == INVALID and call(act=SWIGLU, ys=3) == INVALID
    assert call(E=2) == INVALID and call(off=F, E=0) == INVALID and call(off=F, E=1025) == INVALID
    for name in ("dY", "Z", "dZ"):
        assert call(**{name: None}) == INVALID and call(**{name: H + 1}) == MISALIGNED
    assert call(db=D + 2) == MISALIGNED and call(off=F + 2, E=2, ws=G, wb=4096) == MISALIGNED
    assert call(dZ=A) == INVALID and call(dZ=B + 62) == INVALID and call(db=C + 60) == INVALID
    size = lib.mxfp4_activation_grad_workspace_bytes
    assert size(64, 8, 0) == 0 and size(65, 8, 0) == 2 * 8 * 4 and size(4, 8, 2) == 4 * 8 * 4
    for bad in ((-1, 8, 0), (8, -1, 0), (8, 8, -1), (8, 8, 1025), (1 << 25, 8, 0), (0, 8, 0), (8, 0, 2)):
        assert size(*bad) == 0
    need = size(200, 8, 0)
    assert call(R=200) == INVALID and call(R=200, ws=G, wb=need - 1) == INVALID
    assert call(R=200, ws=G + 2, wb=need) == MISALIGNED
    assert call(R=200, ws=A, wb=need) == INVALID
    assert call(N=0, ys=0, zs=0) == OK and call(R=0, db=None, dY=None) == OK
    if not torch.cuda.is_available():
        assert call() == DEVICE and call(db=None) == DEVICE and call(R=200, ws=G, wb=need) == DEVICE
        assert call(R=200, db=None) == DEVICE                    # no sum, no workspace
        assert call(R=0, dY=None, Z=None, dZ=None) == DEVICE     # dbias = 0
        assert call(off=F, E=2, ws=G, wb=size(4, 8, 2)) == DEVICE and call(off=F, E=2) == INVALID


def test_linear_grad_refusals(lib):  # noqa: F811
    def call(dY=A, dt=0, M=4, ys=8, c=B, s=C, N=8, K=64, dX=D, ws=None, wb=0):
        return lib.mxfp4_linear_grad(dY, dt, M, ys, c, s, N, K, dX, ws, wb, None)
    assert call(dt=2) == INVALID and call(dt=ROWS) == INVALID
    assert call(M=-1) == INVALID and call(N=-1) == INVALID and call(K=-32) == INVALID
    assert call(K=80) == SHAPE and call(ys=7) == INVALID
    for name in ("dY", "c", "s", "dX"):
        assert call(**{name: None}) == INVALID
    assert call(dY=A + 1) == MISALIGNED and call(c=B + 8) == MISALIGNED and call(dX=D + 8) == MISALIGNED
    assert call(dX=A) == INVALID and call(dX=B) == INVALID and call(dX=C) == INVALID
    assert call(M=0, dX=None) == OK and call(K=0, dX=None) == OK
    size = lib.mxfp4_linear_grad_workspace_bytes
    for bad in ((-1, 8, 32), (8, -1, 32), (8, 8, 33), (1 << 25, 8, 32), (0, 8, 64), (8, 8, 0), (8, 0, 64)):
        assert size(*bad) == 0
    M, N, K = 20, 8192, 256
    need = size(M, N, K)
    assert need > 0 and need % (M * K * 4) == 0
    far = 16 * FAKE

    def sliced(ws, wb):
        return call(M=M, N=N, K=K, ys=N, ws=ws, wb=wb)
    assert sliced(far, need - 1) == INVALID and sliced(far + 8, need) == MISALIGNED
    assert sliced(None, need) == INVALID
    for other in (A, B, C, D):
        assert sliced(other - need + 16, need) == INVALID
    if not torch.cuda.is_available():
        assert call() == DEVICE and call(dY=A + 2, ys=9) == DEVICE and call(N=7) == DEVICE
        assert call(N=0, ys=0, dY=None, c=None, s=None) == DEVICE
        assert sliced(far, need) == DEVICE and sliced(None, 0) == DEVICE


def test_grouped_linear_grad_refusals(lib):  # noqa: F811
    def call(dY=A, dt=0, R=4, ys=8, c=B, s=C, off=D, E=2, N=8, K=64, dX=F):
        return lib.mxfp4_grouped_linear_grad(dY, dt, R, ys, c, s, off, E, N, K, dX, None)
    assert call(dt=2) == INVALID and call(dt=ROWS + 2) == INVALID and call(E=0) == INVALID
    assert call(E=1025) == INVALID and call(K=33) == SHAPE and call(ys=7) == INVALID
    for name in ("dY", "c", "s", "off", "dX"):
        assert call(**{name: None}) == INVALID
    assert call(off=D + 2) == MISALIGNED and call(dX=F + 4, dt=ROWS) == MISALIGNED
    for other in (A, B, C, D):
        assert call(dX=other) == INVALID
    # 4 rows of 64 are 512 bytes, in fp32 1024
    assert call(dX=A - 1008, dt=ROWS) == INVALID
    assert call(R=0, dX=None) == OK and call(K=0, dX=None) == OK
    if not torch.cuda.is_available():
        assert call() == DEVICE and call(dt=ROWS + 1) == DEVICE and call(dX=A - 512) == DEVICE


def test_balance_refusals(lib):  # noqa: F811
    size = lib.moe_balance_workspace_bytes
    need = size(1000, 8, 2)
    assert need > 0 and size(0, 8, 2) == 0 and size(128, 64, 2) == 0 and size(4, 1024, 2) > 0
    for bad in ((-1, 8, 2), (1000, 0, 2), (1000, 1025, 2), (1000, 8, 0), (1000, 8, 33), (1 << 25, 8, 2)):
        assert size(*bad) == 0
    far = 16 * FAKE

    def call(x=A, dt=0, T=1000, E=8, st=8, ids=B, k=2, loss=C, n=D, ws=far, wb=need):
        return lib.moe_balance(x, dt, T, E, st, ids, k, loss, n, ws, wb, None)
    assert call(dt=3) == INVALID and call(T=-1) == INVALID and call(E=0) == INVALID
    assert call(E=1025, st=1025) == INVALID and call(k=0) == INVALID and call(k=33) == INVALID
    assert call(st=7) == INVALID
    for name in ("x", "ids", "loss", "n"):
        assert call(**{name: None}) == INVALID and call(**{name: G + 1}) == MISALIGNED
    assert call(x=A + 2, dt=2) == MISALIGNED and call(ws=far + 2) == MISALIGNED
    assert call(ws=None, wb=0) == INVALID and call(wb=need - 1) == INVALID
    assert call(loss=A) == INVALID and call(n=B) == INVALID and call(loss=D + 32) == INVALID
    assert call(ws=A) == INVALID and call(ws=D) == INVALID
    if not torch.cuda.is_available():
        assert call() == DEVICE and call(T=0, x=None, ids=None, ws=None, wb=0) == DEVICE
        assert call(T=100, ws=None, wb=0) == DEVICE and call(loss=D + 36) == DEVICE


def test_route_grad_refusals(lib):  # noqa: F811
    def call(x=A, dt=0, T=4, E=8, st=8, ids=B, k=2, dw=C, n=D, dl=F, out=G):
        return lib.moe_route_grad(x, dt, T, E, st, ids, k, dw, 1, n, dl, out, None)
    assert call(dt=3) == INVALID and call(T=-1) == INVALID and call(E=1025, st=1025) == INVALID
    assert call(k=0) == INVALID and call(k=33) == INVALID and call(st=7) == INVALID
    assert call(x=None) == INVALID and call(out=None) == INVALID and call(ids=None) == INVALID
    assert call(dl=None) == INVALID and call(dw=None, n=None) == INVALID
    for name in ("ids", "dw", "n", "dl"):
        assert call(**{name: H + 2}) == MISALIGNED
    assert call(x=A + 1) == MISALIGNED and call(out=G + 2, dt=2) == MISALIGNED
    for other in (A, B, C, D, F):
        assert call(out=other) == INVALID
    assert call(T=0, x=None, out=None) == OK
    if not torch.cuda.is_available():
        assert call() == DEVICE and call(dw=None, ids=None) == DEVICE
        assert call(n=None, dl=None) == DEVICE


def test_combine_grad_refusals(lib):  # noqa: F811
    def call(dout=A, dt=0, T=2, N=8, Y=B, R=4, tok=C, pos=D, w=F, k=2, dY=G, dw=H):
        return lib.moe_combine_grad(dout, dt, T, N, Y, R, tok, pos, w, k, dY, dw, None)
    assert call(dt=2) == INVALID and call(dt=ROWS + 2) == INVALID and call(T=-1) == INVALID
    assert call(R=-1) == INVALID and call(N=-1) == INVALID and call(k=0) == INVALID and call(k=33) == INVALID
    for name in ("dout", "Y", "tok", "pos", "w", "dY", "dw"):
        assert call(**{name: None}) == INVALID and call(**{name: I + 1}) == MISALIGNED
    assert call(Y=B + 2, dt=ROWS) == MISALIGNED
    for other in (A, B, C, D, F):
        assert call(dY=other) == INVALID and call(dw=other) == INVALID
    assert call(dw=G + 60) == INVALID
    assert call(T=0, R=0, dY=None, dw=None) == OK
    if not torch.cuda.is_available():
        assert call() == DEVICE and call(dt=ROWS + 1) == DEVICE
        assert call(R=0, Y=None, tok=None, dY=None) == DEVICE and call(T=0, dout=None) == DEVICE


def test_binding_refuses_host_and_odd_tensors(lib):  # noqa: F811
    x = torch.zeros(4, 64, dtype=torch.float16)
    u, s = torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(8, 2, dtype=torch.uint8)
    i = torch.zeros(4, 2, dtype=torch.int32)
    for call in (lambda: mxfp4.linear_act(x, u, s), lambda: mxfp4.linear_act(x, u, s, activation="tanh"),
                 lambda: mxfp4.grouped_linear_act(x, u, s, i[0]),
                 lambda: mxfp4.activation_grad(x, x, "relu"), lambda: mxfp4.linear_grad(x, u, s),
                 lambda: mxfp4.grouped_linear_grad(x, u, s, i[0]), lambda: mxfp4.balance(x, i),
                 lambda: mxfp4.route_grad(x, i, x), lambda: mxfp4.combine_grad(x, x, i[0], i, x)):
        with pytest.raises(ValueError):
            call()


# ------------------------------------------------- the reference, by other means

@pytest.mark.parametrize("act", gref.ACTIVATIONS[:-1])
def test_reference_slopes_are_differences(act):
    z = np.linspace(-9, 9, 181) + 0.01                       # off the corner of relu
    h = 2.0 ** -13
    d = (gref.value(z + h, act) - gref.value(z - h, act)) / (2 * h)
    assert np.abs(gref.slope(z, act) - d).max() < h ** 2 + 1e-10


def test_reference_values_are_torch_s():
    z = torch.linspace(-9, 9, 181, dtype=torch.float64)
    nn = torch.nn.functional
    for act, f in (("relu", nn.relu), ("silu", nn.silu), ("gelu", nn.gelu),
                   ("gelu_tanh", lambda v: nn.gelu(v, approximate="tanh"))):
        assert np.abs(gref.value(z.numpy(), act) - f(z).numpy()).max() < 1e-12
    h, dy = torch.randn(5, 8, dtype=torch.float64, requires_grad=True), torch.randn(5, 4).double()
    (nn.silu(h[:, :4]) * h[:, 4:]).backward(dy)
    dz, _ = gref.activation_grad(dy.numpy(), h.detach().numpy(), "swiglu")
    assert np.abs(dz - h.grad.numpy()).max() < 1e-12


def test_reference_router_gradient_is_torch_s():
    x = torch.randn(6, 9, dtype=torch.float64, requires_grad=True)
    ids = torch.topk(x.detach(), 3).indices
    dw = torch.randn(6, 3, dtype=torch.float64)
    loss, counts = gref.balance(x.detach().numpy(), ids.numpy())
    p = torch.softmax(x, dim=1)
    want = 9 * ((torch.bincount(ids.flatten(), minlength=9).double() / 18) * p.mean(dim=0)).sum()
    assert abs(float(want.detach()) - loss) < 1e-12 and counts.sum() == 18 + 6
    for renormalize in (True, False):
        w = torch.softmax(x.gather(1, ids), dim=1) if renormalize else p.gather(1, ids)
        g, = torch.autograd.grad((w * dw).sum() + 0.7 * want, x, retain_graph=True)
        got, _ = gref.route_grad(x.detach().numpy(), ids.numpy(), dw.numpy(), renormalize, counts, 0.7)
        assert np.abs(got - g.numpy()).max() < 1e-12
