"""Which workspace a product with an epilogue asks for, on the host: SwiGLU cannot run unsplit on
tiles of 64 x 128, and takes K slices where those would be fastest for other activations."""
import pytest

from test_mxfp4_host import lib  # noqa: F401


@pytest.mark.parametrize("M,N,K", [(64, 28672, 4096), (300, 4096, 4096), (100, 2048, 2048), (97, 130, 1376)])
def test_workspace_holds_the_slices_of_swiglu(lib, M, N, K):  # noqa: F811
    need = lib.mxfp4_linear_act_workspace_bytes(M, N, K)
    assert need > 0 and need % (M * N * 4) == 0 and need // (M * N * 4) > 1


@pytest.mark.parametrize("M,N,K", [(128, 4096, 256), (2000, 14336, 4096), (1, 4096, 14336), (16, 4096, 4096)])
def test_no_workspace_where_nothing_is_split(lib, M, N, K):  # noqa: F811
    assert lib.mxfp4_linear_act_workspace_bytes(M, N, K) == 0
