"""Workspaces and arguments of the products with coded matrices (not gpu): nothing here
reaches the GPU, fake pointers are never dereferenced."""
import pytest


@pytest.fixture(scope="module")
def ex():
    from exl3_trellis_weight_gb300 import build
    build.build()
    import exl3_trellis_weight_gb300 as ex
    ex.lib()
    return ex


@pytest.mark.parametrize("T", [0, 1, 64, 65, 700, 4096])
@pytest.mark.parametrize("rows,cols", [(512, 1024), (1024, 512), (128, 65536)])
@pytest.mark.parametrize("tr", [False, True])
@pytest.mark.parametrize("n,r", [(0, 0), (1, 1), (5, 48)])
def test_a_workspace_for_the_gradients_serves_the_product(ex, T, rows, cols, tr, n, r):
    grad, product = (f(T, rows, cols, tr, n, r) for f in (ex.linear_backward_workspace_bytes, ex.linear_workspace_bytes))
    assert grad >= product > 0
