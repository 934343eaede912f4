"""CPU check of the projections' workspace: what no call of these sizes writes is not asked for."""

import pytest


@pytest.fixture(scope="module")
def L():
    import mxfp4_expert_layer_gb300 as pkg
    pkg.build()
    pkg._lib.load()
    return pkg._lib


@pytest.mark.parametrize("T,K,N", [(1, 4096, 14336), (16, 2880, 32768), (32, 4096, 14336), (64, 2880, 2880), (64, 4096, 14336)])
def test_backward_of_a_batch(L, T, K, N):
    """The gradient into x of a batch joins its K slices in shared memory, and the weights' has one
    or two groups of K, which are not split: dp (16 bits) and up to 64 rows of the bias gradient's
    partial sums are all."""
    dp, sums = 2 * T * N, 4 * N * 64
    assert dp <= L.moe_linear_workspace_bytes(T, K, N, 1) <= dp + 256 + sums + 256
