"""CPU checks of the operators around experts of one's own: outputs that overlap one another, and a
workspace that overlaps any array, are refused before any launch; arrays that only meet are not.
(A call that passes its checks ends here with MOE_ERR_CUDA: there is no GPU, and nothing is read.)"""

import pytest

FAKE = 1 << 24  # aligned, never dereferenced
FAR = 1 << 36   # arrays that do not overlap those at FAKE


@pytest.fixture(scope="module")
def L():
    import torch
    if torch.cuda.is_available():
        pytest.skip("calls that pass their checks would launch on these addresses")
    import mxfp4_expert_layer_gb300 as pkg
    pkg.build()
    pkg._lib.load()
    return pkg._lib


def at(i):
    return FAR + i * FAKE


def pairs(L, call, sizes, launched=True):
    """call(**{name: address}) with each pair of `sizes` overlapping by a little at either end, and
    with the two meeting."""
    place = {name: at(i) for i, name in enumerate(sizes)}
    assert call(**place) == L.MOE_ERR_CUDA
    for a in sizes:
        for b in sizes:
            if a == b:
                continue
            step = 256 if "ws" in (a, b) else 16
            inside = (sizes[a] - 1) // step * step  # the last aligned place in a
            assert call(**dict(place, **{b: place[a] + inside})) == L.MOE_ERR_INVALID_ARG, (a, b)
            assert call(**dict(place, **{b: place[a]})) == L.MOE_ERR_INVALID_ARG, (a, b)
            behind = -(-sizes[a] // step) * step
            assert call(**dict(place, **{b: place[a] + behind})) == L.MOE_ERR_CUDA, (a, b)


@pytest.mark.parametrize("T,k,E", [(4, 2, 8), (3000, 4, 32)])
def test_sort(L, T, k, E):
    n = T * k

    def call(offsets, perm, inv, rows, row_scales):
        return L.moe_sort_tokens(FAKE, 2 * FAKE, 3 * FAKE, T, k, E, 64, 4, offsets, perm, inv, rows, row_scales, None)
    pairs(L, call, dict(offsets=4 * (E + 1), perm=4 * n, inv=4 * n, rows=64 * n, row_scales=4 * n))


def test_unsort_backward(L):
    def call(dy, dw):
        return L.moe_unsort_tokens_backward(FAKE, 2 * FAKE, 3 * FAKE, 4 * FAKE, 4, 2, 64, 0, dy, dw, None)
    pairs(L, call, dict(dy=1024, dw=32))


@pytest.mark.parametrize("T,K,N", [(4, 64, 32), (160, 256, 512)])
def test_linear_backward(L, T, K, N):
    ws = L.moe_linear_workspace_bytes(T, K, N, 1)
    sizes = dict(dx=2 * T * K, dw=2 * N * K, db=4 * N, ws=ws)

    def call(dx, dw, db, ws, d=FAKE, x=2 * FAKE, w=3 * FAKE, pre=4 * FAKE):
        return L.moe_linear_backward(d, x, w, pre, T, K, N, 0, 0, 0, dx, dw, db, ws, sizes["ws"], None)
    pairs(L, call, sizes)
    place = {name: at(i) for i, name in enumerate(sizes)}
    for name in ("d", "x", "w", "pre"):
        assert call(**dict(place, **{name: place["ws"] + sizes["ws"] // 256 * 256 - 256})) == L.MOE_ERR_INVALID_ARG, name


def test_linear_forward(L):
    T, K, N = 160, 16384, 1024
    need = L.moe_linear_workspace_bytes(T, K, N, 0)
    assert need > 0
    place = dict(x=at(0), w=at(1), b=at(4), r=at(5), pre=at(6), out=at(7), ws=at(8))

    def call(x, w, b, r, pre, out, ws):
        return L.moe_linear_forward(x, w, b, r, T, K, N, 0, 0, 0, pre, out, ws, need, None)
    assert call(**place) == L.MOE_ERR_CUDA
    assert call(**dict(place, out=place["r"])) == L.MOE_ERR_CUDA
    for name in place:
        if name != "ws":
            assert call(**dict(place, ws=place[name])) == L.MOE_ERR_INVALID_ARG, name
            assert call(**dict(place, **{name: place["ws"] + (need - 1) // 256 * 256})) == L.MOE_ERR_INVALID_ARG, name
