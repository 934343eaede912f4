"""What no other row may see, at the sizes whose tokens take the persistent blocks with rings of row
copies (unsort and its gradients), which mask for themselves: dropped assignments that hold NaN and
infinities, places outside the rows, tokens and batches that keep nothing."""

import pytest
import torch

from tests import test_gpu_sort as sort

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def built():
    import mxfp4_expert_layer_gb300 as pkg
    pkg.build()


# tokens for several rounds of every resident block, by one group of rows and by two, by one chunk of
# columns and by several
SIZES = [(2500, 4, 2880, BF16), (2500, 9, 2880, F16), (2000, 3, 16384, F32), (16000, 2, 64, BF16)]


@pytest.mark.parametrize("T,k,H,dtype", SIZES)
def test_what_is_not_finite_stays_where_it_is(T, k, H, dtype):
    import mxfp4_expert_layer_gb300 as pkg
    E = 16
    idx = sort.routing(T, k, E, 0.4, seed=T)
    idx[5:9], idx[T - 1] = -1, -1  # tokens that keep nothing
    y, w, d = sort.rows_of(T * k, H, dtype, 1), torch.rand(T, k, device="cuda"), sort.rows_of(T, H, dtype, 3)
    s = pkg.sort_tokens(d, idx, E)
    gone = s.inv_perm < 0
    first = int(s.offsets[E])
    for bad in (NAN, INF):
        y[first:], w[gone] = bad, -bad
        out = pkg.unsort_tokens(y, s.inv_perm, w)
        sort.check_unsort(out, y, s.inv_perm, w)
        assert not out[gone.all(1)].any()
        g = pkg.unsort_tokens_backward(d, y, s.inv_perm, w)
        sort.check_unsort_grads(g, d, y, s.inv_perm, w)
        assert torch.isfinite(g.y.float()).all() and not g.y[first:].any() and not g.topk_w[gone].any()
        sort.check_unsort(pkg.sort_tokens_backward(y, s.inv_perm), y, s.inv_perm, None)
    live = int((~gone).any(1).nonzero()[-1])
    j = int((~gone[live]).nonzero()[0])
    y[int(s.inv_perm[live, j]), 3] = INF
    out = pkg.unsort_tokens(y, s.inv_perm, w)
    assert int((~torch.isfinite(out.float())).sum()) == 1 and out[live, 3] == INF
    d[live, 5] = NAN
    bad = ~torch.isfinite(pkg.unsort_tokens_backward(d, None, s.inv_perm, w, need_w=False).y.float())
    assert int(bad.sum()) == int((~gone[live]).sum()) and bad[int(s.inv_perm[live, j]), 5]


@pytest.mark.parametrize("T,k,H,dtype", SIZES)
def test_places_outside_the_rows(T, k, H, dtype):
    """Entries beyond the rows count as dropped, in either direction; the rows that they do not name
    are left as they were."""
    import mxfp4_expert_layer_gb300 as pkg
    L, n = pkg._lib, T * k
    inv = torch.randperm(n, generator=torch.Generator().manual_seed(1)).int().view(T, k).cuda()
    outside = torch.tensor([n, n + 5, 2 ** 31 - 1, -2 ** 31, -1 - n, -2 - n], dtype=torch.int32, device="cuda")
    at = torch.arange(0, n, 7, device="cuda")
    unnamed = inv.view(-1)[at].long()
    inv.view(-1)[at] = outside[torch.arange(at.numel(), device="cuda") % outside.numel()]
    clean = torch.where((inv >= 0) & (inv < n), inv, -1)
    y, w, d = sort.rows_of(n, H, dtype, 1), torch.rand(T, k, device="cuda"), sort.rows_of(T, H, dtype, 2)
    y[unnamed] = NAN
    sort.check_unsort(pkg.unsort_tokens(y, inv, w), y, clean, w)
    g = pkg.unsort_tokens_backward(d, y, inv, w)
    sort.check_unsort_grads(g._replace(y=None), d, y, clean, w)
    # d_y between two guards, every byte set before
    room = torch.full((n + 2, H), 7.0, dtype=dtype, device="cuda")
    code = {BF16: L.MOE_DTYPE_BF16, F16: L.MOE_DTYPE_F16, F32: L.MOE_DTYPE_F32}[dtype]
    L.check("moe_unsort_tokens_backward", L.moe_unsort_tokens_backward(
        d.data_ptr(), None, inv.data_ptr(), w.data_ptr(), T, k, H, code, room[1].data_ptr(), None,
        torch.cuda.current_stream().cuda_stream))
    assert (room[0] == 7).all() and (room[n + 1] == 7).all() and (room[1:n + 1][unnamed] == 7).all()
    named = torch.ones(n, dtype=torch.bool, device="cuda")
    named[unnamed] = False
    assert torch.equal(room[1:n + 1][named], g.y[named])


@pytest.mark.parametrize("T,k,H,dtype", SIZES)
def test_nothing_kept_and_all_on_one_expert(T, k, H, dtype):
    import mxfp4_expert_layer_gb300 as pkg
    E = 9
    x, y, w = sort.rows_of(T, H, dtype, 1), sort.rows_of(T * k, H, dtype, 2), torch.rand(T, k, device="cuda")
    for e in (-1, E, 0, E - 1):
        idx = torch.full((T, k), e, dtype=torch.int32, device="cuda")
        s = pkg.sort_tokens(x, idx, E)
        out, g = pkg.unsort_tokens(y, s.inv_perm, w), pkg.unsort_tokens_backward(x, y, s.inv_perm, w)
        sort.check_unsort(out, y, s.inv_perm, w)
        sort.check_unsort_grads(g, x, y, s.inv_perm, w)
        if not 0 <= e < E:
            assert int(s.offsets[E]) == 0 and not s.rows.any() and not out.any() and not g.y.any() and not g.topk_w.any()
