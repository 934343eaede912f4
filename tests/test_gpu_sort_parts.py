"""Scales of a part of a batch: rows of scales that begin at any byte, in and out."""

import pytest
import torch

from tests import test_gpu_sort as sort

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    import mxfp4_expert_layer_gb300 as pkg
    pkg.build()


@pytest.mark.parametrize("dtype,S", [(torch.uint8, 90), (F32, 1), (torch.uint8, 7), (BF16, 5), (torch.uint8, 128), (F32, 40)])
@pytest.mark.parametrize("T,k,E", [(61, 3, 16), (2100, 2, 32)])
def test_scales_of_a_part(T, k, E, dtype, S):
    import mxfp4_expert_layer_gb300 as pkg
    idx = sort.routing(T, k, E, 0.1, seed=T)
    codes, scales = sort.rows_of(T, 2880, torch.float8_e4m3fn, 1), sort.rows_of(T, S, dtype, 2)
    for a, b in ((1, T), (2, T), (3, 40), (20, T)):
        got = pkg.sort_tokens(codes[a:b], idx[a:b], E, scales=scales[a:b])
        sort.check_sort(got, codes[a:b], idx[a:b], E, scales[a:b])


@pytest.mark.parametrize("offset", [1, 2, 3, 4, 8])
@pytest.mark.parametrize("scale_bytes", [4, 6, 7, 90, 640])
@pytest.mark.parametrize("T", [50, 3000])
def test_scales_at_any_byte(T, scale_bytes, offset):
    """Through the C entry: both arrays of scales off their own alignment, and what is around the
    written one left as it was."""
    import mxfp4_expert_layer_gb300 as pkg
    L, k, E, H = pkg._lib, 2, 16, 32
    x, idx = sort.rows_of(T, H, BF16, 1), sort.routing(T, k, E, 0.1, seed=3)
    want = pkg.sort_tokens(x, idx, E)
    held = sort.rows_of(1, T * scale_bytes + offset, torch.uint8, 2)[0]
    scales = held[offset:].view(T, scale_bytes)
    for at in (0, offset):
        to = torch.full((T * k * scale_bytes + 16,), 77, dtype=torch.uint8, device="cuda")
        rows, offsets = torch.empty_like(want.rows), torch.empty_like(want.offsets)
        perm, inv = torch.empty_like(want.perm), torch.empty_like(want.inv_perm)
        L.check("moe_sort_tokens", L.moe_sort_tokens(
            x.data_ptr(), scales.data_ptr(), idx.data_ptr(), T, k, E, 2 * H, scale_bytes, offsets.data_ptr(), perm.data_ptr(),
            inv.data_ptr(), rows.data_ptr(), to.data_ptr() + at, torch.cuda.current_stream().cuda_stream))
        end = at + T * k * scale_bytes
        assert torch.equal(to[at:end].view(T * k, scale_bytes), sort.moved(scales, want.perm, k))
        assert (to[:at] == 77).all() and (to[end:] == 77).all() and torch.equal(perm, want.perm)
