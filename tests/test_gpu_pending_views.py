"""Tensors whose conjugation or negation is pending (a flag of the tensor, not its memory's values):
refused by the operators that read memory, in place of an answer for other values."""

import pytest
import torch

from tests import test_gpu_sort as sort

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    import mxfp4_expert_layer_gb300 as pkg
    pkg.build()


@pytest.mark.parametrize("T", [20, 1500])
def test_conjugated_rows(T):
    import mxfp4_expert_layer_gb300 as pkg
    k, E, H = 2, 8, 16
    x, idx = torch.complex(sort.rows_of(T, H, F32, 1), sort.rows_of(T, H, F32, 2)), sort.routing(T, k, E, seed=3)
    with pytest.raises(ValueError, match="conj"):
        pkg.sort_tokens(x.conj(), idx, E)
    with pytest.raises(ValueError, match="conj"):
        pkg.sort_tokens(sort.rows_of(T, H, BF16, 1), idx, E, scales=x.conj())
    sort.check_sort(pkg.sort_tokens(x.conj().resolve_conj(), idx, E), x.conj().resolve_conj(), idx, E)


def test_negated_tensors():
    import mxfp4_expert_layer_gb300 as pkg
    T, k, E, H = 20, 2, 8, 16
    idx, y, w = sort.routing(T, k, E, seed=3), sort.rows_of(T * k, H, BF16, 1), torch.rand(T, k, device="cuda")
    x, weight = sort.rows_of(T, H, BF16, 2), sort.rows_of(24, H, BF16, 3)
    inv = sort.order(idx, E)[2]
    neg = torch._neg_view
    for call in (lambda: pkg.sort_tokens(neg(x), idx, E), lambda: pkg.unsort_tokens(neg(y), inv, w),
                 lambda: pkg.unsort_tokens(y, inv, neg(w)), lambda: pkg.unsort_tokens_backward(neg(x), y, inv, w),
                 lambda: pkg.linear_forward(neg(x), weight), lambda: pkg.linear_forward(x, neg(weight)),
                 lambda: pkg.unsort_tokens(y, inv, w, out=neg(x))):
        with pytest.raises(ValueError, match="neg"):
            call()
    sort.check_unsort(pkg.unsort_tokens(neg(y).resolve_neg(), inv, w), -y, inv, w)
