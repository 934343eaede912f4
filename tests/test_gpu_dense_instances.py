"""Kernel variants of the dense operators that take a type, a row count, a width and an
argument pattern at once: the norms' persistent kernels in f16, absent arguments in wide
rows and long prompts, large f16 tiles of the feed-forward block, MXFP4 products of many
rows for several groups of tokens.  Bounds as in the operators' own files."""

import pytest
import torch

from tests import test_gpu_block_norm as norm
from tests import test_gpu_ffn as ffn
from tests import test_gpu_matvec as matvec

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32

ABSENT = [(False, True, True, "none"), (False, True, True, "token"), (True, False, True, "full"),
          (True, True, False, "feature"), (False, False, True, "feature"), (True, False, False, "token"),
          (False, True, False, "full"), (True, True, False, "none")]


@pytest.fixture(scope="module", autouse=True)
def built():
    import mxfp4_expert_layer_gb300 as pkg
    pkg.build()


@pytest.fixture(autouse=True)
def healthy(built):
    import mxfp4_expert_layer_gb300 as pkg
    yield
    assert pkg.dense_status() == 0


def absent(T, H, dtype, stream, gate, post, nxt, residual):
    """Forward and backward; without a residual the stream's type is that of the buffer given."""
    import mxfp4_expert_layer_gb300 as pkg
    m, a = norm.make(T, H, dtype, stream, gate, seed=T + H, post=post, nxt=nxt, residual=residual), 0.5
    s, y = norm.forward(m, a, residual_out=torch.empty(T, H, device="cuda", dtype=stream))
    norm.check_forward(m, a, s, y)
    grads = pkg.block_norm_backward(m["ds"], m["dy"], m["z"], s, norm_weight=m["w"], gate=m["g"], residual_scale=a,
                                    next_weight=m["v"], eps=norm.EPS, has_residual=residual)
    assert (grads.residual is None) == (not residual)
    if not residual:  # (the checker's formulas have one)
        grads = grads._replace(residual=(a * norm.ref_ds(m, s)).to(stream))
    norm.check_backward(m, a, s, grads)


@pytest.mark.parametrize("gate", ["none", "feature", "token", "full"])
@pytest.mark.parametrize("stream", [F16, F32])
@pytest.mark.parametrize("T,H", [(2001, 2880), (1300, 4096), (10007, 264), (18301, 8), (3801, 1536)])
def test_many_rows_of_f16(T, H, stream, gate):
    norm.both(norm.make(T, H, F16, stream, gate, seed=T), 0.7)


@pytest.mark.parametrize("gate", ["none", "feature", "token", "full"])
@pytest.mark.parametrize("T,H", [(2001, 2880), (10007, 264), (3801, 1536)])
def test_many_rows_of_bf16_in_an_f32_stream(T, H, gate):
    norm.both(norm.make(T, H, BF16, F32, gate, seed=T + 1), 0.7)


@pytest.mark.parametrize("post,nxt,residual,gate", ABSENT)
@pytest.mark.parametrize("T,H,dtype,stream", [(7, 4104, BF16, BF16), (700, 8192, BF16, F32), (700, 4104, F16, F16),
                                              (500, 8192, F16, F32)])
def test_absent_arguments_of_wide_rows(T, H, dtype, stream, post, nxt, residual, gate):
    """16 values a thread; more rows than the blocks' stages hold (152 blocks, up to three)."""
    absent(T, H, dtype, stream, gate, post, nxt, residual)


@pytest.mark.parametrize("post,nxt,residual,gate", ABSENT)
@pytest.mark.parametrize("T,H,dtype,stream", [(2500, 2880, BF16, BF16), (19, 320, F16, F32), (1300, 4096, F16, F16),
                                              (9000, 64, BF16, F32)])
def test_absent_arguments_of_long_prompts_and_other_types(T, H, dtype, stream, post, nxt, residual, gate):
    absent(T, H, dtype, stream, gate, post, nxt, residual)


@pytest.mark.parametrize("T,H", [(333, 2880), (600, 6000)])
def test_one_incoming_gradient_and_no_residual(T, H):
    """Nothing into the stream from downstream, or nothing into the next norm's output."""
    import mxfp4_expert_layer_gb300 as pkg
    for gone in ("ds", "v"):
        m = norm.make(T, H, BF16, BF16, "feature", seed=T, nxt=gone != "v")
        s, _ = norm.forward(m, 0.7)
        if gone == "ds":
            m["ds"] = None
        norm.check_backward(m, 0.7, s, pkg.block_norm_backward(m["ds"], m["dy"], m["z"], s, norm_weight=m["w"], gate=m["g"],
                                                               residual_scale=0.7, next_weight=m["v"], eps=norm.EPS))


@pytest.mark.parametrize("T,H,I,act", [(1001, 2880, 2880, "gelu"), (2048, 1024, 1032, "silu"), (257, 4104, 4096, "silu"),
                                       (4096, 264, 3000, "silu"), (1500, 2880, 1448, "gelu")])
def test_pair_tiles_of_f16(T, H, I, act):
    ffn.check(ffn.make(T, H, I, F16, seed=T), act)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("T", [5, 12, 30, 47, 64])
def test_many_weight_rows_for_several_groups_of_tokens(T, dtype, gated):
    """More row groups than blocks (several a block, the last round partial), one to two
    groups of up to 32 tokens; K with a tail inside its last unit."""
    matvec.check(matvec.make(T, 2 * 30010, 1632, dtype, seed=T), gated)
    matvec.check(matvec.make(T, 2 * 1001, 4000, dtype, seed=T), gated, "gelu")


@pytest.mark.parametrize("T", [3, 16, 100, 600])
def test_feed_forward_in_place(T):
    import mxfp4_expert_layer_gb300 as pkg
    m = ffn.make(T, 520, 1024, BF16, seed=T)
    want = pkg.ffn_forward(m["x"], m["wgu"], m["wd"])
    x = m["x"].clone()
    out, gu = pkg.ffn_forward(x, m["wgu"], m["wd"], out=x, save=True)
    assert out is x and torch.equal(x, want)
    assert torch.equal(gu, pkg.ffn_forward(m["x"], m["wgu"], m["wd"], save=True)[1])
