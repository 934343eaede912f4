"""The norm's codes with a row scale, value by value, as the header states them: scale = max |y| (1 / 448),
code = E4M3(y (1 / scale)), where 1 / 448, 1 / scale and both products are rounded to f32.  With s = 1
in every place and eps = 0 both norms divide by 1, and y is next_weight itself.  The weights are ties
between two codes of the exact quotient, values next to ties, and random ones; T takes the kernel of a
block per row and that of many rows."""

import pytest
import torch

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    import mxfp4_expert_layer_gb300 as pkg
    pkg.build()


def check(v, T):
    """v: [H] of a 16-bit type, on the CPU."""
    import mxfp4_expert_layer_gb300 as pkg
    H = v.numel()
    one, w = torch.ones(T, H, dtype=v.dtype, device="cuda"), torch.ones(H, dtype=v.dtype, device="cuda")
    n = pkg.block_norm_8bit(one, one, norm_weight=w, residual_scale=0.0, next_weight=v.cuda(), eps=0.0, scales="row")
    assert (n.residual == 1).all()
    y = v.float()
    scale = torch.clamp(y.abs().amax() * (1 / torch.tensor(448.0)), min=2.0 ** -126)
    code = (y * (1 / scale)).to(torch.float8_e4m3fn).view(torch.uint8)
    # three roundings of 2^-24 from the quotient of the exact scale, and another code than its only next to a tie:
    # within them of half a step (2^-10 among the subnormal codes)
    exact = y.double() * 448 / y.abs().amax().double()
    if scale > 2.0 ** -126:
        step = torch.exp2(torch.floor(torch.log2(exact.abs().clamp(min=2.0 ** -6))) - 3)
        assert ((code.view(torch.float8_e4m3fn).double() - exact).abs() <= step / 2 + 4 * 2.0 ** -24 * exact.abs()).all()
    assert (n.scales == scale.item()).all(), (n.scales[0].item(), scale.item())
    for got in (n.codes.view(torch.uint8)[0].cpu(), n.codes.view(torch.uint8)[-1].cpu()):
        bad = (got != code).nonzero().flatten()[:4]
        assert not bad.numel(), [(y[i].item(), scale.item(), got[i].item(), code[i].item()) for i in bad]
    assert (n.codes.view(torch.uint8) == n.codes.view(torch.uint8)[0]).all()


SIZES = [(1, 2880), (1, 512), (1900, 2880), (9800, 512)]


@pytest.mark.parametrize("T,H", SIZES)
def test_ties(T, H):
    """Largest value 7 q: the scale is q / 64 or next to it, and t q / 64 is halfway between two codes
    for the odd t from 17 to 31 and, among the subnormal codes, for odd t 2^-10 with t up to 15.  The
    neighbours of these values in their type are next to the ties."""
    ties = [t * 2.0 ** e for t in range(17, 32, 2) for e in (-7, -3, 0, 3)] + [t * 2.0 ** -10 for t in range(1, 16, 2)]
    for q in range(1, 66, 2 if T == 1 else 16):
        at = torch.tensor([t * q / 64 for t in ties], dtype=torch.float64)
        v = at.to(F16)
        assert (v.double() == at).all()
        near = torch.cat([v, (v.view(torch.int16) + 1).view(F16), (v.view(torch.int16) - 1).view(F16)])
        near = torch.cat([near, -near])
        v = near.repeat(H // near.numel() + 1)[:H].clone()
        v[v.abs() > 7 * q] = 0
        v[H // 2], v[5] = 7 * q, -0.0
        check(v, T)


@pytest.mark.parametrize("dtype,size", [(F16, 1.0), (BF16, 1.0), (BF16, 3e37), (BF16, 1e-20), (BF16, 1e-24), (BF16, 1e-25), (BF16, 1e-30),
                                        (BF16, 1e-34), (BF16, 1e-37), (BF16, 1e-39)])
@pytest.mark.parametrize("T,H", SIZES)
def test_random_values(T, H, dtype, size):
    """Of every magnitude, scales at the least one among them."""
    for seed in range(6):
        g = torch.Generator().manual_seed(seed)
        spread = torch.exp2(-12 * torch.rand(H, generator=g)) if seed % 2 else 1.0
        check((torch.randn(H, generator=g) * spread * size).to(dtype), T)
