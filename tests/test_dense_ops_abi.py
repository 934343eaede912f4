"""CPU checks of the dense operators' entry points: what they refuse, before any launch."""

import pytest


@pytest.fixture(scope="module")
def L():
    import mxfp4_expert_layer_gb300 as pkg
    pkg.build()
    pkg._lib.load()
    return pkg._lib


FAKE = 1 << 20  # aligned, never dereferenced: every call below fails its checks first


def test_block_norm_refusals(L):
    def f(block=FAKE, nw=FAKE, gate=None, kind=0, res=FAKE, a=1.0, nxt=FAKE, eps=1e-5, T=4, H=64, dt=0, sdt=0, ro=2 * FAKE,
          out=FAKE):
        return L.moe_block_norm(block, nw, gate, kind, res, a, nxt, eps, T, H, dt, sdt, ro, out, None)
    for kw in (dict(T=0), dict(T=(1 << 24) + 1), dict(H=0), dict(H=12), dict(H=8200)):
        assert f(**kw) == L.MOE_ERR_UNSUPPORTED_SHAPE, kw
    for kw in (dict(block=None), dict(block=FAKE + 8), dict(nw=FAKE + 2), dict(nxt=FAKE + 8), dict(res=FAKE + 8),
               dict(ro=FAKE + 8), dict(out=FAKE + 8), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
               dict(a=float("inf")), dict(a=float("nan")), dict(dt=2), dict(dt=3), dict(sdt=1), dict(kind=4, gate=FAKE),
               dict(kind=1), dict(gate=FAKE), dict(kind=2, gate=FAKE + 2), dict(kind=3, gate=FAKE + 4), dict(out=None),
               dict(nxt=None), dict(nxt=None, out=None, ro=None), dict(ro=FAKE, out=FAKE)):
        assert f(**kw) == L.MOE_ERR_INVALID_ARG, kw


def test_block_norm_backward_refusals(L):
    ws = L.moe_block_norm_workspace_bytes(4, 64)
    assert ws == 1 * 3 * 64 * 4  # four narrow rows share a block
    assert L.moe_block_norm_workspace_bytes(100000, 4096) == 152 * 3 * 4096 * 4
    assert L.moe_block_norm_workspace_bytes(4, 60) == 0 and L.moe_block_norm_workspace_bytes(0, 64) == 0

    def f(ds=FAKE, dy=FAKE, z=FAKE, nw=FAKE, gate=None, kind=0, s=FAKE, nxt=FAKE, dz=FAKE, dr=FAKE, dw=FAKE, dg=None, dn=FAKE,
          w=FAKE, n=ws, T=4, H=64, dt=0, sdt=0):
        return L.moe_block_norm_backward(ds, dy, z, nw, gate, kind, s, 1.0, nxt, 1e-5, T, H, dt, sdt, dz, dr, dw, dg, dn, w, n,
                                         None)
    assert f(T=0) == L.MOE_ERR_UNSUPPORTED_SHAPE and f(H=8200) == L.MOE_ERR_UNSUPPORTED_SHAPE
    assert f(n=ws - 1) == L.MOE_ERR_WORKSPACE_TOO_SMALL
    for kw in (dict(ds=FAKE + 8), dict(dy=None), dict(nxt=None), dict(nxt=None, dy=None), dict(s=None), dict(z=None),
               dict(dz=None), dict(dz=FAKE + 8), dict(dr=FAKE + 4), dict(dw=FAKE + 4), dict(dn=FAKE + 4), dict(nw=None),
               dict(dg=FAKE), dict(gate=FAKE, kind=2, dg=FAKE + 2), dict(gate=FAKE, kind=1, dg=FAKE + 4), dict(w=None),
               dict(w=FAKE + 16), dict(ds=None, dy=None, nxt=None, dn=None), dict(dt=2)):
        assert f(**kw) == L.MOE_ERR_INVALID_ARG, kw


def test_matvec_sizes_and_refusals(L):
    DOWN, GU = L.MOE_WEIGHTS_DOWN, L.MOE_WEIGHTS_GATEUP
    # 1024 bytes of codes and 64 of scales per 16 rows x 128 codes, 16 per tile, tiles in eights, a 256-byte trailer
    assert L.moe_prepared_matvec_bytes(2880, 2880, DOWN) == (184 * (23 * 1088 + 16) + 255) // 256 * 256 + 256
    assert L.moe_prepared_matvec_bytes(130, 128, GU) == (16 * (1088 + 16) + 255) // 256 * 256 + 256  # 65 features: nine tiles
    assert L.moe_matvec_workspace_bytes(1, 2880) == 0                        # staged by the kernel itself
    assert L.moe_matvec_workspace_bytes(16, 4096) == 32 * 2 * 2048 + 256     # f16 values, 64 scales
    assert L.moe_matvec_workspace_bytes(33, 4000) == 2 * 32 * 4 * 2048 + 256  # two groups of 32 tokens
    assert L.moe_matvec_workspace_bytes(65, 4096) == 0 and L.moe_matvec_workspace_bytes(4, 4100) == 0
    for rows, K, kind in ((0, 64, DOWN), (8, 48, DOWN), (8, 0, DOWN), (7, 64, GU), (8, 64, 2), (8, 65536 + 32, DOWN),
                          ((1 << 22) + 1, 64, DOWN)):
        assert L.moe_prepared_matvec_bytes(rows, K, kind) == 0
        assert L.moe_prepare_matvec(FAKE, FAKE, rows, K, kind, FAKE, 1 << 40, None) == L.MOE_ERR_UNSUPPORTED_SHAPE
        assert L.moe_matvec_mxfp4(FAKE, FAKE, None, 1, rows, K, kind, 0, 0, FAKE, None, 0, None) == L.MOE_ERR_UNSUPPORTED_SHAPE
    assert L.moe_prepare_matvec(FAKE, FAKE, 32, 64, DOWN, FAKE, 16, None) == L.MOE_ERR_WORKSPACE_TOO_SMALL
    for a in ((None, FAKE, FAKE), (FAKE, None, FAKE), (FAKE, FAKE, None), (FAKE + 8, FAKE, FAKE), (FAKE, FAKE, FAKE + 16)):
        assert L.moe_prepare_matvec(a[0], a[1], 32, 64, DOWN, a[2], 1 << 20, None) == L.MOE_ERR_INVALID_ARG

    def f(x=FAKE, w=FAKE, b=None, T=1, act=0, dt=0, out=FAKE, K=64, ws=None, n=0):
        return L.moe_matvec_mxfp4(x, w, b, T, 32, K, DOWN, act, dt, out, ws, n, None)
    need = L.moe_matvec_workspace_bytes(16, 4096)
    assert f(T=16, K=4096, ws=FAKE, n=need - 1) == L.MOE_ERR_WORKSPACE_TOO_SMALL
    assert f(T=16, K=4096, ws=None, n=need) == L.MOE_ERR_INVALID_ARG
    assert f(T=16, K=4096, ws=FAKE + 16, n=need) == L.MOE_ERR_INVALID_ARG
    assert f(T=0) == L.MOE_ERR_UNSUPPORTED_SHAPE and f(T=65) == L.MOE_ERR_UNSUPPORTED_SHAPE
    for kw in (dict(x=None), dict(w=None), dict(out=None), dict(x=FAKE + 8), dict(w=FAKE + 16), dict(out=FAKE + 8),
               dict(b=FAKE + 2), dict(act=2), dict(dt=2)):
        assert f(**kw) == L.MOE_ERR_INVALID_ARG, kw


def test_wrappers_refuse_what_they_cannot_pass_on(L):
    import torch
    import mxfp4_expert_layer_gb300 as pkg
    z = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        pkg.block_norm(z)                                             # not on a GPU
    with pytest.raises(ValueError):
        pkg.block_norm(z.float())                                     # not a 16-bit type
    with pytest.raises(ValueError):
        pkg.block_norm(z, z.half())                                   # a stream of the other 16-bit type
    with pytest.raises(ValueError):
        pkg.block_norm(z, gate=torch.ones(4, 1, dtype=torch.bfloat16))  # a token gate is f32
    with pytest.raises(ValueError):
        pkg.block_norm(z, out=z)                                      # out without next_weight
    with pytest.raises(ValueError):
        pkg.block_norm(z.t())                                         # not contiguous
    with pytest.raises(L.MoEError):
        pkg.MatvecMXFP4(torch.zeros(4, 24, dtype=torch.uint8), torch.zeros(4, 1, dtype=torch.uint8))
