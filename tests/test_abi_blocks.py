"""Host-side checks of the block-scaled FP8, grouped and combine calls (no GPU
needed): bad arguments give the documented status before any launch, calls
with no rows do nothing, and the binding refuses tensors that do not fit."""
import ctypes

import pytest
import torch

FAKE = 1 << 20  # never dereferenced: every call below ends in its validation


@pytest.fixture(scope="module")
def m():
    import nvfp4_moe_skinny_amd as m
    return m


def test_quantize_rows_validation(m):
    def call(x=FAKE, t=0, M=4, K=256, ldx=256, swiglu=0, codes=FAKE, scales=FAKE):
        return m.lib.fp8_quantize_rows(x, t, M, K, ldx, swiglu, codes, scales, None)
    for kw in (dict(x=None), dict(codes=None), dict(scales=None)):
        assert call(**kw) == m.NVFP4MOE_ERR_NULL_ARG, kw
    for kw in (dict(t=2), dict(t=-1), dict(M=-1), dict(K=0), dict(K=-16), dict(ldx=255),
               dict(ldx=0), dict(swiglu=2, ldx=512), dict(swiglu=1, ldx=511)):
        assert call(**kw) == m.NVFP4MOE_ERR_BAD_SHAPE, kw
    for kw in (dict(K=24, ldx=24), dict(K=65552, ldx=65552), dict(M=(1 << 24) + 1),
               dict(M=1 << 60), dict(x=FAKE + 8), dict(codes=FAKE + 8), dict(scales=FAKE + 2),
               dict(ldx=260), dict(t=1, ldx=258), dict(M=1 << 20, K=65536, ldx=65536)):
        assert call(**kw) == m.NVFP4MOE_ERR_UNSUPPORTED, kw
    assert m.last_error_detail()
    assert call(M=0, x=None, codes=None, scales=None) == m.NVFP4MOE_OK
    assert m.last_error_detail() == ""


def test_quantize_blocks_validation(m):
    def call(x=FAKE, t=0, G=2, N=100, K=256, codes=FAKE, scales=FAKE):
        return m.lib.fp8_quantize_blocks(x, t, G, N, K, codes, scales, None)
    for kw in (dict(x=None), dict(codes=None), dict(scales=None)):
        assert call(**kw) == m.NVFP4MOE_ERR_NULL_ARG, kw
    for kw in (dict(t=2), dict(G=-1), dict(N=0), dict(K=0)):
        assert call(**kw) == m.NVFP4MOE_ERR_BAD_SHAPE, kw
    for kw in (dict(K=40), dict(K=1 << 17), dict(N=(1 << 20) + 1), dict(G=1 << 21),
               dict(G=1 << 20, N=1 << 20, K=65536), dict(G=4096, N=8192, K=8192),
               dict(x=FAKE + 4), dict(codes=FAKE + 4),
               dict(scales=FAKE + 1)):
        assert call(**kw) == m.NVFP4MOE_ERR_UNSUPPORTED, kw
    assert call(G=0, x=None, codes=None, scales=None) == m.NVFP4MOE_OK


def test_block_gemm_validation(m):
    def call(x=FAKE, xs=FAKE, M=4, K=256, w=FAKE, ws=FAKE, N=100, y=FAKE, t=0, ldy=100):
        return m.lib.fp8_block_gemm(x, xs, M, K, w, ws, N, y, t, ldy, None)
    for kw in (dict(x=None), dict(xs=None), dict(w=None), dict(ws=None), dict(y=None)):
        assert call(**kw) == m.NVFP4MOE_ERR_NULL_ARG, kw
    for kw in (dict(t=2), dict(M=-1), dict(N=0), dict(K=0), dict(ldy=99), dict(ldy=1 << 33)):
        assert call(**kw) == m.NVFP4MOE_ERR_BAD_SHAPE, kw
    for kw in (dict(K=8), dict(K=100), dict(K=65552), dict(N=(1 << 20) + 1, ldy=1 << 21),
               dict(M=(1 << 24) + 1), dict(x=FAKE + 8), dict(w=FAKE + 8), dict(xs=FAKE + 2),
               dict(ws=FAKE + 1), dict(y=FAKE + 1), dict(t=1, y=FAKE + 2),
               dict(M=1 << 24, N=1 << 20, ldy=1 << 20)):  # more tiles than a grid holds
        assert call(**kw) == m.NVFP4MOE_ERR_UNSUPPORTED, kw
    assert call(M=0, x=None, xs=None, w=None, ws=None, y=None) == m.NVFP4MOE_OK


def _args(m, **kw):
    a = m.GroupedArgs()
    for f in ("x", "x_scales", "w", "w_scales", "pairs", "active", "active_offsets", "n_active",
              "y"):
        setattr(a, f, FAKE)
    a.ldy, a.R, a.x_rows, a.pairs_per_row = 100, 32, 4, 8
    a.E, a.N, a.K, a.type, a.y_type = 64, 100, 256, m.NVFP4MOE_FP8, m.NVFP4MOE_BF16
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def test_grouped_validation(m):
    def call(**kw):
        return m.lib.moe_grouped_gemm(ctypes.byref(_args(m, **kw)), None)
    assert m.lib.moe_grouped_gemm(None, None) == m.NVFP4MOE_ERR_NULL_ARG
    for f in ("x", "x_scales", "w", "w_scales", "pairs", "active", "active_offsets", "n_active",
              "y"):
        assert call(**{f: None}) == m.NVFP4MOE_ERR_NULL_ARG, f
    for kw in (dict(type=1), dict(type=3), dict(y_type=2), dict(R=-1), dict(x_rows=-1),
               dict(pairs_per_row=0), dict(E=0), dict(N=0), dict(K=0), dict(ldy=99),
               dict(x_rows=3), dict(pairs_per_row=7)):
        assert call(**kw) == m.NVFP4MOE_ERR_BAD_SHAPE, kw
    for kw in (dict(K=8), dict(K=1 << 17), dict(E=1025), dict(R=1 << 24, x_rows=1 << 24),
               dict(x_rows=(1 << 24) + 1), dict(pairs_per_row=1 << 60), dict(x=FAKE + 8),
               dict(w=FAKE + 8), dict(w_scales=FAKE + 2), dict(pairs=FAKE + 2),
               dict(n_active=FAKE + 1), dict(y=FAKE + 1), dict(y_type=1, y=FAKE + 2),
               dict(R=(1 << 24) - 1, x_rows=1 << 24, N=1 << 20, ldy=1 << 20)):
        assert call(**kw) == m.NVFP4MOE_ERR_UNSUPPORTED, kw
    assert call(R=0, x=None, w=None, y=None, pairs=None) == m.NVFP4MOE_OK
    # a BF16 product needs no scales (validated up to its alignment check)
    assert call(type=0, x_scales=None, w_scales=None, y=FAKE + 1) == m.NVFP4MOE_ERR_UNSUPPORTED


def test_combine_validation(m):
    def call(y=FAKE, t=0, w=FAKE, shared=None, residual=None, M=4, k=8, H=64, out=FAKE):
        return m.lib.moe_combine(y, t, w, shared, residual, M, k, H, out, None)
    for kw in (dict(y=None), dict(w=None), dict(out=None)):
        assert call(**kw) == m.NVFP4MOE_ERR_NULL_ARG, kw
    for kw in (dict(t=2), dict(M=-1), dict(k=0), dict(H=0)):
        assert call(**kw) == m.NVFP4MOE_ERR_BAD_SHAPE, kw
    for kw in (dict(k=9), dict(M=(1 << 24) + 1), dict(H=(1 << 20) + 1),
               dict(M=1 << 16, H=(1 << 15) + 1),
               dict(y=FAKE + 1), dict(t=1, y=FAKE + 2), dict(w=FAKE + 2), dict(shared=FAKE + 1),
               dict(residual=FAKE + 1), dict(out=FAKE + 1)):
        assert call(**kw) == m.NVFP4MOE_ERR_UNSUPPORTED, kw
    assert call(M=0, y=None, w=None, out=None) == m.NVFP4MOE_OK


def test_binding_refuses_what_does_not_fit(m):
    """Shape, type and device checks come before anything reaches the library."""
    bf, u8, f32 = torch.bfloat16, torch.uint8, torch.float32
    z = torch.zeros
    rows = m.Fp8Rows(z((4, 256), dtype=u8), z((2, 4)))
    blocks = m.Fp8Blocks(z((1, 100, 256), dtype=u8), z((1, 1, 2)))
    for bad in (lambda: m.fp8_quantize_rows(z((4, 256), dtype=bf)),             # on the CPU
                lambda: m.fp8_quantize_rows(z((4, 256), dtype=torch.float16)),
                lambda: m.fp8_quantize_rows(z((256,), dtype=bf)),
                lambda: m.fp8_quantize_rows(z((4, 33), dtype=bf), swiglu=True),
                lambda: m.fp8_quantize_rows(z((256, 4), dtype=bf).t()),         # columns strided
                lambda: m.fp8_quantize_rows(z((1, 256), dtype=bf).expand(4, 256)),
                lambda: m.fp8_quantize_blocks(z((2, 3, 4, 16), dtype=bf)),
                lambda: m.fp8_block_gemm(rows, blocks),                          # on the CPU
                lambda: m.fp8_block_gemm(rows, m.Fp8Blocks(z((1, 100, 240), dtype=u8),
                                                           z((1, 1, 2)))),
                lambda: m.fp8_block_gemm(rows, m.Fp8Blocks(z((2, 100, 256), dtype=u8),
                                                           z((2, 1, 2)))),
                lambda: m.fp8_block_gemm(m.Fp8Rows(rows.codes, z((4, 2))), blocks),
                lambda: m.fp8_block_gemm(rows, blocks, out_dtype=torch.float16),
                lambda: m.moe_combine(z((32, 64), dtype=bf), z((5, 8)))):
        with pytest.raises(ValueError):
            bad()
    r = m.Routing(z((4, 8), dtype=torch.int32), z((4, 8)), *[None] * 6)
    with pytest.raises(ValueError):  # FP8 rows with BF16 weights
        m.moe_grouped_gemm(rows, r, z((64, 100, 256), dtype=bf))
    with pytest.raises(ValueError):  # neither 4 token rows nor 32 pair rows
        m.moe_grouped_gemm(z((5, 256), dtype=bf), r, z((64, 100, 256), dtype=bf))
