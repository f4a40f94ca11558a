"""Argument checks of the FP8 and grouped products (no GPU: every call here returns before any launch)."""
import pytest

from expert_cached_ffn_amd import _lib, ops


def _err(fn, *a, **kw):
    with pytest.raises(ops.FtError) as e:
        fn(*a, stream=0, **kw)
    return e.value.status


EINVAL, ENOTSUP = _lib.FT_EINVAL, _lib.FT_ENOTSUP
BF16, F32, FP8 = _lib.FT_BF16, _lib.FT_F32, _lib.FT_FP8


def test_fp8_layout():
    L = ops.ft_expert_layout_init(FP8, 4096, 2048)
    assert (L.off_gate, L.off_up, L.off_down) == (0, 8_388_608, 16_777_216)
    assert (L.off_sgate, L.off_sup, L.off_sdown) == (25_165_824, 25_167_872, 25_169_920)  # 32 x 16 fp32 each
    assert L.expert_bytes == 25_174_016 and L.off_tscale == 0
    L = ops.ft_expert_layout_init(FP8, 208, 144)       # partial blocks: 2 x 2 scales, 256-byte parts
    assert L.off_up == 29_952 and L.off_sgate == 3 * 29_952 and L.off_sup == L.off_sgate + 256
    for bad in [(FP8, 200, 64), (FP8, 64, 40)]:
        assert _err_layout(*bad) == EINVAL


def _err_layout(*a):
    with pytest.raises(ops.FtError) as e:
        ops.ft_expert_layout_init(*a)
    return e.value.status


def test_workspace_holds_the_fp8_stages():
    T, k, H, I = 33, 8, 2048, 768
    rows = T * k + T
    need = rows * I * 4 + rows * I + T * H
    assert ops.ft_workspace_bytes(_lib.FT_WS_FFN, T, k, 128, H, I) >= need


def test_quantize_refusals():
    f = ops.ft_fp8_quantize
    ok = dict(x=16, x_dtype=BF16, ldx=128, n=4, K=128, block_rows=1, codes=16, ldc=128, scales=16)

    def err(**kw):
        return _err(f, **{**ok, **kw})

    assert err(x_dtype=FP8) == EINVAL
    assert err(block_rows=64) == EINVAL
    assert err(n=-1) == EINVAL
    assert err(K=120) == ENOTSUP
    assert err(ldx=112) == EINVAL and err(ldc=112) == EINVAL
    assert err(ldx=132) == EINVAL and err(ldc=136) == EINVAL
    assert err(x=None) == EINVAL and err(codes=None) == EINVAL and err(scales=None) == EINVAL
    assert err(x=8) == EINVAL and err(codes=8) == EINVAL and err(scales=2) == EINVAL
    assert err(n=1 << 31) == ENOTSUP
    f(None, BF16, 128, 0, 128, 1, None, 128, None, stream=0)   # n = 0
    f(None, F32, 0, 5, 0, 128, None, 0, None, stream=0)        # K = 0


def test_launch_limits():
    # one launch holds 2^32 threads: 2^28 blocks of a quantizer's rows, 2^23 of the largest tiles
    assert _err(ops.ft_fp8_quantize, 16, BF16, 128, (1 << 28) - 16, 128, 1, 16, 128, 16) == ENOTSUP
    assert _err(ops.ft_fp8_quantize, 16, BF16, 1 << 24, 1 << 15, 1 << 24, 1, 16, 1 << 24, 16) == ENOTSUP
    assert _err(ops.ft_fp8_gemm, 16, 16, 16, 16, 16, 16, (1 << 31) - 513, 4096, 16, BF16, 16, 4096) == ENOTSUP


def test_workspace_of_other_weights_unchanged():
    """FP8's FFN needs more than the others': their calls are not held to it.  (x is misaligned: nothing is launched.)"""
    T, k, E, H, I = 600, 8, 128, 2048, 768
    rows = T * (k + 1)
    assert rows * I * 4 <= ops.ft_noalloc_scratch_bytes() < rows * I * 5
    f = ops.ft_moe_grouped_ffn_noalloc
    for wdtype, scratch in ((1, True), (FP8, False)):
        L = ops.ft_expert_layout_init(wdtype, H, I)
        got = _err(f, L, 256, None, None, 8, BF16, T, k, E, 256, 256, 256, None, 0, n_slots=E)
        assert (got != -3) == scratch


def test_gemm_refusals():
    f = ops.ft_fp8_gemm
    ok = dict(a=16, lda=256, a_scales=16, w=16, ldw=256, w_scales=16, M=4, N=8, K=256, out_dtype=BF16, out=16, ldo=8)

    def err(**kw):
        return _err(f, **{**ok, **kw})

    assert err(out_dtype=FP8) == EINVAL
    assert err(K=0) == EINVAL and err(M=-1) == EINVAL and err(N=-1) == EINVAL
    assert err(K=250) == ENOTSUP
    assert err(lda=240) == EINVAL and err(ldw=240) == EINVAL and err(ldo=7) == EINVAL
    assert err(lda=264) == EINVAL and err(ldw=264) == EINVAL
    assert err(lda=(4 << 20) + 16) == ENOTSUP and err(ldw=(4 << 20) + 16) == ENOTSUP
    assert err(M=(1 << 31) - 512) == ENOTSUP
    for p in ("a", "a_scales", "w", "w_scales", "out"):
        assert err(**{p: None}) == EINVAL, p
    for p in ("a", "w", "out"):
        assert err(**{p: 8}) == EINVAL, p
    f(None, 256, None, None, 256, None, 0, 8, 256, BF16, None, 8, stream=0)
    f(None, 256, None, None, 256, None, 4, 0, 256, BF16, None, 0, stream=0)


def test_grouped_refusals():
    f = ops.ft_grouped_gemm
    ok = dict(dtype=FP8, a=16, lda=256, a_scales=16, slot_pool=256, expert_bytes=4096, off_w=0, off_s=2048, n_slots=8,
              slot_of_expert=None, T=4, k=2, E=8, expert_offsets=16, sorted_rows=16, N=8, K=256, out_dtype=BF16, out=16, ldo=8)

    def err(**kw):
        return _err(f, **{**ok, **kw})

    assert err(dtype=F32) == EINVAL and err(out_dtype=FP8) == EINVAL
    assert err(k=0) == EINVAL and err(E=0) == EINVAL and err(T=-1) == EINVAL and err(N=-1) == EINVAL and err(K=0) == EINVAL
    assert err(E=4097, n_slots=5000) == ENOTSUP
    assert err(K=248, lda=256) == ENOTSUP and err(dtype=BF16, K=252, lda=256) == ENOTSUP
    assert err(T=1 << 30, k=2) == EINVAL
    assert err(lda=240) == EINVAL and err(ldo=7) == EINVAL and err(lda=264) == EINVAL
    assert err(lda=(4 << 20) + 16) == ENOTSUP
    assert err(T=1 << 20, lda=4096, k=1) == ENOTSUP        # gathered rows of 4 GiB
    assert err(n_slots=7) == EINVAL and err(n_slots=0, slot_of_expert=16) == EINVAL
    for p in ("a", "a_scales", "slot_pool", "expert_offsets", "out"):
        assert err(**{p: None}) == EINVAL, p
    assert err(a=8) == EINVAL and err(out=8) == EINVAL and err(slot_pool=8) == EINVAL
    assert err(expert_bytes=4104) == EINVAL and err(off_w=8) == EINVAL and err(off_s=2050) == EINVAL
    assert err(off_w=2064) == EINVAL        # weights past the slot's end
    assert err(off_s=4092) == EINVAL        # 1 x 2 scales past it
    assert err(off_w=4112) == EINVAL and err(off_s=4100) == EINVAL
    f(FP8, None, 256, None, None, 4096, 0, 2048, 8, None, 0, 2, 8, None, None, 8, 256, BF16, None, 8, stream=0)


def test_ffn_refusals():
    f = ops.ft_moe_grouped_ffn
    L = ops.ft_expert_layout_init(FP8, 512, 256)
    ok = dict(workspace=256, workspace_bytes=1 << 30)
    assert _err(f, L, 256, None, None, 256, F32, 1, 2, 8, 256, 256, 256, None, 0, **ok) == EINVAL       # x dtype
    assert _err(f, L, 256, None, None, 256, BF16, 1, 2, 8, 256, 256, 256, None, 1, **ok) == ENOTSUP     # native MX mode
    assert _err(f, L, 256, None, None, 256, BF16, 1, 2, 8, 256, 256, 256, None, 0, workspace=256, workspace_bytes=64) == EINVAL
    from ctypes import c_float
    buf = (c_float * 512)()
    import ctypes
    with pytest.raises(ops.FtError) as e:      # the host expert kernel has no FP8 path
        ops.ft_cpu_expert_ffn(L, ctypes.addressof(buf), ctypes.addressof(buf), 1, ctypes.addressof(buf))
    assert e.value.status == ENOTSUP
