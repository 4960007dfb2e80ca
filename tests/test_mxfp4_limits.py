"""Sizes past what the MXFP4 kernels' launches and index types hold are refused on the host."""
import ctypes as C


def test_sizes_past_the_limits():
    import fine_grained_blockwise_amd as fgb
    L, f = fgb.lib(), C.c_void_p(0x1000)

    def qt(dt, rows, cols, G=1):
        return L.mxfp4_quant_t(f, dt, G, rows, cols, cols, 0, f, f, f, f, None)
    assert qt(0, 4, 1 << 30) == 1 and b"2^30" in L.fgb_last_error()
    assert qt(0, 1 << 23, 64) == 1 and qt(1, 4, 64, G=1 << 16) == 1

    def g(M, N, K):
        return L.mxfp4_gemm(f, f, 2, f, f, M, N, K, K // 2, K // 2, f, 1, N, 0, None)
    assert g(1 << 31, 64, 64) == 1 and g(4, 1 << 29, 64) == 1 and g(4, 64, 1 << 23) == 1
    assert L.mxfp4_grouped_gemm(f, f, 2, f, f, f, 4, 64, 1 << 29, 64, f, 1, None) == 1


def test_the_kernel_that_a_product_takes():
    """The choice, by sizes: a row, a decode batch and a small prompt on the kernel for few rows; a long prompt, a
    training step and a full expert batch on tiles; nothing to compute and what is refused on neither."""
    import fine_grained_blockwise_amd as fgb
    for fmt in (fgb.E2M1, fgb.E4M3):
        for M, N, K, G in ((1, 2048, 7168, 0), (64, 28672, 8192, 0), (77, 2112, 1536, 0), (488, 4096, 7168, 32),
                           (0, 64, 128, 0), (64, 0, 128, 0), (64, 64, 0, 0)):
            assert not fgb.mxfp4_gemm_tiled(M, N, K, a_fmt=fmt, groups=G)
        for M, N, K, G in ((4096, 28672, 8192, 0), (8192, 2048, 7168, 0), (8192, 7168, 2048, 0), (131552, 4096, 7168, 32)):
            assert fgb.mxfp4_gemm_tiled(M, N, K, a_fmt=fmt, groups=G)
    assert not fgb.mxfp4_gemm_tiled(4096, 4096, 4100) and not fgb.mxfp4_gemm_tiled(4096, 4096, 4096, a_fmt=fgb.E5M2)
    assert not fgb.mxfp4_gemm_tiled(4096, 4096, 4096, groups=-1)
