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
