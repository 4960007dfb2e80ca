// gemm.hip -- the FP8 GEMM entry points: argument checks and the choice of the
// kernel's instantiation (gemm_kernel.h holds the kernel and its description).
#include "gemm_kernel.h"

namespace fgb {

template <int MODE, int GK>
static int dispatch_mode(int ag, int bg, bool bf16, const GemmArgs &p, int64_t grid, hipStream_t st)
{
    if constexpr (GK == GK_M || GK == GK_MM) {
        if (ag == AG_ROW128 && bg == BG_BLOCK)
            return launch_out<MODE, AG_ROW128, BG_BLOCK, GK>(bf16, p, grid, st);
    } else if constexpr (GK == GK_K) {
        if (ag == AG_ROW128 && bg == BG_ROW128)
            return launch_out<MODE, AG_ROW128, BG_ROW128, GK_K>(bf16, p, grid, st);
    } else {
        if (ag == AG_ROW128 && bg == BG_BLOCK)
            return launch_out<MODE, AG_ROW128, BG_BLOCK, GK_NONE>(bf16, p, grid, st);
        if (ag == AG_ROW128 && bg == BG_ROW128)
            return launch_out<MODE, AG_ROW128, BG_ROW128, GK_NONE>(bf16, p, grid, st);
        if (ag == AG_ROW32 && bg == BG_ROW32)
            return launch_out<MODE, AG_ROW32, BG_ROW32, GK_NONE>(bf16, p, grid, st);
    }
    return set_error(FGB_EUNSUPPORTED, "gemm: unsupported scale granularity pair (%d, %d)", ag, bg);
}

template <int GK>
static int dispatch(int mode, int ag, int bg, bool bf16, const GemmArgs &p, int64_t grid, hipStream_t st)
{
    if (mode == FGB_GEMM_FAST)
        return dispatch_mode<MODE_FAST, GK>(ag, bg, bf16, p, grid, st);
    return dispatch_mode<MODE_EXACT, GK>(ag, bg, bf16, p, grid, st);
}

// E5M2 A operand (gradients): dense, 1x128 A scales, 128x128 or 1x128 B scales.
template <int MODE>
static int dispatch_e5m2_mode(int bg, bool bf16, const GemmArgs &p, int64_t grid, hipStream_t st)
{
    if (bg == BG_BLOCK)
        return launch_out<MODE, AG_ROW128, BG_BLOCK, GK_NONE, FMT_E5M2>(bf16, p, grid, st);
    return launch_out<MODE, AG_ROW128, BG_ROW128, GK_NONE, FMT_E5M2>(bf16, p, grid, st);
}

} // namespace fgb

using namespace fgb;

extern "C" int fp8_block_gemm_fmt(const uint8_t *a, const uint8_t *sa, int a_gran, int a_fmt, const uint8_t *b,
                                  const uint8_t *sb, int b_gran, int b_fmt, const float *b_l1, int64_t g1, int64_t M,
                                  int64_t N, int64_t K, int64_t lda, int64_t ldb, void *d, int d_dtype, int64_t ldd,
                                  int accumulate, int mode, void *stream)
{
    clear_error();
    FGB_REQUIRE(a_fmt == FGB_E4M3 || a_fmt == FGB_E5M2, FGB_EUNSUPPORTED,
                "fp8_block_gemm: a_fmt must be FGB_E4M3 or FGB_E5M2");
    FGB_REQUIRE(b_fmt == FGB_E4M3, FGB_EUNSUPPORTED, "fp8_block_gemm: b_fmt must be FGB_E4M3");
    FGB_REQUIRE(a_fmt == FGB_E4M3 || (a_gran == FGB_ROW1x128 && b_gran != FGB_ROW1x32 && !b_l1), FGB_EUNSUPPORTED,
                "fp8_block_gemm: an E5M2 A needs 1x128 A scales, 128x128 or 1x128 B scales and no b_l1");
    FGB_REQUIRE(M >= 0 && N >= 0 && K >= 0 && K % 128 == 0, FGB_EINVAL,
                "fp8_block_gemm: need M, N >= 0 and K a multiple of 128 (M=%lld N=%lld K=%lld)",
                (long long)M, (long long)N, (long long)K);
    // Empty D: nothing to write (the operands may be empty tensors without storage).
    if (M == 0 || N == 0)
        return FGB_OK;
    FGB_REQUIRE(d && (K == 0 || (a && sa && b && sb)), FGB_EINVAL, "fp8_block_gemm: null pointer");
    // (with K = 0 no operand is read: their layouts are not checked)
    FGB_REQUIRE(K == 0 || (lda >= K && ldb >= K && lda % 16 == 0 && ldb % 16 == 0), FGB_EINVAL,
                "fp8_block_gemm: lda/ldb must be >= K and multiples of 16");
    FGB_REQUIRE(K == 0 || (256 * lda < (1ll << 32) && 256 * ldb < (1ll << 32)), FGB_EINVAL,
                "fp8_block_gemm: lda/ldb too large");
    FGB_REQUIRE(ldd >= N, FGB_EINVAL, "fp8_block_gemm: ldd must be >= N");
    FGB_REQUIRE(K == 0 || (aligned16(a) && aligned16(b)), FGB_EINVAL,
                "fp8_block_gemm: a and b must be 16-byte aligned");
    FGB_REQUIRE(d_dtype == FGB_F32 || d_dtype == FGB_BF16, FGB_EUNSUPPORTED,
                "fp8_block_gemm: d_dtype must be FGB_F32 or FGB_BF16");
    FGB_REQUIRE(mode == FGB_GEMM_EXACT || mode == FGB_GEMM_FAST, FGB_EUNSUPPORTED,
                "fp8_block_gemm: mode must be FGB_GEMM_EXACT or FGB_GEMM_FAST");
    FGB_REQUIRE(!(accumulate && d_dtype != FGB_F32), FGB_EUNSUPPORTED,
                "fp8_block_gemm: accumulate needs FP32 output");
    int ag, bg;
    if (a_gran == FGB_ROW1x128)
        ag = AG_ROW128;
    else if (a_gran == FGB_ROW1x32)
        ag = AG_ROW32;
    else
        return set_error(FGB_EUNSUPPORTED, "fp8_block_gemm: a_gran must be FGB_ROW1x128 or FGB_ROW1x32");
    if (b_gran == FGB_BLOCK128)
        bg = BG_BLOCK;
    else if (b_gran == FGB_ROW1x128)
        bg = BG_ROW128;
    else if (b_gran == FGB_ROW1x32)
        bg = BG_ROW32;
    else
        return set_error(FGB_EUNSUPPORTED, "fp8_block_gemm: unknown b_gran");
    FGB_REQUIRE((ag == AG_ROW32) == (bg == BG_ROW32), FGB_EUNSUPPORTED,
                "fp8_block_gemm: FGB_ROW1x32 scales must be used on both operands");
    FGB_REQUIRE(!b_l1 || b_gran == FGB_ROW1x32, FGB_EUNSUPPORTED,
                "fp8_block_gemm: b_l1 needs 1x32 B scales (the level-2 scales of the two-level format)");
    FGB_REQUIRE(!b_l1 || (g1 > 0 && K <= g1), FGB_EUNSUPPORTED,
                "fp8_block_gemm: b_l1 needs K <= g1 (one level-1 group along K)");
    if (ag == AG_ROW32 && K > 0)
        FGB_REQUIRE(((uintptr_t)sa & 3) == 0 && ((uintptr_t)sb & 3) == 0, FGB_EINVAL,
                    "fp8_block_gemm: 1x32 scale tensors must be 4-byte aligned");
    GemmArgs p{};
    p.a = a; p.sa = sa; p.b = b; p.sb = sb; p.l1 = b_l1; p.d = d;
    p.M = M; p.N = N; p.K = K; p.lda = lda; p.ldb = ldb; p.ldd = ldd;
    p.accumulate = accumulate;
    p.tiles_n = (int)((N + BN - 1) / BN);
    int64_t tiles = ((M + BM - 1) / BM) * p.tiles_n;
    FGB_REQUIRE(tiles < (1ll << 31), FGB_EINVAL, "fp8_block_gemm: too many tiles");
    if (a_fmt == FGB_E5M2)
        return mode == FGB_GEMM_FAST
                   ? dispatch_e5m2_mode<MODE_FAST>(bg, d_dtype == FGB_BF16, p, tiles, (hipStream_t)stream)
                   : dispatch_e5m2_mode<MODE_EXACT>(bg, d_dtype == FGB_BF16, p, tiles, (hipStream_t)stream);
    return dispatch<GK_NONE>(mode, ag, bg, d_dtype == FGB_BF16, p, tiles, (hipStream_t)stream);
}

extern "C" int fp8_block_gemm(const uint8_t *a, const uint8_t *sa, int a_gran, const uint8_t *b, const uint8_t *sb,
                              int b_gran, const float *b_l1, int64_t g1, int64_t M, int64_t N, int64_t K, int64_t lda,
                              int64_t ldb, void *d, int d_dtype, int64_t ldd, int accumulate, int mode,
                              void *workspace, size_t ws_bytes, void *stream)
{
    (void)workspace;
    (void)ws_bytes;
    return fp8_block_gemm_fmt(a, sa, a_gran, FGB_E4M3, b, sb, b_gran, FGB_E4M3, b_l1, g1, M, N, K, lda, ldb, d,
                              d_dtype, ldd, accumulate, mode, stream);
}

extern "C" int fp8_grouped_gemm(const uint8_t *a, const uint8_t *sa, const uint8_t *b,
                                const uint8_t *sb, const int32_t *group_offsets, int G,
                                int64_t M_cap, int64_t N, int64_t K, void *d, int d_dtype,
                                int mode, void *stream)
{
    clear_error();
    FGB_REQUIRE(a && sa && b && sb && d && group_offsets, FGB_EINVAL, "fp8_grouped_gemm: null pointer");
    FGB_REQUIRE(G >= 1 && G <= 1024, FGB_EINVAL, "fp8_grouped_gemm: G must be in [1, 1024]");
    FGB_REQUIRE(M_cap >= 0 && N > 0 && K > 0 && K % 128 == 0, FGB_EINVAL,
                "fp8_grouped_gemm: need N > 0 and K a positive multiple of 128");
    FGB_REQUIRE(256 * K < (1ll << 32), FGB_EINVAL, "fp8_grouped_gemm: K too large");
    FGB_REQUIRE(aligned16(a) && aligned16(b), FGB_EINVAL, "fp8_grouped_gemm: a and b must be 16-byte aligned");
    FGB_REQUIRE(d_dtype == FGB_F32 || d_dtype == FGB_BF16, FGB_EUNSUPPORTED,
                "fp8_grouped_gemm: d_dtype must be FGB_F32 or FGB_BF16");
    FGB_REQUIRE(mode == FGB_GEMM_EXACT || mode == FGB_GEMM_FAST, FGB_EUNSUPPORTED,
                "fp8_grouped_gemm: mode must be FGB_GEMM_EXACT or FGB_GEMM_FAST");
    if (M_cap == 0)
        return FGB_OK;
    GemmArgs p{};
    p.a = a; p.sa = sa; p.b = b; p.sb = sb; p.l1 = nullptr; p.d = d;
    p.M = M_cap; p.N = N; p.K = K; p.lda = K; p.ldb = K; p.ldd = N;
    p.accumulate = 0;
    p.tiles_n = (int)((N + BN - 1) / BN);
    p.offs = group_offsets;
    p.G = G;
    p.b_stride = N * K;
    p.sb_stride = ((N + 127) / 128) * (K / 128);
    // sum over experts of ceil(rows_e / BM) <= ceil(M_cap / BM) + G
    int64_t tiles = ((M_cap + BM - 1) / BM + G) * p.tiles_n;
    FGB_REQUIRE(tiles < (1ll << 31), FGB_EINVAL, "fp8_grouped_gemm: too many tiles");
    return dispatch<GK_M>(mode, AG_ROW128, BG_BLOCK, d_dtype == FGB_BF16, p, tiles, (hipStream_t)stream);
}

extern "C" int fp8_grouped_gemm_masked(const uint8_t *a, const uint8_t *sa, const uint8_t *b, const uint8_t *sb,
                                       const int32_t *masked_m, int G, int64_t M_max, int64_t N, int64_t K, void *d,
                                       int d_dtype, int mode, void *stream)
{
    clear_error();
    FGB_REQUIRE(a && sa && b && sb && d && masked_m, FGB_EINVAL, "fp8_grouped_gemm_masked: null pointer");
    FGB_REQUIRE(G >= 1 && G <= 1024, FGB_EINVAL, "fp8_grouped_gemm_masked: G must be in [1, 1024]");
    FGB_REQUIRE(M_max > 0 && N > 0 && K > 0 && K % 128 == 0, FGB_EINVAL,
                "fp8_grouped_gemm_masked: need M_max, N > 0 and K a positive multiple of 128");
    FGB_REQUIRE(256 * K < (1ll << 32), FGB_EINVAL, "fp8_grouped_gemm_masked: K too large");
    FGB_REQUIRE(aligned16(a) && aligned16(b), FGB_EINVAL, "fp8_grouped_gemm_masked: a and b must be 16-byte aligned");
    FGB_REQUIRE(d_dtype == FGB_F32 || d_dtype == FGB_BF16, FGB_EUNSUPPORTED,
                "fp8_grouped_gemm_masked: d_dtype must be FGB_F32 or FGB_BF16");
    FGB_REQUIRE(mode == FGB_GEMM_EXACT || mode == FGB_GEMM_FAST, FGB_EUNSUPPORTED,
                "fp8_grouped_gemm_masked: mode must be FGB_GEMM_EXACT or FGB_GEMM_FAST");
    GemmArgs p{};
    p.a = a; p.sa = sa; p.b = b; p.sb = sb; p.l1 = nullptr; p.d = d;
    p.M = (int64_t)G * M_max; p.N = N; p.K = K; p.lda = K; p.ldb = K; p.ldd = N;
    p.accumulate = 0;
    p.tiles_n = (int)((N + BN - 1) / BN);
    p.G = G;
    p.b_stride = N * K;
    p.sb_stride = ((N + 127) / 128) * (K / 128);
    p.masked_m = masked_m;
    p.m_max = M_max;
    const int64_t tiles = (int64_t)G * ((M_max + BM - 1) / BM) * p.tiles_n;
    FGB_REQUIRE(tiles < (1ll << 31), FGB_EINVAL, "fp8_grouped_gemm_masked: too many tiles");
    return dispatch<GK_MM>(mode, AG_ROW128, BG_BLOCK, d_dtype == FGB_BF16, p, tiles, (hipStream_t)stream);
}

extern "C" int fp8_kgrouped_gemm(const uint8_t *a, const uint8_t *sa, const uint8_t *b, const uint8_t *sb,
                                 const int32_t *k_offsets, int G, int64_t M, int64_t N, int64_t K_cap, void *d,
                                 int d_dtype, int accumulate, int mode, void *stream)
{
    clear_error();
    FGB_REQUIRE(a && sa && b && sb && d && k_offsets, FGB_EINVAL, "fp8_kgrouped_gemm: null pointer");
    FGB_REQUIRE(G >= 1 && G <= 1024, FGB_EINVAL, "fp8_kgrouped_gemm: G must be in [1, 1024]");
    FGB_REQUIRE(M > 0 && N > 0 && K_cap > 0 && K_cap % 128 == 0, FGB_EINVAL,
                "fp8_kgrouped_gemm: need M, N > 0 and K_cap a positive multiple of 128");
    FGB_REQUIRE(256 * K_cap < (1ll << 32), FGB_EINVAL, "fp8_kgrouped_gemm: K_cap too large");
    FGB_REQUIRE(aligned16(a) && aligned16(b), FGB_EINVAL, "fp8_kgrouped_gemm: a and b must be 16-byte aligned");
    FGB_REQUIRE(d_dtype == FGB_F32 || d_dtype == FGB_BF16, FGB_EUNSUPPORTED,
                "fp8_kgrouped_gemm: d_dtype must be FGB_F32 or FGB_BF16");
    FGB_REQUIRE(mode == FGB_GEMM_EXACT || mode == FGB_GEMM_FAST, FGB_EUNSUPPORTED,
                "fp8_kgrouped_gemm: mode must be FGB_GEMM_EXACT or FGB_GEMM_FAST");
    FGB_REQUIRE(!(accumulate && d_dtype != FGB_F32), FGB_EUNSUPPORTED, "fp8_kgrouped_gemm: accumulate needs FP32 output");
    GemmArgs p{};
    p.a = a; p.sa = sa; p.b = b; p.sb = sb; p.l1 = nullptr; p.d = d;
    p.M = M; p.N = N; p.K = K_cap; p.lda = K_cap; p.ldb = K_cap; p.ldd = N;
    p.accumulate = accumulate;
    p.tiles_n = (int)((N + BN - 1) / BN);
    p.G = G;
    p.koffs = k_offsets;
    p.d_stride = M * N;
    const int64_t tiles = ((M + BM - 1) / BM) * p.tiles_n * G;
    FGB_REQUIRE(tiles < (1ll << 31), FGB_EINVAL, "fp8_kgrouped_gemm: too many tiles");
    return dispatch<GK_K>(mode, AG_ROW128, BG_ROW128, d_dtype == FGB_BF16, p, tiles, (hipStream_t)stream);
}
