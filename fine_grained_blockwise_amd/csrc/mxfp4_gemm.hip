// mxfp4_gemm.hip -- products with MXFP4 operands, D = A * B^T, dense and per expert.
//
// B holds E2M1 codes with 1x32 scales; A the same, or E4M3 codes with 1x128 scales.
//   E2M1 A: the scaled matrix instruction takes 32 codes and one scale byte per
//     lane.  A product of two E2M1 values is a multiple of 1/4 up to 36, so the 32
//     products of a group add up exactly, and the unit's sums across groups were
//     measured at FP32 rounding (worst 5.6e-7 of the largest product with scales
//     2^-20 .. 2^20 apart; scale byte 255 gives NaN).
//   E4M3 A: both operands become bf16 with their power of two folded in (exact),
//     multiplied on the bf16 matrix unit with FP32 sums, as FGB_GEMM_EXACT does.
#include "gemm_kernel.h"

namespace fgb {

struct Mx4Args {
    const uint8_t *a, *sa, *b, *sb;
    void *d;
    int64_t M, N, K, lda, ldb, ldd; // lda, ldb in bytes
    int accumulate;
    const int32_t *offs; // grouped: [G + 1], else NULL
    int G;
};

// One wave per 32 x 32 tile of D, operands straight from memory: lane l holds row
// l % 32 of both and the 32-element group l / 32 of each 64 columns.
template <bool A8, bool OUT_BF16>
__global__ __launch_bounds__(64) void mx4_gemm_kernel(Mx4Args p)
{
    const int lane = threadIdx.x, r = lane & 31, h = lane >> 5;
    const int64_t n0 = (int64_t)blockIdx.x * 32;
    const int e = blockIdx.z;
    int64_t lo = 0, hi = p.M;
    const uint8_t *b = p.b, *sb = p.sb;
    const int64_t steps = (p.K + 255) / 256;
    if (p.offs) {
        lo = p.offs[e];
        hi = p.offs[e + 1];
        b += (int64_t)e * p.N * p.ldb;
        sb += (int64_t)e * p.N * steps * 8;
    }
    const int64_t n = n0 + r < p.N ? n0 + r : p.N - 1;
    for (int64_t m0 = lo + (int64_t)blockIdx.y * 32; m0 < hi; m0 += (int64_t)gridDim.y * 32) {
        const int64_t m = m0 + r < hi ? m0 + r : hi - 1;
        v16f acc = {};
        for (int64_t k = 0; k < p.K; k += 64) {
            const int64_t g = k / 32 + h; // this lane's group
            const bool in = g < p.K / 32;
            const int64_t gc = in ? g : 0;
            const uint4 bw = *reinterpret_cast<const uint4 *>(b + n * p.ldb + gc * 16);
            const uint32_t bs = sb[((gc >> 3) * p.N + n) * 8 + (gc & 7)];
            if constexpr (!A8) {
                uint4 aw = *reinterpret_cast<const uint4 *>(p.a + m * p.lda + gc * 16);
                const uint32_t as = p.sa[((gc >> 3) * p.M + m) * 8 + (gc & 7)];
                if (!in)
                    aw = make_uint4(0, 0, 0, 0);
                acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                    (v8i){(int)aw.x, (int)aw.y, (int)aw.z, (int)aw.w, 0, 0, 0, 0},
                    (v8i){(int)bw.x, (int)bw.y, (int)bw.z, (int)bw.w, 0, 0, 0, 0}, acc, 4, 4, 0, (int)as, 0, (int)bs);
            } else {
                const uint4 *ap = reinterpret_cast<const uint4 *>(p.a + m * p.lda + gc * 32);
                const uint4 a0 = ap[0], a1 = ap[1];
                const float fa = __uint_as_float((uint32_t)p.sa[m * (p.K / 128) + gc / 4] << 23);
                const float fb = __uint_as_float(bs << 23);
                acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(cvt8_bf16(a0.x, a0.y, fa), cvt8_bf16_e2m1(bw.x, fb), acc, 0, 0, 0);
                acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(cvt8_bf16(a0.z, a0.w, fa), cvt8_bf16_e2m1(bw.y, fb), acc, 0, 0, 0);
                acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(cvt8_bf16(a1.x, a1.y, fa), cvt8_bf16_e2m1(bw.z, fb), acc, 0, 0, 0);
                acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(cvt8_bf16(a1.z, a1.w, fa), cvt8_bf16_e2m1(bw.w, fb), acc, 0, 0, 0);
            }
        }
        // register i of lane l: row (i / 4) * 8 + (l / 32) * 4 + i % 4, column l % 32
#pragma unroll
        for (int i = 0; i < 16; i++) {
            const int64_t row = m0 + (i / 4) * 8 + h * 4 + i % 4;
            if (row < hi && n0 + r < p.N) {
                const int64_t at = row * p.ldd + n0 + r;
                if constexpr (OUT_BF16)
                    ((__bf16 *)p.d)[at] = (__bf16)acc[i];
                else
                    ((float *)p.d)[at] = p.accumulate ? ((float *)p.d)[at] + acc[i] : acc[i];
            }
        }
    }
}

static int check_mx4(const char *name, int a_fmt, int64_t M, int64_t N, int64_t K, int d_dtype)
{
    FGB_REQUIRE(a_fmt == FGB_E2M1 || a_fmt == FGB_E4M3, FGB_EUNSUPPORTED, "%s: a_fmt must be FGB_E2M1 or FGB_E4M3", name);
    FGB_REQUIRE(M >= 0 && N >= 0 && K >= 0 && K % (a_fmt == FGB_E4M3 ? 128 : 32) == 0, FGB_EINVAL,
                "%s: need M, N >= 0 and K a multiple of 32 (128 with an E4M3 A) (M=%lld N=%lld K=%lld)", name,
                (long long)M, (long long)N, (long long)K);
    FGB_REQUIRE(M < (1ll << 31) && N < (1ll << 31) && K < (1ll << 23), FGB_EINVAL,
                "%s: M and N must be below 2^31 and K below 2^23", name);
    FGB_REQUIRE(d_dtype == FGB_F32 || d_dtype == FGB_BF16, FGB_EUNSUPPORTED, "%s: d_dtype must be FGB_F32 or FGB_BF16",
                name);
    return FGB_OK;
}

// The 256 x 256-tiled kernel of gemm_kernel.h.
template <int GK> static int launch_tiled(const Mx4Args &x, int a_fmt, bool bf16, hipStream_t st)
{
    GemmArgs p{};
    p.a = x.a; p.sa = x.sa; p.b = x.b; p.sb = x.sb; p.d = x.d;
    p.M = x.M; p.N = x.N; p.K = x.K; p.lda = x.lda; p.ldb = x.ldb; p.ldd = x.ldd;
    p.accumulate = x.accumulate;
    p.tiles_n = (int)((x.N + BN - 1) / BN);
    p.offs = x.offs;
    p.G = x.G;
    p.b_stride = x.N * (x.K / 2);
    p.sb_stride = (x.K + 255) / 256 * x.N * 8;
    const int64_t tiles = ((x.M + BM - 1) / BM + (GK == GK_M ? x.G : 0)) * p.tiles_n;
    FGB_REQUIRE(tiles < (1ll << 31), FGB_EINVAL, "mxfp4 gemm: too many tiles");
    if (a_fmt == FGB_E4M3)
        return launch_out<MODE_EXACT, AG_ROW128, BG_STEP32, GK, FMT_E4M3, FMT_E2M1>(bf16, p, tiles, st);
    return launch_out<MODE_FP4, AG_STEP32, BG_STEP32, GK, FMT_E2M1, FMT_E2M1>(bf16, p, tiles, st);
}

static int launch_mx4(const char *name, const Mx4Args &p, int a_fmt, int d_dtype, hipStream_t st)
{
    if (p.offs ? p.M > 64 * p.G : p.M > 64)
        return p.offs ? launch_tiled<GK_M>(p, a_fmt, d_dtype == FGB_BF16, st)
                      : launch_tiled<GK_NONE>(p, a_fmt, d_dtype == FGB_BF16, st);
    const int64_t gx = (p.N + 31) / 32, tiles = (p.M + 31) / 32;
    const dim3 grid((unsigned)gx, (unsigned)(p.offs ? (tiles < 16 ? tiles : 16) : (tiles < 65535 ? tiles : 65535)),
                    (unsigned)p.G);
    if (a_fmt == FGB_E4M3)
        d_dtype == FGB_BF16 ? mx4_gemm_kernel<true, true><<<grid, 64, 0, st>>>(p)
                            : mx4_gemm_kernel<true, false><<<grid, 64, 0, st>>>(p);
    else
        d_dtype == FGB_BF16 ? mx4_gemm_kernel<false, true><<<grid, 64, 0, st>>>(p)
                            : mx4_gemm_kernel<false, false><<<grid, 64, 0, st>>>(p);
    FGB_LAUNCHED(name);
    return FGB_OK;
}

} // namespace fgb

using namespace fgb;

extern "C" int mxfp4_gemm(const uint8_t *a, const uint8_t *sa, int a_fmt, const uint8_t *b, const uint8_t *sb, int64_t M,
                          int64_t N, int64_t K, int64_t lda, int64_t ldb, void *d, int d_dtype, int64_t ldd,
                          int accumulate, void *stream)
{
    clear_error();
    const int rc = check_mx4("mxfp4_gemm", a_fmt, M, N, K, d_dtype);
    if (rc != FGB_OK)
        return rc;
    FGB_REQUIRE(!(accumulate && d_dtype != FGB_F32), FGB_EUNSUPPORTED, "mxfp4_gemm: accumulate needs FP32 output");
    if (M == 0 || N == 0)
        return FGB_OK;
    FGB_REQUIRE(d && (K == 0 || (a && sa && b && sb)), FGB_EINVAL, "mxfp4_gemm: null pointer");
    const int64_t row_a = a_fmt == FGB_E4M3 ? K : K / 2;
    FGB_REQUIRE(K == 0 || (lda >= row_a && ldb >= K / 2 && lda % 16 == 0 && ldb % 16 == 0), FGB_EINVAL,
                "mxfp4_gemm: lda and ldb (bytes) must hold a row and be multiples of 16");
    FGB_REQUIRE(K == 0 || (lda < (1ll << 23) && ldb < (1ll << 23)), FGB_EINVAL,
                "mxfp4_gemm: lda and ldb must be below 2^23 bytes");
    FGB_REQUIRE(ldd >= N, FGB_EINVAL, "mxfp4_gemm: ldd must be >= N");
    FGB_REQUIRE(d_dtype == FGB_BF16 || ldd < (1ll << 23), FGB_EUNSUPPORTED,
                "mxfp4_gemm: FP32 output rows (ldd) must be shorter than 2^23 elements");
    FGB_REQUIRE(K == 0 || (aligned16(a) && aligned16(b) && aligned16(sb) && (a_fmt == FGB_E4M3 || aligned16(sa))),
                FGB_EINVAL, "mxfp4_gemm: a, b and their 1x32 scales must be 16-byte aligned");
    FGB_REQUIRE(((uintptr_t)d & (d_dtype == FGB_BF16 ? 1 : 3)) == 0, FGB_EINVAL, "mxfp4_gemm: d misaligned");
    Mx4Args p{};
    p.a = a; p.sa = sa; p.b = b; p.sb = sb; p.d = d;
    p.M = M; p.N = N; p.K = K; p.lda = lda; p.ldb = ldb; p.ldd = ldd;
    p.accumulate = accumulate;
    p.G = 1;
    return launch_mx4("mxfp4_gemm", p, a_fmt, d_dtype, (hipStream_t)stream);
}

extern "C" int mxfp4_grouped_gemm(const uint8_t *a, const uint8_t *sa, int a_fmt, const uint8_t *b, const uint8_t *sb,
                                  const int32_t *group_offsets, int G, int64_t M_cap, int64_t N, int64_t K, void *d,
                                  int d_dtype, void *stream)
{
    clear_error();
    const int rc = check_mx4("mxfp4_grouped_gemm", a_fmt, M_cap, N, K, d_dtype);
    if (rc != FGB_OK)
        return rc;
    FGB_REQUIRE(G >= 1 && G <= 1024, FGB_EINVAL, "mxfp4_grouped_gemm: G must be in [1, 1024]");
    if (M_cap == 0 || N == 0)
        return FGB_OK;
    FGB_REQUIRE(d_dtype == FGB_BF16 || N < (1ll << 23), FGB_EUNSUPPORTED,
                "mxfp4_grouped_gemm: FP32 output rows must be shorter than 2^23 elements");
    FGB_REQUIRE(d && group_offsets && (K == 0 || (a && sa && b && sb)), FGB_EINVAL, "mxfp4_grouped_gemm: null pointer");
    FGB_REQUIRE(K == 0 || (aligned16(a) && aligned16(b) && aligned16(sb) && (a_fmt == FGB_E4M3 || aligned16(sa))),
                FGB_EINVAL, "mxfp4_grouped_gemm: a, b and their 1x32 scales must be 16-byte aligned");
    FGB_REQUIRE(((uintptr_t)d & (d_dtype == FGB_BF16 ? 1 : 3)) == 0 && ((uintptr_t)group_offsets & 3) == 0, FGB_EINVAL,
                "mxfp4_grouped_gemm: d or group_offsets misaligned");
    Mx4Args p{};
    p.a = a; p.sa = sa; p.b = b; p.sb = sb; p.d = d;
    p.M = M_cap; p.N = N; p.K = K; p.lda = a_fmt == FGB_E4M3 ? K : K / 2; p.ldb = K / 2; p.ldd = N;
    p.offs = group_offsets;
    p.G = G;
    return launch_mx4("mxfp4_grouped_gemm", p, a_fmt, d_dtype, (hipStream_t)stream);
}
