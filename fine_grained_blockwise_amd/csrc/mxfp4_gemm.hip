// mxfp4_gemm.hip -- products with MXFP4 operands, D = A * B^T, dense and per expert.
//
// B holds E2M1 codes with 1x32 scales; A the same, or E4M3 codes with 1x128 scales.
//   E2M1 A: the scaled matrix instruction takes 32 codes and one scale byte per
//     lane.  A product of two E2M1 values is a multiple of 1/4 up to 36, so the 32
//     products of a group add up exactly; with the unit's sums across groups, scales
//     2^-20 .. 2^20 apart among them, D stays within the bound of K products summed in
//     FP32 (the tests hold it there).  Scale byte 255 gives NaN.
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

// Few rows (decode, short prompts, few rows per expert): the weights' bytes bound
// it.  A workgroup of W waves owns 16 NB columns of D and 16 MB rows at a time;
// its waves split K by 256 elements (a 128-byte line of each weight row) and their
// sums are added through LDS in wave order.  The weights are the first operand of
// the 16-row matrix instructions and the activations the second, both straight from
// memory: lane l holds row l % 16 and the 32-element groups l / 16 and 4 + l / 16 of
// a unit, so a load instruction covers 64 contiguous bytes of 16 rows, and a lane
// ends with four consecutive columns of one row of D.  The next unit's loads are
// issued before a unit is multiplied.  One token's eight experts (4096x7168, E4M3 A,
// 125 MB): 30 us, 4.2 TB/s; 28672x8192: 29 us, 4.3 TB/s with 4 us of launch in it.
//
// Buffer loads: what lies past an operand's last row reads as zeros.  The range check
// holds the lane's offset alone against the record count, so a row block's and unit's
// offset goes into the descriptor (scalar instructions; in the lanes' offsets it took
// 4 to 24 registers and spilled 18), never into the load's scalar offset.
template <bool A8, int MB, int NB> struct NarrowUnit {
    uint4 b[NB][2], a[MB][A8 ? 4 : 2];
    uint2 bs[NB], as[MB]; // scale bytes of a row: all eight groups (an E4M3 A: .x holds its two)
};

typedef float v4f __attribute__((ext_vector_type(4)));

// A raw buffer descriptor of `bytes` bytes at a wave-uniform address.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const uint8_t *q, int64_t bytes)
{
    const uint64_t v = (uint64_t)(uintptr_t)q;
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v), hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
    return __builtin_amdgcn_make_buffer_rsrc((void *)(uintptr_t)(((uint64_t)hi << 32) | lo), 0,
                                             __builtin_amdgcn_readfirstlane((int)bytes), BUF_DWORD3);
}

// The same from byte `skip` of the `bytes` on: nothing where that is past them.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_from(const uint8_t *q, int bytes, int skip)
{
    return buffer(q + skip, max(bytes - skip, 0));
}

// (64 rows of an MXFP4 A, 64 columns: held to 256 registers for two waves a SIMD, 256x7168x2048
// 17.6 -> 15.7 us; an E4M3 A would spill there.)
template <bool A8, int MB, int NB, int W, bool OUT_BF16>
__global__ __launch_bounds__(W * 64) __attribute__((amdgpu_waves_per_eu(!A8 && MB == 4 && NB == 4 ? 2 : 1))) void mx4_narrow_kernel(Mx4Args p, int tiles_n, int chunks)
{
    __shared__ v4f part[W][MB * NB][64];
    const int lane = threadIdx.x & 63, r = lane & 15, h = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int units = (int)((p.K + 255) / 256), groups = (int)(p.K / 32);
    // Dense: workgroup -> (column tile, row chunk): eight column tiles, then their next
    // chunk, so that the chunks of a column tile run on one XCD (b % 8) and find its
    // weights in that L2.  Per expert: the (expert with rows, column tile) pairs in turn,
    // by as many workgroups as run at once (8 busy experts of 32, 7168x2048: 22.6 us
    // with a workgroup for every pair of the host's bound, 20.7 us so).
    for (int64_t task = blockIdx.x;; task += gridDim.x) {
        int tn, chunk = 0;
        int64_t lo = 0, hi = p.M;
        const uint8_t *b = p.b, *sb = p.sb;
        if (!p.offs) {
            tn = (int)(task / (8 * chunks)) * 8 + (int)(task & 7);
            chunk = (int)(task / 8 % chunks);
            if (tn >= tiles_n)
                return;
        } else {
            tn = (int)(task % tiles_n);
            int want = (int)(task / tiles_n), e = -1;
            for (int g0 = 0; g0 < p.G && e < 0; g0 += 64) {
                const int g = g0 + lane;
                const int32_t o0 = g < p.G ? p.offs[g] : 0, o1 = g < p.G ? p.offs[g + 1] : 0;
                const uint64_t live = __ballot(o1 > o0);
                const int rank = __builtin_amdgcn_mbcnt_hi((uint32_t)(live >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)live, 0));
                const uint64_t hit = __ballot(o1 > o0 && rank == want);
                if (hit) {
                    const int l = __builtin_ctzll(hit);
                    e = g0 + l;
                    lo = __builtin_amdgcn_readlane(o0, l);
                    hi = __builtin_amdgcn_readlane(o1, l);
                }
                want -= __builtin_popcountll(live);
            }
            if (e < 0)
                return; // uniform over the workgroup: no pair is left
            b += (int64_t)e * p.N * p.ldb;
            sb += (int64_t)e * p.N * units * 8;
        }
        const int64_t n0 = (int64_t)tn * (16 * NB);
        b += n0 * p.ldb;
        sb += n0 * 8;
        const int bn = (int)min((int64_t)(16 * NB), p.N - n0);
        const int bbytes = (int)((bn - 1) * p.ldb + p.K / 2), bblock = (int)(16 * p.ldb);
        const uint32_t boff = (uint32_t)(r * p.ldb + h * 16);
        for (int64_t m0 = lo + (int64_t)chunk * (16 * MB); m0 < hi; m0 += (int64_t)chunks * (16 * MB)) {
            const int am = (int)min((int64_t)(16 * MB), hi - m0);
            const uint8_t *const a = p.a + m0 * p.lda;
            const int abytes = (int)((am - 1) * p.lda + (A8 ? p.K : p.K / 2)), ablock = (int)(16 * p.lda);
            const uint32_t aoff = (uint32_t)(r * p.lda + h * (A8 ? 32 : 16));
            const int as_row = (int)(p.K / 128); // E4M3 A: its scales, row-major
            const uint8_t *const sa8 = p.sa + m0 * as_row;
            v4f acc[MB][NB];
#pragma unroll
            for (int i = 0; i < MB; i++)
#pragma unroll
                for (int j = 0; j < NB; j++)
                    acc[i][j] = (v4f){0.f, 0.f, 0.f, 0.f};
            // (What is read of groups past K is replaced in product(), not here: nothing
            // may wait for a load where it is issued.)
            auto load = [&](int u, NarrowUnit<A8, MB, NB> &x) {
                const auto bsrs = buffer(sb + (int64_t)u * p.N * 8, bn * 8);
#pragma unroll
                for (int j = 0; j < NB; j++) {
                    const auto brs = buffer_from(b, bbytes, j * bblock + u * 128);
                    x.b[j][0] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(brs, boff, 0, 0));
                    x.b[j][1] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(brs, boff + 64, 0, 0));
                    x.bs[j] = __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(bsrs, r * 8 + j * 128, 0, 0));
                }
                if constexpr (A8) {
#pragma unroll
                    for (int i = 0; i < MB; i++) {
                        const auto ars = buffer_from(a, abytes, i * ablock + u * 256);
#pragma unroll
                        for (int k = 0; k < 4; k++)
                            x.a[i][k] = __builtin_bit_cast(
                                uint4, __builtin_amdgcn_raw_buffer_load_b128(ars, aoff + (k / 2) * 128 + (k & 1) * 16, 0, 0));
                        const auto asrs = buffer_from(sa8, am * as_row, i * 16 * as_row + 2 * u);
                        x.as[i].x = __builtin_amdgcn_raw_buffer_load_b8(asrs, r * as_row, 0, 0);
                        x.as[i].y = __builtin_amdgcn_raw_buffer_load_b8(asrs, r * as_row + 1, 0, 0);
                    }
                } else {
                    const auto asrs = buffer(p.sa + ((int64_t)u * p.M + m0) * 8, am * 8);
#pragma unroll
                    for (int i = 0; i < MB; i++) {
                        const auto ars = buffer_from(a, abytes, i * ablock + u * 128);
                        x.a[i][0] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(ars, aoff, 0, 0));
                        x.a[i][1] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(ars, aoff + 64, 0, 0));
                        x.as[i] = __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(asrs, r * 8 + i * 128, 0, 0));
                    }
                }
            };
            auto product = [&](int u, NarrowUnit<A8, MB, NB> &x) {
                if (u * 8 + 8 > groups) { // uniform: the last unit of a K that is no multiple of 256
                    const bool in0 = u * 8 + h < groups, in1 = u * 8 + 4 + h < groups;
                    constexpr int Q = A8 ? 2 : 1;
#pragma unroll
                    for (int i = 0; i < MB; i++)
#pragma unroll
                        for (int q = 0; q < Q; q++) {
                            if (!in0)
                                x.a[i][q] = make_uint4(0, 0, 0, 0);
                            if (!in1)
                                x.a[i][Q + q] = make_uint4(0, 0, 0, 0);
                            if (A8 && !in1) // the byte after the row's last is another row's
                                x.as[i].y = 0;
                        }
                }
                if constexpr (!A8) {
#pragma unroll
                    for (int half = 0; half < 2; half++)
#pragma unroll
                        for (int i = 0; i < MB; i++)
#pragma unroll
                            for (int j = 0; j < NB; j++) {
                                const uint4 bw = x.b[j][half], aw = x.a[i][half];
                                acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                                    (v8i){(int)bw.x, (int)bw.y, (int)bw.z, (int)bw.w, 0, 0, 0, 0},
                                    (v8i){(int)aw.x, (int)aw.y, (int)aw.z, (int)aw.w, 0, 0, 0, 0}, acc[i][j], 4, 4, 0,
                                    (int)((half ? x.bs[j].y : x.bs[j].x) >> (8 * h)), 0,
                                    (int)((half ? x.as[i].y : x.as[i].x) >> (8 * h)));
                            }
                } else {
#pragma unroll
                    for (int half = 0; half < 2; half++) {
                        float fa[MB], fb[NB];
#pragma unroll
                        for (int i = 0; i < MB; i++)
                            fa[i] = scale_f32(half ? x.as[i].y : x.as[i].x);
#pragma unroll
                        for (int j = 0; j < NB; j++)
                            fb[j] = scale_f32(((half ? x.bs[j].y : x.bs[j].x) >> (8 * h)) & 0xFFu);
#pragma unroll
                        for (int s = 0; s < 4; s++) {
                            v8bf bv[NB];
#pragma unroll
                            for (int j = 0; j < NB; j++) {
                                const uint4 w = x.b[j][half];
                                bv[j] = cvt8_bf16_e2m1(s == 0 ? w.x : s == 1 ? w.y : s == 2 ? w.z : w.w, fb[j]);
                            }
#pragma unroll
                            for (int i = 0; i < MB; i++) {
                                const uint4 w = x.a[i][2 * half + s / 2];
                                const v8bf av = s % 2 ? cvt8_bf16(w.z, w.w, fa[i]) : cvt8_bf16(w.x, w.y, fa[i]);
#pragma unroll
                                for (int j = 0; j < NB; j++)
                                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bv[j], av, acc[i][j], 0, 0, 0);
                            }
                        }
                    }
                }
            };
            if (wave < units) {
                NarrowUnit<A8, MB, NB> x;
                load(wave, x);
                int u = wave;
                for (; u + W < units; u += W) {
                    NarrowUnit<A8, MB, NB> next;
                    load(u + W, next);
                    product(u, x);
                    x = next;
                }
                product(u, x);
            }
#pragma unroll
            for (int i = 0; i < MB; i++)
#pragma unroll
                for (int j = 0; j < NB; j++)
                    part[wave][i * NB + j][lane] = acc[i][j];
            __syncthreads();
            // register t of lane l: column (l / 16) * 4 + t, row l % 16 of a 16 x 16 block
            for (int o = threadIdx.x; o < MB * NB * 64; o += W * 64) {
                const int blk = o >> 6, l = o & 63;
                v4f sum = part[0][blk][l];
#pragma unroll
                for (int w = 1; w < W; w++)
                    sum += part[w][blk][l];
                const int64_t m = m0 + (blk / NB) * 16 + (l & 15), n = n0 + (blk % NB) * 16 + (l >> 4) * 4;
                if (m < hi) {
                    const int64_t at = m * p.ldd + n;
#pragma unroll
                    for (int t = 0; t < 4; t++)
                        if (n + t < p.N) {
                            if constexpr (OUT_BF16)
                                ((__bf16 *)p.d)[at + t] = (__bf16)sum[t];
                            else
                                ((float *)p.d)[at + t] = p.accumulate ? ((float *)p.d)[at + t] + sum[t] : sum[t];
                        }
                }
            }
            __syncthreads();
        }
        if (!p.offs)
            return;
    }
}

template <bool A8, int MB, int NB, int W> static void launch_narrow(const Mx4Args &p, bool bf16, hipStream_t st)
{
    const int tiles_n = (int)((p.N + 16 * NB - 1) / (16 * NB));
    const int64_t all = (p.M + 16 * MB - 1) / (16 * MB);
    const int64_t pairs = (int64_t)tiles_n * p.G, tiles = (int64_t)((tiles_n + 7) / 8) * 8;
    // (experts' rows: a workgroup takes all; the runtime keeps the low 32 bits of a launch's threads)
    const int64_t most = (1ll << 31) / (W * 64) / tiles, cap = most < 1 ? 1 : most < 64 ? most : 64;
    const int chunks = p.offs ? 1 : (int)(all < cap ? all : cap);
    const int64_t grid = p.offs ? (pairs < 512 ? pairs : 512) : tiles * chunks;
    if (bf16)
        mx4_narrow_kernel<A8, MB, NB, W, true><<<(unsigned)grid, W * 64, 0, st>>>(p, tiles_n, chunks);
    else
        mx4_narrow_kernel<A8, MB, NB, W, false><<<(unsigned)grid, W * 64, 0, st>>>(p, tiles_n, chunks);
}

// The narrow kernel's tile: the largest of (16 MB rows, 16 NB columns) whose rows are
// needed and whose tiles still number three quarters of the 256 CUs.  (Tiles, not
// workgroups that run at once: a column tile's chunks stay on one XCD, so fewer than
// eight column tiles leave XCDs idle, which this count does not see.)  For one row
// of 2048x7168, 28672x8192: (1, 1) 5.7, 32 us, (1, 4) 12, 29 us; 64 rows: (1, 2) 8.7,
// 91 us, (4, 4) 20, 45 us, (4, 8) -, 38 us (E4M3 A 74 and 53 us: fewer reads of A, one
// wave a SIMD).
template <bool A8> static void launch_narrow_for(const Mx4Args &p, int64_t blocks, bool bf16, hipStream_t st)
{
    auto fills = [&](int MB, int NB) {
        return (p.N + 16 * NB - 1) / (16 * NB) * (p.offs ? p.G : (blocks + MB - 1) / MB) >= 192;
    };
    if (blocks > 2 && fills(4, 8))
        launch_narrow<A8, 4, 8, 4>(p, bf16, st);
    else if (blocks > 2 && fills(4, 4))
        launch_narrow<A8, 4, 4, 4>(p, bf16, st);
    else if (blocks > 1 && fills(2, 4))
        launch_narrow<A8, 2, 4, 4>(p, bf16, st);
    else if (fills(1, 4))
        launch_narrow<A8, 1, 4, 4>(p, bf16, st);
    else if (fills(1, 2))
        launch_narrow<A8, 1, 2, 8>(p, bf16, st);
    else
        launch_narrow<A8, 1, 1, 8>(p, bf16, st);
}

static int check_mx4(const char *name, int a_fmt, int64_t M, int64_t N, int64_t K, int d_dtype)
{
    FGB_REQUIRE(a_fmt == FGB_E2M1 || a_fmt == FGB_E4M3, FGB_EUNSUPPORTED, "%s: a_fmt must be FGB_E2M1 or FGB_E4M3", name);
    FGB_REQUIRE(M >= 0 && N >= 0 && K >= 0 && K % (a_fmt == FGB_E4M3 ? 128 : 32) == 0, FGB_EINVAL,
                "%s: need M, N >= 0 and K a multiple of 32 (128 with an E4M3 A) (M=%lld N=%lld K=%lld)", name,
                (long long)M, (long long)N, (long long)K);
    FGB_REQUIRE(M < (1ll << 31) && N < (1ll << 29) && K < (1ll << 23), FGB_EINVAL,
                "%s: M must be below 2^31, N below 2^29 and K below 2^23", name);
    FGB_REQUIRE(d_dtype == FGB_F32 || d_dtype == FGB_BF16, FGB_EUNSUPPORTED, "%s: d_dtype must be FGB_F32 or FGB_BF16",
                name);
    return FGB_OK;
}

// (Weights' scales are read in pieces of 8 bytes a row, whose runs start at any row: an
// expert's slice of a stack with odd rows and steps starts at a multiple of 8.)
static int check_aligned(const char *name, const uint8_t *a, const uint8_t *sa, int a_fmt, const uint8_t *b,
                         const uint8_t *sb, int64_t K)
{
    FGB_REQUIRE(K == 0 || (aligned16(a) && aligned16(b) && ((uintptr_t)sb & 7) == 0 &&
                           (a_fmt == FGB_E4M3 || aligned16(sa))),
                FGB_EINVAL, "%s: a, b and an MXFP4 A's scales must be 16-byte aligned, B's scales 8-byte", name);
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

// Narrow or tiled, by what each was measured to take.  The tiled kernel runs its
// tiles 256 at a time, each round 8 us and 1.25 us a 256-element step (1.9 us a
// 128-element step with an E4M3 A), 1.4 times that where every tile reads other
// weights (experts of few rows); the narrow one reads the weights once per 16-64 rows
// and reaches 0.78 (0.55 at K = 2048, 0.7 at K = 7168) PFLOP/s, less only where it is
// bound by bytes and far ahead; its 64 x 128 blocks of a dense product of more than 64
// rows run 256 at a time too.
// Measured, narrow against tiled, MXFP4 A: 512x2048x7168 19 / 42 us, 1024x2048x7168
// 29 / 42, 256x7168x2048 15 / 18, 320x7168x2048 27 / 18.6, 64x28672x8192 38 / 53,
// 128x28672x8192 64 / 52, 32 experts of 32 rows (4096x7168) 113 / 135; E4M3 A:
// 1024x2048x7168 42 / 115, 256x7168x2048 21 / 38, 768x7168x2048 58 / 40, 128x28672x8192
// 98 / 134, 192x28672x8192 145 / 134, 32 experts of 64 rows 178 / 332, of 128 327 / 332
// (7168x2048: 260 / 199).
// G: experts, 0 for a dense product.
static bool takes_narrow(int64_t M, int64_t N, int64_t K, int G, int a_fmt)
{
    const bool a8 = a_fmt == FGB_E4M3, grouped = G > 0;
    const double step_us = a8 ? (double)(K / 128) * 1.9 : (double)((K + 255) / 256) * 1.25;
    const double tile_us = (8.0 + step_us) * (grouped ? 1.4 : 1.0);
    const int64_t tiles = ((M + 255) / 256 + G / 2) * ((N + 255) / 256);
    double work = (double)M * (double)N;
    if (!grouped && M > 64)
        work = (double)(((M + 63) / 64 * ((N + 127) / 128) + 255) / 256 * 256) * (64 * 128);
    const double narrow_us = 2e-9 * work * (double)K / (a8 ? 0.55 : 0.78);
    return narrow_us <= tile_us * (double)((tiles + 255) / 256);
}

static int launch_mx4(const char *name, const Mx4Args &p, int a_fmt, int d_dtype, hipStream_t st)
{
    const bool bf16 = d_dtype == FGB_BF16;
    if (!takes_narrow(p.M, p.N, p.K, p.offs ? p.G : 0, a_fmt))
        return p.offs ? launch_tiled<GK_M>(p, a_fmt, bf16, st) : launch_tiled<GK_NONE>(p, a_fmt, bf16, st);
    // 16-row blocks, per expert for a grouped product: half a padding to 16 off the
    // average, since M_cap is a bound
    const int64_t rows = p.offs ? p.M / p.G - 8 : p.M, blocks = rows > 16 ? (rows + 15) / 16 : 1;
    if (a_fmt == FGB_E4M3)
        launch_narrow_for<true>(p, blocks, bf16, st);
    else
        launch_narrow_for<false>(p, blocks, bf16, st);
    FGB_LAUNCHED(name);
    return FGB_OK;
}

} // namespace fgb

using namespace fgb;

extern "C" int mxfp4_gemm_tiled(int a_fmt, int64_t M, int64_t N, int64_t K, int G)
{
    clear_error();
    if (check_mx4("mxfp4_gemm_tiled", a_fmt, M, N, K, FGB_BF16) != FGB_OK || G < 0)
        return 0;
    return M > 0 && N > 0 && !takes_narrow(M, N, K, G, a_fmt);
}

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
    const int rc_align = check_aligned("mxfp4_gemm", a, sa, a_fmt, b, sb, K);
    if (rc_align != FGB_OK)
        return rc_align;
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
    const int rc_align = check_aligned("mxfp4_grouped_gemm", a, sa, a_fmt, b, sb, K);
    if (rc_align != FGB_OK)
        return rc_align;
    FGB_REQUIRE(((uintptr_t)d & (d_dtype == FGB_BF16 ? 1 : 3)) == 0 && ((uintptr_t)group_offsets & 3) == 0, FGB_EINVAL,
                "mxfp4_grouped_gemm: d or group_offsets misaligned");
    Mx4Args p{};
    p.a = a; p.sa = sa; p.b = b; p.sb = sb; p.d = d;
    p.M = M_cap; p.N = N; p.K = K; p.lda = a_fmt == FGB_E4M3 ? K : K / 2; p.ldb = K / 2; p.ldd = N;
    p.offs = group_offsets;
    p.G = G;
    return launch_mx4("mxfp4_grouped_gemm", p, a_fmt, d_dtype, (hipStream_t)stream);
}
