// norm.hip -- RMSNorm with the residual's addition, into E4M3 codes with power-of-two
// scales (1 x 128 or 1 x 32), and its gradient.
//
//   h = x + residual (FP32 sum, rounded to the residual's type; h = x without one),
//   rstd = 1 / sqrt(mean_c h^2 + eps), y = h rstd w, codes and scales of the FP32 y by
//   the quantizers' ceil rule; y itself on request.
// Gradient, with a = dy w and hat = h rstd:
//   dx = dh + rstd (a - hat mean_c(a hat)), dw = sum over the rows of dy hat.
//
// Both are bound by memory: every input is read once, into registers, and every output
// written once.  A row belongs to W waves (1, 4, 8 or 16: columns up to 2048, 8192, 16384,
// 32768), a lane holds up to four chunks of eight neighbouring columns, so the row's sum, the
// groups' amax (16 or 4 neighbouring lanes) and the outputs all come from one read.
// 8192 x 7168 BF16: forward 70 us (5.9 TB/s), gradient 78 us (6.0 TB/s) and 5 us for dw.
//
// BF16 loads are streaming (FP32 ones not: load8), stores ordinary: with streaming ones the
// gradient took 85 us, the forward and a reader of its codes 103 (96 so).  A row's loads go out
// together, without branches; waiting for each chunk in turn the gradient took 146 us.
#include "fgb_internal.h"

namespace fgb {

struct NormArgs {
    const void *x, *r, *w;
    void *h, *y;
    uint8_t *q, *s;
    float *rstd;
    int64_t rows, ldx, ldr, ldh, ldy;
    int cols;
    float eps;
    int w_bf16, y_bf16, group, emin;
};

struct NormGradArgs {
    const void *dy, *h, *w, *dh;
    const float *rstd;
    void *dx;
    float *part, *dw; // part [parts][cols]
    int64_t rows, lddy, ldh, lddh, lddx;
    int cols, w_bf16, parts;
};

// Eight neighbouring elements as they lie in memory.
template <bool BF16> struct Raw8 {
    uint4 v[BF16 ? 1 : 2];
};
template <bool BF16> __device__ __forceinline__ Raw8<BF16> load8(const void *p, int64_t at)
{
    Raw8<BF16> o;
    const uint8_t *b = (const uint8_t *)p + at * (BF16 ? 2 : 4);
    // (FP32: the lanes' first and second halves lie in the same lines, which the second load
    // finds in the cache: 4096 x 7168 58.5 us past it, 54.5 so)
    if constexpr (BF16) {
        o.v[0] = ld_stream16(b);
    } else {
        o.v[0] = *reinterpret_cast<const uint4 *>(b);
        o.v[1] = *reinterpret_cast<const uint4 *>(b + 16);
    }
    return o;
}
template <bool BF16> __device__ __forceinline__ void widen(const Raw8<BF16> &o, float (&f)[8])
{
    if constexpr (BF16) {
        const uint32_t u[4] = {o.v[0].x, o.v[0].y, o.v[0].z, o.v[0].w};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            f[2 * i] = bf16lo(u[i]);
            f[2 * i + 1] = bf16hi(u[i]);
        }
    } else {
        __builtin_memcpy(f, o.v, 32);
    }
}
// Eight values into a Raw8 (BF16: to nearest even).
template <bool BF16> __device__ __forceinline__ Raw8<BF16> narrow(const float (&f)[8])
{
    Raw8<BF16> o;
    if constexpr (BF16)
        o.v[0] = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                            pack_bf16x2(f[6], f[7]));
    else
        __builtin_memcpy(o.v, f, 32);
    return o;
}
template <bool BF16> __device__ __forceinline__ void store8(void *p, int64_t at, const Raw8<BF16> &o)
{
    uint8_t *b = (uint8_t *)p + at * (BF16 ? 2 : 4);
    st_plain16(b, o.v[0]);
    if constexpr (!BF16)
        st_plain16(b + 16, o.v[1]);
}
__device__ __forceinline__ void load_weight(const void *w, int bf16, int64_t at, float (&f)[8])
{
    if (bf16) {
        Raw8<true> o;
        o.v[0] = *reinterpret_cast<const uint4 *>((const uint16_t *)w + at);
        widen<true>(o, f);
    } else {
        __builtin_memcpy(f, (const float *)w + at, 32);
    }
}

__device__ __forceinline__ float wave_sum(float v)
{
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1)
        v += __shfl_xor(v, d);
    return v;
}

// The sum over a row's W waves; every lane gets it, the waves' parts added in order.
// red: a slot a wave, taken in turn by even and odd rows, so one barrier a row is enough.
template <int W> __device__ __forceinline__ float row_sum(float v, float *red)
{
    v = wave_sum(v);
    if constexpr (W == 1)
        return v;
    if (lane_id() == 0)
        red[threadIdx.x >> 6] = v;
    __syncthreads();
    float t = red[0];
#pragma unroll
    for (int i = 1; i < W; i++)
        t += red[i];
    return t;
}

template <int W> constexpr int NORM_THREADS = W == 1 ? 256 : 64 * W;
template <int W> constexpr int NORM_ROWS = W == 1 ? 4 : 1; // rows of a workgroup at a time

// Chunk u's first column in this lane, and where it is loaded from: lanes past the last
// column load the last chunk once more, so that the loads of a row are issued together.
template <int W> __device__ __forceinline__ int chunk_col(int u, int t) { return 8 * (u * 64 * W + t); }
template <bool BF16, int W, int CH>
__device__ __forceinline__ void load_row(Raw8<BF16> (&o)[CH], const void *p, int64_t at, int cols, int t)
{
#pragma unroll
    for (int u = 0; u < CH; u++)
        o[u] = load8<BF16>(p, at + min(chunk_col<W>(u, t), cols - 8));
}

template <bool XBF, bool HBF, bool RES, int W, int CH>
__global__ __launch_bounds__(NORM_THREADS<W>) void rmsnorm_kernel(NormArgs a)
{
    __shared__ float red[2][16];
    const int t = threadIdx.x % (64 * W); // lane of the row
    int odd = 0;
    const int64_t first = (int64_t)blockIdx.x * NORM_ROWS<W> + (W == 1 ? threadIdx.x >> 6 : 0);
    Raw8<XBF> x[CH];
    Raw8<HBF> r[CH];
    for (int64_t row = first; row < a.rows; row += (int64_t)gridDim.x * NORM_ROWS<W>) {
        load_row<XBF, W>(x, a.x, row * a.ldx, a.cols, t);
        if constexpr (RES)
            load_row<HBF, W>(r, a.r, row * a.ldr, a.cols, t);
        float f[CH][8];
        float sum = 0.0f;
#pragma unroll
        for (int u = 0; u < CH; u++) {
            const int c = chunk_col<W>(u, t);
            widen<XBF>(x[u], f[u]);
            if constexpr (RES) {
                float v[8];
                widen<HBF>(r[u], v);
#pragma unroll
                for (int i = 0; i < 8; i++)
                    v[i] = f[u][i] + v[i];
                const Raw8<HBF> h = narrow<HBF>(v); // the norm is that of the stream as it is stored
                if (c < a.cols)
                    store8<HBF>(a.h, row * a.ldh + c, h);
                widen<HBF>(h, f[u]);
            }
            float part = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; i++)
                part = fmaf(f[u][i], f[u][i], part);
            sum += c < a.cols ? part : 0.0f;
        }
        sum = row_sum<W>(sum, red[odd]);
        odd ^= 1;
        const float rstd = 1.0f / sqrtf(sum / (float)a.cols + a.eps);
        if (t == 0)
            a.rstd[row] = rstd;
#pragma unroll
        for (int u = 0; u < CH; u++) {
            const int c = chunk_col<W>(u, t);
            if (c < a.cols) { // (whole groups of lanes: cols is a multiple of the group)
                float w[8], y[8];
                load_weight(a.w, a.w_bf16, c, w);
                uint32_t m = 0;
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    y[i] = f[u][i] * rstd * w[i];
                    m = max(m, __float_as_uint(y[i]) & 0x7FFFFFFFu);
                }
                if (a.y) {
                    if (a.y_bf16)
                        store8<true>(a.y, row * a.ldy + c, narrow<true>(y));
                    else
                        store8<false>(a.y, row * a.ldy + c, narrow<false>(y));
                }
                if (a.q) {
                    m = group_max_u32<4>(m);
                    if (a.group == 128) { // uniform
                        m = max(m, dpp<FGB_DPP_HALF_MIRROR>(m));
                        m = max(m, dpp<FGB_DPP_ROW_ROR8>(m));
                    }
                    const int e = scale_exp_from_bits(m, a.emin);
                    const float sc = pow2f(-e);
                    const uint2 o = make_uint2(cvt4_e4m3(y[0] * sc, y[1] * sc, y[2] * sc, y[3] * sc),
                                               cvt4_e4m3(y[4] * sc, y[5] * sc, y[6] * sc, y[7] * sc));
                    *reinterpret_cast<uint2 *>(a.q + row * a.cols + c) = o;
                    if (c % a.group == 0)
                        a.s[row * (a.cols / a.group) + c / a.group] = (uint8_t)(e + 127);
                }
            }
        }
    }
}

// A row's gradient from registers.
template <bool HBF> __device__ __forceinline__ void store_dx(const NormGradArgs &a, int64_t at, const float (&d)[8],
                                                             const float (&h)[8], const float (&e)[8], float rstd, float mean)
{
    float o[8];
#pragma unroll
    for (int i = 0; i < 8; i++)
        o[i] = fmaf(rstd, fmaf(h[i], -mean, d[i]), e[i]);
    store8<HBF>(a.dx, at, narrow<HBF>(o));
}

// Sixteen waves have 128 registers a lane, which a row and its part of dw do not fit: they read
// the row again after the sum (4096 x 32768 BF16: 304 us under a trace, from registers that spill
// 720).
template <bool DBF, bool HBF, int W, int CH>
__global__ __launch_bounds__(NORM_THREADS<W>) void rmsnorm_grad_kernel(NormGradArgs a)
{
    constexpr bool AGAIN = W == 16;
    __shared__ float red[2][16];
    const int t = threadIdx.x % (64 * W);
    const int64_t first = (int64_t)blockIdx.x * NORM_ROWS<W> + (W == 1 ? threadIdx.x >> 6 : 0);
    if (W == 1 && first >= a.parts) // (a whole wave, and no barrier follows)
        return;
    float w[AGAIN ? 1 : CH][8], dw[CH][8];
#pragma unroll
    for (int u = 0; u < CH; u++) {
        const int c = chunk_col<W>(u, t);
#pragma unroll
        for (int i = 0; i < 8; i++) {
            dw[u][i] = 0.0f;
            if constexpr (!AGAIN)
                w[u][i] = 0.0f; // (columns past the last one: not stored, not summed)
        }
        if constexpr (!AGAIN)
            if (c < a.cols)
                load_weight(a.w, a.w_bf16, c, w[u]);
    }
    int odd = 0;
    for (int64_t row = first; row < a.rows; row += a.parts) {
        const float rstd = a.rstd[row];
        float sum = 0.0f;
        if constexpr (AGAIN) {
#pragma unroll 1
            for (int u = 0; u < CH; u++) {
                const int c = chunk_col<W>(u, t);
                if (c < a.cols) {
                    float d[8], h[8];
                    widen<DBF>(load8<DBF>(a.dy, row * a.lddy + c), d);
                    widen<HBF>(load8<HBF>(a.h, row * a.ldh + c), h);
                    load_weight(a.w, a.w_bf16, c, w[0]);
#pragma unroll
                    for (int i = 0; i < 8; i++)
                        sum = fmaf(d[i] * w[0][i], h[i] * rstd, sum);
                }
            }
            const float mean = row_sum<W>(sum, red[odd]) / (float)a.cols;
            odd ^= 1;
#pragma unroll
            for (int u = 0; u < CH; u++) {
                const int c = chunk_col<W>(u, t);
                if (c < a.cols) {
                    float d[8], h[8], e[8] = {};
                    widen<DBF>(load8<DBF>(a.dy, row * a.lddy + c), d);
                    widen<HBF>(load8<HBF>(a.h, row * a.ldh + c), h);
                    if (a.dh)
                        widen<HBF>(load8<HBF>(a.dh, row * a.lddh + c), e);
                    load_weight(a.w, a.w_bf16, c, w[0]);
#pragma unroll
                    for (int i = 0; i < 8; i++) {
                        h[i] *= rstd;
                        dw[u][i] = fmaf(d[i], h[i], dw[u][i]);
                        d[i] *= w[0][i];
                    }
                    store_dx<HBF>(a, row * a.lddx + c, d, h, e, rstd, mean);
                }
                __builtin_amdgcn_sched_barrier(0); // (a chunk at a time, for its registers)
            }
        } else {
            Raw8<DBF> rd[CH];
            Raw8<HBF> rh[CH], re[CH];
            load_row<DBF, W>(rd, a.dy, row * a.lddy, a.cols, t);
            load_row<HBF, W>(rh, a.h, row * a.ldh, a.cols, t);
            if (a.dh)
                load_row<HBF, W>(re, a.dh, row * a.lddh, a.cols, t);
            float d[CH][8], h[CH][8], e[CH][8];
#pragma unroll
            for (int u = 0; u < CH; u++) {
                widen<DBF>(rd[u], d[u]);
                widen<HBF>(rh[u], h[u]);
                if (a.dh)
                    widen<HBF>(re[u], e[u]);
                const float before = sum;
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    h[u][i] *= rstd;
                    dw[u][i] = fmaf(d[u][i], h[u][i], dw[u][i]);
                    d[u][i] *= w[u][i];
                    sum = fmaf(d[u][i], h[u][i], sum);
                    if (!a.dh)
                        e[u][i] = 0.0f;
                }
                // (a weight of 0 does not keep out the infinities of columns that are loaded once more)
                sum = chunk_col<W>(u, t) < a.cols ? sum : before;
            }
            const float mean = row_sum<W>(sum, red[odd]) / (float)a.cols;
            odd ^= 1;
#pragma unroll
            for (int u = 0; u < CH; u++) {
                const int c = chunk_col<W>(u, t);
                if (c < a.cols)
                    store_dx<HBF>(a, row * a.lddx + c, d[u], h[u], e[u], rstd, mean);
            }
        }
    }
#pragma unroll
    for (int u = 0; u < CH; u++) {
        const int c = chunk_col<W>(u, t);
        if (c < a.cols) {
            float *p = a.part + first * a.cols + c;
            *reinterpret_cast<float4 *>(p) = make_float4(dw[u][0], dw[u][1], dw[u][2], dw[u][3]);
            *reinterpret_cast<float4 *>(p + 4) = make_float4(dw[u][4], dw[u][5], dw[u][6], dw[u][7]);
        }
    }
}

// dw: the sum of the parts, 32 columns a workgroup, 32 threads a column, in a fixed order.
__global__ __launch_bounds__(1024) void rmsnorm_dw_kernel(NormGradArgs a)
{
    __shared__ float red[32][33];
    const int col = threadIdx.x & 31, slice = threadIdx.x >> 5, c = blockIdx.x * 32 + col;
    const float *p = a.part + c; // (cols is a multiple of 32)
    float v = 0.0f;
    for (int i = slice; i < a.parts; i += 32 * 8) { // eight loads together, the last part again past the end
        float f[8];
#pragma unroll
        for (int k = 0; k < 8; k++)
            f[k] = p[(int64_t)min(i + 32 * k, a.parts - 1) * a.cols];
#pragma unroll
        for (int k = 0; k < 8; k++)
            v += i + 32 * k < a.parts ? f[k] : 0.0f;
    }
    red[slice][col] = v;
    __syncthreads();
    if (threadIdx.x < 32) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; i++)
            s += red[i][col];
        a.dw[c] = s;
    }
}

static int norm_waves(int64_t cols) { return cols <= 2048 ? 1 : cols <= 8192 ? 4 : cols <= 16384 ? 8 : 16; }
static bool norm_two_chunks(int64_t cols) { return cols <= 1024 * norm_waves(cols); }

// Rows that add up separately for dw: a wave's, or a workgroup's for two a CU (more than 8192
// columns: one; 4096 x 16384 97 + 5 us, with two 102 + 7).
static int64_t norm_parts(int64_t rows, int64_t cols)
{
    const int64_t most = norm_waves(cols) == 1 ? 2048 : cols <= 8192 ? 512 : 256;
    return rows < 1 ? 1 : rows < most ? rows : most;
}

static int check_norm(const char *name, int64_t rows, int64_t cols)
{
    FGB_REQUIRE(rows >= 0 && cols > 0 && cols % 32 == 0 && cols <= 32768, FGB_EINVAL,
                "%s: cols must be a multiple of 32 up to 32768 (rows=%lld cols=%lld)", name, (long long)rows,
                (long long)cols);
    return FGB_OK;
}
static int check_rows(const char *name, const char *what, const void *p, int dtype, int64_t cols, int64_t ld)
{
    FGB_REQUIRE(dtype == FGB_F32 || dtype == FGB_BF16, FGB_EUNSUPPORTED, "%s: %s must be FGB_F32 or FGB_BF16", name, what);
    FGB_REQUIRE(p, FGB_EINVAL, "%s: %s is null", name, what);
    FGB_REQUIRE(ld >= cols && ld * (dtype == FGB_BF16 ? 2 : 4) % 16 == 0 && aligned16(p), FGB_EINVAL,
                "%s: %s must be 16-byte aligned with a row stride >= cols that is a multiple of 16 bytes", name, what);
    return FGB_OK;
}

// Rows in memory that a call reads or writes: `rows` of them of `bytes`, `ld` bytes apart.
struct Rows {
    const char *name;
    uintptr_t p;
    int64_t rows, bytes, ld;
};
static Rows rows_at(const char *name, const void *p, int64_t rows, int64_t cols, int64_t ld, int dtype)
{
    const int each = dtype == FGB_BF16 ? 2 : 4;
    return {name, (uintptr_t)p, p ? rows : 0, cols * each, ld * each};
}
static Rows bytes_at(const char *name, const void *p, int64_t bytes) { return {name, (uintptr_t)p, p ? 1 : 0, bytes, bytes}; }

// Whether two of them share a byte.  Views of one buffer (one row stride) are compared at once,
// as rows i of a and j of b meet or not by i - j alone; others a row of the shorter at a time.
static bool share(const Rows &a, const Rows &b)
{
    if (a.rows > b.rows)
        return share(b, a);
    if (a.rows < 1 || a.bytes < 1 || b.bytes < 1)
        return false;
    const int64_t lda = a.rows == 1 ? b.ld : a.ld, to = (int64_t)(b.p - a.p); // (b.p from a.p)
    if (to >= (a.rows - 1) * lda + a.bytes || to + (b.rows - 1) * b.ld + b.bytes <= 0)
        return false;
    // the first row of b that ends behind row i of a
    const auto meets = [&](int64_t i) {
        const int64_t past = i * lda - to - b.bytes, j = past < 0 ? 0 : past / b.ld + 1;
        return j < b.rows && to + j * b.ld < i * lda + a.bytes;
    };
    if (lda == b.ld && a.bytes <= lda) {
        // with i - j = m: m ld < to + b.bytes and m ld + a.bytes > to
        const int64_t q = to / b.ld;
        for (int64_t m = q - 2; m <= q + 2; m++)
            if (m > -b.rows && m < a.rows && m * b.ld < to + b.bytes && m * b.ld + a.bytes > to)
                return true;
        return false;
    }
    for (int64_t i = 0; i < a.rows; i++)
        if (meets(i))
            return true;
    return false;
}
// The very same rows: what an output may be of an input, as a row is written after it was read.
static bool same(const Rows &a, const Rows &b)
{
    return a.p == b.p && a.bytes == b.bytes && (a.ld == b.ld || a.rows == 1);
}
static int check_apart(const char *name, const Rows &out, const Rows &other)
{
    FGB_REQUIRE(!share(out, other), FGB_EINVAL, "%s: %s lies over %s", name, out.name, other.name);
    return FGB_OK;
}
static int check_apart_or_same(const char *name, const Rows &out, const Rows &in)
{
    return same(out, in) ? FGB_OK : check_apart(name, out, in);
}

// The variant by the columns: waves a row and chunks a lane.
#define FGB_NORM_VARIANT(COLS, LAUNCH)                                                                                 \
    do {                                                                                                               \
        const bool two_ = norm_two_chunks(COLS);                                                                       \
        switch (norm_waves(COLS)) {                                                                                    \
        case 1:                                                                                                        \
            if (two_) { LAUNCH(1, 2); } else { LAUNCH(1, 4); }                                                         \
            break;                                                                                                     \
        case 4:                                                                                                        \
            if (two_) { LAUNCH(4, 2); } else { LAUNCH(4, 4); }                                                         \
            break;                                                                                                     \
        case 8:                                                                                                        \
            LAUNCH(8, 4);                                                                                              \
            break;                                                                                                     \
        default:                                                                                                       \
            LAUNCH(16, 4);                                                                                             \
        }                                                                                                              \
    } while (0)

template <bool XBF, bool HBF, bool RES> static void launch_norm(const NormArgs &a, hipStream_t st)
{
#define FGB_N(W, CH)                                                                                                   \
    do {                                                                                                               \
        const int64_t n = (a.rows + NORM_ROWS<W> - 1) / NORM_ROWS<W>; /* eight workgroups a CU take rows in turn:   */ \
        /* 8192 x 7168 with a reader of the codes 96 us, a workgroup a row 101.5, 1536 of them 107 */                  \
        rmsnorm_kernel<XBF, HBF, RES, W, CH>                                                                           \
            <<<(unsigned)(n < 2048 ? n : 2048), NORM_THREADS<W>, 0, st>>>(a);                                          \
    } while (0)
    FGB_NORM_VARIANT(a.cols, FGB_N);
#undef FGB_N
}

template <bool DBF, bool HBF> static void launch_norm_grad(const NormGradArgs &a, hipStream_t st)
{
#define FGB_N(W, CH)                                                                                                   \
    rmsnorm_grad_kernel<DBF, HBF, W, CH>                                                                               \
        <<<(unsigned)((a.parts + NORM_ROWS<W> - 1) / NORM_ROWS<W>), NORM_THREADS<W>, 0, st>>>(a)
    FGB_NORM_VARIANT(a.cols, FGB_N);
#undef FGB_N
}

} // namespace fgb

using namespace fgb;

extern "C" int rmsnorm_quant(const void *x, int x_dtype, int64_t rows, int64_t cols, int64_t ldx, const void *residual,
                             int r_dtype, int64_t ldr, const void *weight, int w_dtype, float eps, int group, void *h,
                             int64_t ldh, float *rstd, uint8_t *q, uint8_t *s, void *y, int y_dtype, int64_t ldy,
                             void *stream)
{
    clear_error();
    const char *name = "rmsnorm_quant";
    int rc = check_norm(name, rows, cols);
    if (rc != FGB_OK)
        return rc;
    FGB_REQUIRE(group == 128 || group == 32, FGB_EUNSUPPORTED, "%s: group must be 128 or 32", name);
    FGB_REQUIRE(eps > 0.0f, FGB_EINVAL, "%s: eps must be positive", name);
    if (rows == 0)
        return FGB_OK;
    FGB_REQUIRE(!q || cols % group == 0, FGB_EINVAL, "%s: cols must be a multiple of the group", name);
    FGB_REQUIRE((q != nullptr) == (s != nullptr) && (q || y), FGB_EINVAL,
                "%s: codes and scales come together, and they or y must be asked for", name);
    if ((rc = check_rows(name, "x", x, x_dtype, cols, ldx)) != FGB_OK ||
        (rc = check_rows(name, "weight", weight, w_dtype, cols, (cols + 7) & ~7)) != FGB_OK)
        return rc;
    if (residual && ((rc = check_rows(name, "residual", residual, r_dtype, cols, ldr)) != FGB_OK ||
                     (rc = check_rows(name, "h", h, r_dtype, cols, ldh)) != FGB_OK))
        return rc;
    if (y && (rc = check_rows(name, "y", y, y_dtype, cols, ldy)) != FGB_OK)
        return rc;
    FGB_REQUIRE(aligned16(q), FGB_EINVAL, "%s: q must be 16-byte aligned", name);
    const Rows ins[] = {rows_at("x", x, rows, cols, ldx, x_dtype), rows_at("residual", residual, rows, cols, ldr, r_dtype)};
    const Rows outs[] = {rows_at("h", residual ? h : nullptr, rows, cols, ldh, r_dtype), rows_at("y", y, rows, cols, ldy, y_dtype),
                         bytes_at("q", q, rows * cols), bytes_at("s", s, rows * (cols / group)), bytes_at("rstd", rstd, 4 * rows)};
    const Rows w_rows = rows_at("weight", weight, 1, cols, cols, w_dtype);
    for (int i = 0; i < 5; i++) {
        for (const Rows &in : ins)
            if ((rc = i < 2 ? check_apart_or_same(name, outs[i], in) : check_apart(name, outs[i], in)) != FGB_OK)
                return rc;
        if ((rc = check_apart(name, outs[i], w_rows)) != FGB_OK)
            return rc;
        for (int j = 0; j < i; j++)
            if ((rc = check_apart(name, outs[i], outs[j])) != FGB_OK)
                return rc;
    }
    FGB_REQUIRE(rstd && ((uintptr_t)rstd & 3) == 0, FGB_EINVAL, "%s: rstd null or misaligned", name);
    NormArgs a{};
    a.x = x; a.r = residual; a.w = weight; a.h = h; a.y = y; a.q = q; a.s = s; a.rstd = rstd;
    a.rows = rows; a.ldx = ldx; a.ldr = ldr; a.ldh = ldh; a.ldy = ldy; a.cols = (int)cols;
    a.eps = eps; a.w_bf16 = w_dtype == FGB_BF16; a.y_bf16 = y_dtype == FGB_BF16;
    a.group = group; a.emin = group == 128 ? -22 : -127;
    const bool xb = x_dtype == FGB_BF16, rb = r_dtype == FGB_BF16;
    const hipStream_t st = (hipStream_t)stream;
    if (!residual)
        xb ? launch_norm<true, true, false>(a, st) : launch_norm<false, false, false>(a, st);
    else if (xb)
        rb ? launch_norm<true, true, true>(a, st) : launch_norm<true, false, true>(a, st);
    else
        rb ? launch_norm<false, true, true>(a, st) : launch_norm<false, false, true>(a, st);
    FGB_LAUNCHED("rmsnorm_kernel");
    return FGB_OK;
}

extern "C" size_t rmsnorm_backward_workspace_size(int64_t rows, int64_t cols)
{
    if (rows < 0 || cols <= 0 || cols > 32768)
        return 0;
    return (size_t)norm_parts(rows, cols) * (size_t)cols * 4;
}

extern "C" int rmsnorm_backward(const void *dy, int dy_dtype, int64_t rows, int64_t cols, int64_t lddy, const void *h,
                                int h_dtype, int64_t ldh, const void *weight, int w_dtype, const float *rstd,
                                const void *dh, int64_t lddh, void *dx, int64_t lddx, float *dweight, void *workspace,
                                size_t ws_bytes, void *stream)
{
    clear_error();
    const char *name = "rmsnorm_backward";
    int rc = check_norm(name, rows, cols);
    if (rc != FGB_OK)
        return rc;
    if (rows > 0 && ((rc = check_rows(name, "dy", dy, dy_dtype, cols, lddy)) != FGB_OK ||
                     (rc = check_rows(name, "h", h, h_dtype, cols, ldh)) != FGB_OK ||
                     (rc = check_rows(name, "dx", dx, h_dtype, cols, lddx)) != FGB_OK))
        return rc;
    if (rows > 0 && dh && (rc = check_rows(name, "dh", dh, h_dtype, cols, lddh)) != FGB_OK)
        return rc;
    if ((rc = check_rows(name, "weight", weight, w_dtype, cols, (cols + 7) & ~7)) != FGB_OK)
        return rc;
    FGB_REQUIRE(dweight && ((uintptr_t)dweight & 3) == 0 && (rows == 0 || (rstd && ((uintptr_t)rstd & 3) == 0)),
                FGB_EINVAL, "%s: dweight or rstd null or misaligned", name);
    const size_t need = rmsnorm_backward_workspace_size(rows, cols);
    FGB_REQUIRE(workspace && ws_bytes >= need, FGB_EWORKSPACE, "%s: workspace of %zu bytes needed", name, need);
    const Rows dx_rows = rows_at("dx", dx, rows, cols, lddx, h_dtype), w_rows = rows_at("weight", weight, 1, cols, cols, w_dtype);
    const Rows part = bytes_at("workspace", workspace, (int64_t)need), scale = bytes_at("rstd", rstd, 4 * rows);
    const Rows sum = bytes_at("dweight", dweight, 4 * cols);
    const Rows ins[] = {rows_at("dy", dy, rows, cols, lddy, dy_dtype), rows_at("h", h, rows, cols, ldh, h_dtype),
                        rows_at("dh", dh, rows, cols, lddh, h_dtype)};
    for (const Rows &in : ins)
        if ((rc = check_apart_or_same(name, dx_rows, in)) != FGB_OK || (rc = check_apart(name, part, in)) != FGB_OK)
            return rc;
    for (const Rows *other : {&w_rows, &scale, &sum})
        if ((rc = check_apart(name, dx_rows, *other)) != FGB_OK || (rc = check_apart(name, part, *other)) != FGB_OK)
            return rc;
    if ((rc = check_apart(name, part, dx_rows)) != FGB_OK)
        return rc;
    FGB_REQUIRE(aligned16(workspace), FGB_EINVAL, "%s: workspace must be 16-byte aligned", name);
    NormGradArgs a{};
    a.dy = dy; a.h = h; a.w = weight; a.dh = dh; a.rstd = rstd; a.dx = dx;
    a.part = (float *)workspace; a.dw = dweight;
    a.rows = rows; a.lddy = lddy; a.ldh = ldh; a.lddh = lddh; a.lddx = lddx; a.cols = (int)cols;
    a.w_bf16 = w_dtype == FGB_BF16; a.parts = (int)norm_parts(rows, cols);
    const bool db = dy_dtype == FGB_BF16, hb = h_dtype == FGB_BF16;
    const hipStream_t st = (hipStream_t)stream;
    if (db)
        hb ? launch_norm_grad<true, true>(a, st) : launch_norm_grad<true, false>(a, st);
    else
        hb ? launch_norm_grad<false, true>(a, st) : launch_norm_grad<false, false>(a, st);
    FGB_LAUNCHED("rmsnorm_grad_kernel");
    rmsnorm_dw_kernel<<<(unsigned)(cols / 32), 1024, 0, st>>>(a);
    FGB_LAUNCHED("rmsnorm_dw_kernel");
    return FGB_OK;
}
