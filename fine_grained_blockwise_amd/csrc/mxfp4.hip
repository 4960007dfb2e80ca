// mxfp4.hip -- MXFP4: E2M1 codes with one power-of-two scale per 32 elements.
//
// An element is sign, two exponent bits (bias 1) and one mantissa bit: the
// magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6.  A group of 32 consecutive columns
// shares the scale 2^e.  With amax = (1 + f) 2^Ea over the group, the ceil rule
// takes the smallest e with amax <= 6 * 2^e = 1.5 * 2^(e + 2), i.e. Ea - 2, or
// Ea - 1 where f > 1/2; the MX standard's floor rule takes Ea - 2 and lets the
// largest elements clip at 6.  x * 2^-e is exact in fp32, and the hardware
// conversion rounds it to nearest even and saturates; both were checked on
// gfx950 against that definition over codes, ties, signs and exponents.  A group
// with an infinity or NaN gets the scale byte 255 (E8M0's NaN), so what reads it
// sees NaN instead of a silently clipped value.
#include "fgb_internal.h"

namespace fgb {

// Scale byte of a group from the fp32 bits of its amax.
template <int RULE> __device__ __forceinline__ uint32_t mxfp4_scale_byte(uint32_t amax_bits)
{
    if (amax_bits >= 0x7F800000u)
        return 255;
    int e = (int)(amax_bits >> 23) - 127 - 2;
    if constexpr (RULE == RULE_CEIL)
        e += (amax_bits & 0x7FFFFFu) > 0x400000u ? 1 : 0;
    e = amax_bits < 0x00800000u || e < -127 ? -127 : e;
    return (uint32_t)(e + 127);
}

// Eight values / 2^(b - 127) -> eight codes, value i in bits 4i .. 4i+3.  The
// conversion divides by the power of two whose fp32 exponent field its scale
// operand holds (field 0 meaning 2^-127), rounds to nearest even and clips at 6.
__device__ __forceinline__ uint32_t mxfp4_encode8(const float (&v)[8], uint32_t b)
{
    const float sc = __uint_as_float(b << 23);
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], sc, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], sc, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], sc, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], sc, 3);
    return w;
}

// Eight consecutive elements of a row as fp32.
template <bool BF16> __device__ __forceinline__ void load8(const void *x, int64_t at, float (&v)[8])
{
    if constexpr (BF16) {
        const uint4 u = *reinterpret_cast<const uint4 *>((const uint16_t *)x + at);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            v[2 * i] = bf16lo(w[i]);
            v[2 * i + 1] = bf16hi(w[i]);
        }
    } else {
        const float4 a = *reinterpret_cast<const float4 *>((const float *)x + at);
        const float4 b = *reinterpret_cast<const float4 *>((const float *)x + at + 4);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
}

__device__ __forceinline__ uint32_t amax8(const float (&v)[8])
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; i++)
        m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    return m;
}

// Scales are stored step-major: byte j of entry (i, r) is group 8 i + j of row r
// (columns 256 i + 32 j ..).  A matrix tile's scales for 256 columns are then one
// contiguous run, 8 bytes a row.
__device__ __forceinline__ int64_t scale_at(int64_t row, int64_t group, int64_t rows)
{
    return ((group >> 3) * rows + row) * 8 + (group & 7);
}

// Four lanes per group, eight elements per lane.  HBM-bound: 2 (4) bytes read
// and 17/32 written per element.
template <bool BF16, int RULE>
__global__ __launch_bounds__(256) void mxfp4_quant_kernel(const void *x, int64_t all, int64_t rows, int64_t cols,
                                                          int64_t ldx, uint8_t *q, uint8_t *s)
{
    const int64_t ng = cols / 32, ngp = (cols + 255) / 256 * 8; // groups, and with the last step's unused bytes
    const int64_t item = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> 2;
    const int sub = threadIdx.x & 3;
    if (item >= all * ngp)
        return; // whole quads
    const int64_t row = item / ngp, g = item % ngp; // row of all stacked matrices
    uint32_t b = 0;
    if (g < ng) {
        float v[8];
        load8<BF16>(x, row * ldx + g * 32 + sub * 8, v);
        b = mxfp4_scale_byte<RULE>(group_max_u32<4>(amax8(v)));
        *reinterpret_cast<uint32_t *>(q + (row * cols + g * 32) / 2 + sub * 4) = mxfp4_encode8(v, b);
    }
    if (sub == 0)
        s[row / rows * rows * ngp + scale_at(row % rows, g, rows)] = (uint8_t)b;
}

// Both directions from one read: a workgroup takes 128 rows x 128 columns,
// quantises the rows as it reads them, keeps the values in LDS and quantises the
// columns from there.  Row r of the tile starts at word r * 128 + (r / 32) * 16,
// so the four 32-row groups of a column, read by neighbouring lanes, sit 16 banks
// apart.
constexpr int QT = 128;
template <bool BF16, int RULE>
__global__ __launch_bounds__(256) void mxfp4_quant_t_kernel(const void *x, int64_t rows, int64_t cols, int64_t ldx,
                                                            uint8_t *q, uint8_t *s, uint8_t *qt, uint8_t *st)
{
    __shared__ float tile[QT * QT + 64];
    const int64_t r0 = (int64_t)blockIdx.y * QT, c0 = (int64_t)blockIdx.x * QT;
    const int64_t rows_p = (rows + 31) / 32 * 32, z = blockIdx.z; // matrix z of the stack
    x = BF16 ? (const void *)((const uint16_t *)x + z * rows * ldx) : (const void *)((const float *)x + z * rows * ldx);
    q += z * rows * (cols / 2);
    s += z * ((cols + 255) / 256) * rows * 8;
    qt += z * cols * (rows_p / 2);
    st += z * ((rows + 255) / 256) * cols * 8;
    // rows: 16 lanes x 8 elements cover the tile's 128 columns, 16 rows a pass
    const int lr = threadIdx.x >> 4, lc = threadIdx.x & 15;
    const int64_t col = c0 + lc * 8;
    for (int p = 0; p < QT / 16; p++) {
        const int r = p * 16 + lr;
        const int64_t row = r0 + r;
        float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        const bool in = row < rows && col < cols; // whole quads (32 columns)
        if (in)
            load8<BF16>(x, row * ldx + col, v);
        const uint32_t b = mxfp4_scale_byte<RULE>(group_max_u32<4>(amax8(v)));
        if (in) {
            *reinterpret_cast<uint32_t *>(q + (row * cols + col) / 2) = mxfp4_encode8(v, b);
            if ((lc & 3) == 0)
                s[scale_at(row, col / 32, rows)] = (uint8_t)b;
        } else if (row < rows && col < (cols + 255) / 256 * 256 && (lc & 3) == 0) {
            s[scale_at(row, col / 32, rows)] = 0; // the last step's unused bytes
        }
#pragma unroll
        for (int i = 0; i < 8; i++)
            tile[r * QT + (r >> 5) * 16 + lc * 8 + i] = v[i];
    }
    __syncthreads();
    // columns: lane = 4 * column + row group, 64 columns a pass
    const int64_t gt = (rows + 255) / 256 * 8; // row groups with the last step's unused bytes
    for (int p = 0; p < 2; p++) {
        const int c = p * 64 + (threadIdx.x >> 2), g = threadIdx.x & 3;
        const int64_t ct = c0 + c, gr = r0 / 32 + g;
        if (ct >= cols)
            continue;
        float v[32];
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 32; i++) {
            v[i] = tile[(g * 32 + i) * QT + g * 16 + c];
            m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
        }
        const uint32_t b = mxfp4_scale_byte<RULE>(m);
        if (gr * 32 < rows) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; k++) {
                float u[8];
#pragma unroll
                for (int i = 0; i < 8; i++)
                    u[i] = v[8 * k + i];
                w[k] = mxfp4_encode8(u, b);
            }
            *reinterpret_cast<uint4 *>(qt + (ct * rows_p) / 2 + gr * 16) = make_uint4(w[0], w[1], w[2], w[3]);
            st[scale_at(ct, gr, cols)] = (uint8_t)b;
        } else if (gr < gt) {
            st[scale_at(ct, gr, cols)] = 0;
        }
    }
    // A last tile of up to 128 rows leaves the step's other half, if it starts one.
    if (blockIdx.y == gridDim.y - 1 && (gridDim.y & 1)) {
        const int c = threadIdx.x >> 1, h = threadIdx.x & 1;
        if (c0 + c < cols)
            *reinterpret_cast<uint16_t *>(st + scale_at(c0 + c, r0 / 32 + 4 + 2 * h, cols)) = 0;
    }
    if (blockIdx.x == gridDim.x - 1 && (gridDim.x & 1)) {
        const int r = threadIdx.x >> 1, h = threadIdx.x & 1;
        if (r0 + r < rows)
            *reinterpret_cast<uint16_t *>(s + scale_at(r0 + r, c0 / 32 + 4 + 2 * h, rows)) = 0;
    }
}

// Eight codes per lane.
template <bool BF16>
__global__ __launch_bounds__(256) void mxfp4_dequant_kernel(const uint8_t *q, const uint8_t *s, int64_t rows,
                                                            int64_t cols, void *out)
{
    const int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
    if (at >= rows * cols)
        return;
    const int64_t row = at / cols, col = at % cols;
    const uint32_t w = *reinterpret_cast<const uint32_t *>(q + at / 2);
    const float sc = __uint_as_float((uint32_t)s[scale_at(row, col / 32, rows)] << 23);
    if constexpr (BF16) {
        uint4 o;
        o.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, sc, 0));
        o.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, sc, 1));
        o.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, sc, 2));
        o.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, sc, 3));
        st_plain16((uint16_t *)out + at, o);
    } else {
        const auto a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, sc, 0);
        const auto b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, sc, 1);
        const auto c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, sc, 2);
        const auto d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, sc, 3);
        float4 *o = reinterpret_cast<float4 *>((float *)out + at);
        o[0] = make_float4(a[0], a[1], b[0], b[1]);
        o[1] = make_float4(c[0], c[1], d[0], d[1]);
    }
}

static int check_quant(const char *name, const void *x, int x_dtype, int G, int64_t rows, int64_t cols, int64_t ldx, int rule,
                       const void *q, const void *s)
{
    FGB_REQUIRE(G >= 0 && rows >= 0 && cols >= 0 && cols % 32 == 0, FGB_EINVAL,
                "%s: need G, rows >= 0 and cols a multiple of 32 (G=%d rows=%lld cols=%lld)", name, G, (long long)rows,
                (long long)cols);
    FGB_REQUIRE(x_dtype == FGB_F32 || x_dtype == FGB_BF16, FGB_EUNSUPPORTED, "%s: x_dtype must be FGB_F32 or FGB_BF16",
                name);
    FGB_REQUIRE(rule == FGB_SCALE_CEIL || rule == FGB_SCALE_OCP_FLOOR, FGB_EUNSUPPORTED,
                "%s: rule must be FGB_SCALE_CEIL or FGB_SCALE_OCP_FLOOR", name);
    if (G == 0 || rows == 0 || cols == 0)
        return FGB_OK;
    FGB_REQUIRE(x && q && s, FGB_EINVAL, "%s: null pointer", name);
    FGB_REQUIRE(ldx >= cols && ldx % (x_dtype == FGB_BF16 ? 8 : 4) == 0, FGB_EINVAL,
                "%s: ldx must be >= cols and a multiple of 16 bytes", name);
    FGB_REQUIRE(aligned16(x) && aligned16(q) && aligned16(s), FGB_EINVAL, "%s: x, q and s must be 16-byte aligned",
                name);
    FGB_REQUIRE(rows < (1ll << 31) && cols < (1ll << 31) && G * rows < (1ll << 31) &&
                    G * rows * ((cols + 255) / 256) < (1ll << 33),
                FGB_EINVAL, "%s: too many elements", name);
    return FGB_OK;
}

} // namespace fgb

using namespace fgb;

#define FGB_BY_TYPE_AND_RULE(KERNEL, ...)                                                                              \
    do {                                                                                                               \
        if (x_dtype == FGB_BF16)                                                                                       \
            rule == FGB_SCALE_CEIL ? KERNEL<true, RULE_CEIL> __VA_ARGS__ : KERNEL<true, RULE_OCP_FLOOR> __VA_ARGS__;   \
        else                                                                                                           \
            rule == FGB_SCALE_CEIL ? KERNEL<false, RULE_CEIL> __VA_ARGS__ : KERNEL<false, RULE_OCP_FLOOR> __VA_ARGS__; \
    } while (0)

extern "C" int mxfp4_quant(const void *x, int x_dtype, int G, int64_t rows, int64_t cols, int64_t ldx, int rule, uint8_t *q,
                           uint8_t *s, void *stream)
{
    clear_error();
    const int rc = check_quant("mxfp4_quant", x, x_dtype, G, rows, cols, ldx, rule, q, s);
    if (rc != FGB_OK || G == 0 || rows == 0 || cols == 0)
        return rc;
    const int64_t grid = (G * rows * ((cols + 255) / 256 * 8) * 4 + 255) / 256;
    FGB_BY_TYPE_AND_RULE(mxfp4_quant_kernel, <<<(unsigned)grid, 256, 0, (hipStream_t)stream>>>(x, G * rows, rows, cols, ldx, q,
                                                                                             s));
    FGB_LAUNCHED("mxfp4_quant_kernel");
    return FGB_OK;
}

extern "C" int mxfp4_quant_t(const void *x, int x_dtype, int G, int64_t rows, int64_t cols, int64_t ldx, int rule, uint8_t *q,
                             uint8_t *s, uint8_t *qt, uint8_t *st, void *stream)
{
    clear_error();
    const int rc = check_quant("mxfp4_quant_t", x, x_dtype, G, rows, cols, ldx, rule, q, s);
    if (rc != FGB_OK || G == 0 || rows == 0 || cols == 0)
        return rc;
    FGB_REQUIRE(qt && st, FGB_EINVAL, "mxfp4_quant_t: null pointer");
    FGB_REQUIRE(aligned16(qt) && aligned16(st), FGB_EINVAL, "mxfp4_quant_t: qt and st must be 16-byte aligned");
    const int64_t gy = (rows + QT - 1) / QT;
    FGB_REQUIRE(gy < 65536 && G < 65536, FGB_EINVAL, "mxfp4_quant_t: rows must be below 2^23 and G below 2^16");
    const dim3 grid((unsigned)((cols + QT - 1) / QT), (unsigned)gy, (unsigned)G);
    FGB_BY_TYPE_AND_RULE(mxfp4_quant_t_kernel,
                         <<<grid, 256, 0, (hipStream_t)stream>>>(x, rows, cols, ldx, q, s, qt, st));
    FGB_LAUNCHED("mxfp4_quant_t_kernel");
    return FGB_OK;
}

extern "C" int mxfp4_dequant(const uint8_t *q, const uint8_t *s, int64_t rows, int64_t cols, void *out, int out_dtype,
                             void *stream)
{
    clear_error();
    FGB_REQUIRE(rows >= 0 && cols >= 0 && cols % 32 == 0, FGB_EINVAL,
                "mxfp4_dequant: need rows >= 0 and cols a multiple of 32");
    FGB_REQUIRE(out_dtype == FGB_F32 || out_dtype == FGB_BF16, FGB_EUNSUPPORTED,
                "mxfp4_dequant: out_dtype must be FGB_F32 or FGB_BF16");
    if (rows == 0 || cols == 0)
        return FGB_OK;
    FGB_REQUIRE(q && s && out, FGB_EINVAL, "mxfp4_dequant: null pointer");
    FGB_REQUIRE(aligned16(q) && aligned16(s) && aligned16(out), FGB_EINVAL,
                "mxfp4_dequant: q, s and out must be 16-byte aligned");
    FGB_REQUIRE(rows < (1ll << 31) && cols < (1ll << 31) && rows * (cols / 32) < (1ll << 33), FGB_EINVAL,
                "mxfp4_dequant: too many elements");
    const int64_t grid = (rows * cols / 8 + 255) / 256;
    if (out_dtype == FGB_BF16)
        mxfp4_dequant_kernel<true><<<(unsigned)grid, 256, 0, (hipStream_t)stream>>>(q, s, rows, cols, out);
    else
        mxfp4_dequant_kernel<false><<<(unsigned)grid, 256, 0, (hipStream_t)stream>>>(q, s, rows, cols, out);
    FGB_LAUNCHED("mxfp4_dequant_kernel");
    return FGB_OK;
}
