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

// Scales are stored step-major: byte j of entry (i, r) is group 8 i + j of row r
// (columns 256 i + 32 j ..).  A matrix tile's scales for 256 columns are then one
// contiguous run, 8 bytes a row.
__device__ __forceinline__ int64_t scale_at(int64_t row, int64_t group, int64_t rows)
{
    return ((group >> 3) * rows + row) * 8 + (group & 7);
}

// Eight bf16 (four words): the largest magnitude as fp32 bits, and the codes.  The
// pairs stay packed: bf16 magnitudes compare as 16-bit integers, and the conversion
// takes two bf16 at once.
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t max2_abs(uint32_t m, uint32_t w)
{
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, m),
                                                                  __builtin_bit_cast(u16x2, w & 0x7FFF7FFFu)));
}
__device__ __forceinline__ uint32_t max2_bits(uint32_t m) { return max(m << 16, m & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t encode8_bf16(const uint32_t (&w)[4], uint32_t b)
{
    const float sc = __uint_as_float(b << 23);
    uint32_t q = 0;
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2, w[0]), sc, 0);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2, w[1]), sc, 1);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2, w[2]), sc, 2);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2, w[3]), sc, 3);
    return q;
}

// A lane's eight consecutive elements: bf16 as four words, fp32 as eight.
template <bool BF16> struct Eight {
    uint32_t w[BF16 ? 4 : 8];
    __device__ __forceinline__ void load(const void *x, int64_t at)
    {
        const uint4 *p = reinterpret_cast<const uint4 *>((const uint8_t *)x + at * (BF16 ? 2 : 4));
#pragma unroll
        for (int i = 0; i < (BF16 ? 1 : 2); i++) {
            const uint4 u = BF16 ? ld_stream16(p + i) : p[i]; // (two half-lines a lane: through the cache)
            w[4 * i] = u.x;
            w[4 * i + 1] = u.y;
            w[4 * i + 2] = u.z;
            w[4 * i + 3] = u.w;
        }
    }
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < (BF16 ? 4 : 8); i++)
            w[i] = 0;
    }
    __device__ __forceinline__ uint32_t amax() const
    {
        uint32_t m = 0;
        if constexpr (BF16) {
#pragma unroll
            for (int i = 0; i < 4; i++)
                m = max2_abs(m, w[i]);
            return max2_bits(m);
        }
#pragma unroll
        for (int i = 0; i < (BF16 ? 4 : 8); i++)
            m = max(m, w[i] & 0x7FFFFFFFu);
        return m;
    }
    __device__ __forceinline__ uint32_t encode(uint32_t b) const
    {
        if constexpr (BF16) {
            return encode8_bf16(w, b);
        } else {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; i++)
                v[i] = __uint_as_float(w[i]);
            return mxfp4_encode8(v, b);
        }
    }
};

// The scale bytes of 16 lanes' four groups (a byte per quad of lanes) as one word.
__device__ __forceinline__ uint32_t four_bytes(uint32_t b)
{
    uint32_t v = b << (8 * ((threadIdx.x >> 2) & 3));
    v |= dpp<FGB_DPP_HALF_MIRROR>(v);
    v |= dpp<FGB_DPP_ROW_ROR8>(v);
    return v;
}

// Rows: a workgroup takes 32 rows x 256 columns (one scale step), a half-wave a row
// and four rows in flight, so that the step's scales leave as whole lines.  HBM-bound:
// 2 (4) bytes read and 17/32 written per element.  8192x28672 bf16: 103 us, 5.8 TB/s;
// fp32: 192 us, 5.5 TB/s.
template <bool BF16, int RULE>
__global__ __launch_bounds__(256) void mxfp4_quant_kernel(const void *x, int64_t rows, int64_t cols, int64_t ldx,
                                                          uint8_t *q, uint8_t *s, int steps, int tiles_m, int first)
{
    constexpr int U = 4;
    const int step = blockIdx.x % steps, tile = first + blockIdx.x / steps, z = tile / tiles_m;
    const int64_t row0 = (int64_t)(tile % tiles_m) * (8 * U) + (threadIdx.x >> 5);
    const int64_t col = (int64_t)step * 256 + (threadIdx.x & 31) * 8;
    x = (const uint8_t *)x + z * rows * ldx * (BF16 ? 2 : 4);
    q += z * rows * (cols / 2);
    s += ((int64_t)z * steps + step) * rows * 8;
    const bool in = col < cols; // whole quads
    Eight<BF16> v[U];
#pragma unroll
    for (int u = 0; u < U; u++) {
        const int64_t row = row0 + u * 8;
        if (in && row < rows)
            v[u].load(x, row * ldx + col);
        else
            v[u].zero();
    }
#pragma unroll
    for (int u = 0; u < U; u++) {
        const int64_t row = row0 + u * 8;
        const uint32_t b = in ? mxfp4_scale_byte<RULE>(group_max_u32<4>(v[u].amax())) : 0u;
        const uint32_t word = four_bytes(b);
        if (row < rows) {
            if (in)
                *reinterpret_cast<uint32_t *>(q + (row * cols + col) / 2) = v[u].encode(b);
            if ((threadIdx.x & 15) == 0)
                *reinterpret_cast<uint32_t *>(s + row * 8 + ((threadIdx.x >> 2) & 4)) = word;
        }
    }
}

// Both directions of a bf16 matrix from one read: a workgroup takes 256 rows x 128
// columns, quantises the rows as it reads them, keeps the bf16 in LDS (64 KB) and
// quantises the columns from there, a lane two columns of 32 rows.  Both copies
// leave in 64- and 128-byte pieces (the halves of a line of q come from neighbouring
// workgroups of one XCD).  Chunk c (16 bytes) of row r lies at chunk c ^ 2 (r / 32 % 8):
// the eight row groups that neighbouring lanes read are then eight words apart, and
// a wave's reads meet every bank once.  8192x28672: 143 us, 5.0 TB/s.
//
// Workgroups, two per CU, take tiles in turn; the next tile's rows are read while
// this one's columns are quantised (one tile a workgroup: 146 us, 8192x7168 41 against 40).
constexpr int TM = 256, TN = 128;
template <int RULE>
__global__ __launch_bounds__(512) void mxfp4_quant_t_bf16_kernel(const void *x, int64_t rows, int64_t cols, int64_t ldx,
                                                                 uint8_t *q, uint8_t *s, uint8_t *qt, uint8_t *st,
                                                                 int tiles_n, int tiles_m, int tiles)
{
    __shared__ __attribute__((aligned(16))) uint8_t tile[TM * TN * 2];
    const int64_t rows_p = (rows + 31) / 32 * 32, s_step = rows * 8, st_step = cols * 8;
    // XCD b % 8 takes a contiguous range of tiles, columns fastest, its workgroups in turn
    const int xcd = blockIdx.x & 7, mine = (int)(gridDim.x - xcd + 7) / 8;
    const int per = tiles >> 3, more = tiles & 7, begin = xcd * per + min(xcd, more), end = begin + per + (xcd < more);
    int id = begin + (int)(blockIdx.x >> 3);
    if (id >= end)
        return;
    // rows: 16 lanes x 8 elements a row, 32 rows a pass
    const int lr = threadIdx.x >> 4, lc = threadIdx.x & 15;
    Eight<true> v[TM / 32];
    auto load = [&](int t) {
        const int tn = t % tiles_n, tm = t / tiles_n % tiles_m, z = t / tiles_n / tiles_m;
        const int64_t col = (int64_t)tn * TN + lc * 8, row = (int64_t)tm * TM + lr;
        const uint16_t *from = (const uint16_t *)x + ((int64_t)z * rows + row) * ldx + col;
#pragma unroll
        for (int p = 0; p < TM / 32; p++) {
            if (col < cols && row + p * 32 < rows) // whole quads
                v[p].load(from, (int64_t)p * 32 * ldx);
            else
                v[p].zero();
        }
    };
    load(id);
    for (; id < end; id += mine) {
        const int tn = id % tiles_n, tm = id / tiles_n % tiles_m, z = id / tiles_n / tiles_m;
        const int64_t r0 = (int64_t)tm * TM, c0 = (int64_t)tn * TN;
        uint8_t *const q_z = q + (int64_t)z * rows * (cols / 2);
        uint8_t *const s_z = s + ((int64_t)z * ((cols + 255) / 256) + (c0 >> 8)) * s_step + ((c0 >> 5) & 4);
        uint8_t *const qt_z = qt + (int64_t)z * cols * (rows_p / 2);
        uint8_t *const st_z = st + ((int64_t)z * ((rows + 255) / 256) + tm) * st_step;
        {
            const int64_t col = c0 + lc * 8;
            const bool in = col < cols;
            // the step's other four bytes, where no other tile has them
            const bool alone = !((c0 >> 7) & 1) && c0 + TN >= cols;
#pragma unroll
            for (int p = 0; p < TM / 32; p++) {
                const int r = p * 32 + lr;
                const int64_t row = r0 + r;
                const uint32_t b = in ? mxfp4_scale_byte<RULE>(group_max_u32<4>(v[p].amax())) : 0u;
                const uint32_t word = four_bytes(b);
                if (row < rows) {
                    if (in)
                        *reinterpret_cast<uint32_t *>(q_z + (row * cols + col) / 2) = v[p].encode(b);
                    if (lc == 0) {
                        *reinterpret_cast<uint32_t *>(s_z + row * 8) = word;
                        if (alone)
                            *reinterpret_cast<uint32_t *>(s_z + row * 8 + 4) = 0;
                    }
                }
                *reinterpret_cast<uint4 *>(tile + r * (TN * 2) + ((lc ^ (2 * p)) * 16)) =
                    make_uint4(v[p].w[0], v[p].w[1], v[p].w[2], v[p].w[3]);
            }
        }
        __syncthreads();
        if (id + mine < end)
            load(id + mine);
        // columns: lane = row group g + 8 * column pair
        const int g = threadIdx.x & 7, cp = threadIdx.x >> 3;
        const int64_t c = c0 + 2 * cp;
        uint32_t w[32], m = 0;
#pragma unroll
        for (int k = 0; k < 32; k++) {
            w[k] = *reinterpret_cast<const uint32_t *>(tile + (g * 32 + k) * (TN * 2) + ((cp * 4) ^ (g * 32)));
            m = max2_abs(m, w[k]);
        }
        if (c < cols) { // (pairs are whole: cols is even)
            const bool in = r0 + g * 32 < rows;
#pragma unroll
            for (int h = 0; h < 2; h++) {
                const uint32_t b = in ? mxfp4_scale_byte<RULE>(h ? m & 0xFFFF0000u : m << 16) : 0u;
                uint32_t o[4];
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    uint32_t pr[4];
#pragma unroll
                    for (int j = 0; j < 4; j++) // rows 8k + 2j and the next, of column h of the pair
                        pr[j] = __builtin_amdgcn_perm(w[8 * k + 2 * j + 1], w[8 * k + 2 * j], h ? 0x07060302u : 0x05040100u);
                    o[k] = encode8_bf16(pr, b);
                }
                uint32_t word = b << (8 * (g & 3));
                word |= dpp<FGB_DPP_QUAD_XOR1>(word);
                word |= dpp<FGB_DPP_QUAD_XOR2>(word);
                if (in)
                    *reinterpret_cast<uint4 *>(qt_z + (c + h) * (rows_p / 2) + (r0 / 2 + g * 16)) =
                        make_uint4(o[0], o[1], o[2], o[3]);
                if ((g & 3) == 0)
                    *reinterpret_cast<uint32_t *>(st_z + (c + h) * 8 + g) = word;
            }
        }
        __syncthreads(); // the columns are read: the tile may be overwritten
    }
}

// The same for fp32 (8192x7168: 63 us, 4.7 TB/s): a workgroup takes 128 rows x 128 columns,
// quantises the rows as it reads them, keeps the values in LDS and quantises the
// columns from there.  Row r of the tile starts at word r * 128 + (r / 32) * 16,
// so the four 32-row groups of a column, read by neighbouring lanes, sit 16 banks
// apart.
constexpr int QT = 128;
template <int RULE>
__global__ __launch_bounds__(512) void mxfp4_quant_t_f32_kernel(const void *x, int64_t rows, int64_t cols, int64_t ldx,
                                                            uint8_t *q, uint8_t *s, uint8_t *qt, uint8_t *st)
{
    __shared__ float tile[QT * QT + 64];
    const int64_t r0 = (int64_t)blockIdx.y * QT, c0 = (int64_t)blockIdx.x * QT;
    const int64_t rows_p = (rows + 31) / 32 * 32, z = blockIdx.z; // matrix z of the stack
    x = (const float *)x + z * rows * ldx;
    q += z * rows * (cols / 2);
    s += z * ((cols + 255) / 256) * rows * 8;
    qt += z * cols * (rows_p / 2);
    st += z * ((rows + 255) / 256) * cols * 8;
    // rows: 16 lanes x 8 elements cover the tile's 128 columns, 32 rows a pass, all four in flight
    const int lr = threadIdx.x >> 4, lc = threadIdx.x & 15;
    const int64_t col = c0 + lc * 8;
    const bool cin = col < cols; // whole quads (32 columns)
    Eight<false> v4[4];
#pragma unroll
    for (int p = 0; p < 4; p++) {
        const int64_t row = r0 + p * 32 + lr;
        if (cin && row < rows)
            v4[p].load(x, row * ldx + col);
        else
            v4[p].zero();
    }
#pragma unroll
    for (int p = 0; p < 4; p++) {
        const int r = p * 32 + lr;
        const int64_t row = r0 + r;
        const uint32_t b = cin ? mxfp4_scale_byte<RULE>(group_max_u32<4>(v4[p].amax())) : 0u;
        const uint32_t word = four_bytes(b);
        if (row < rows) {
            if (cin)
                *reinterpret_cast<uint32_t *>(q + (row * cols + col) / 2) = v4[p].encode(b);
            if (lc == 0)
                *reinterpret_cast<uint32_t *>(s + scale_at(row, c0 / 32, rows)) = word;
        }
        float4 *to = reinterpret_cast<float4 *>(tile + r * QT + p * 16 + lc * 8);
        to[0] = make_float4(__uint_as_float(v4[p].w[0]), __uint_as_float(v4[p].w[1]), __uint_as_float(v4[p].w[2]),
                            __uint_as_float(v4[p].w[3]));
        to[1] = make_float4(__uint_as_float(v4[p].w[4]), __uint_as_float(v4[p].w[5]), __uint_as_float(v4[p].w[6]),
                            __uint_as_float(v4[p].w[7]));
    }
    __syncthreads();
    // columns: lane = 4 * column + row group
    const int64_t gt = (rows + 255) / 256 * 8; // row groups with the last step's unused bytes
    {
        const int c = threadIdx.x >> 2, g = threadIdx.x & 3;
        const int64_t ct = c0 + c, gr = r0 / 32 + g;
        float v[32];
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 32; i++) {
            v[i] = tile[(g * 32 + i) * QT + g * 16 + c];
            m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
        }
        const uint32_t b = mxfp4_scale_byte<RULE>(m);
        if (ct < cols && gr * 32 < rows) {
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
        } else if (ct < cols && gr < gt) {
            st[scale_at(ct, gr, cols)] = 0;
        }
    }
    // A last tile of up to 128 rows leaves the step's other half, if it starts one.
    if (threadIdx.x < 256 && blockIdx.y == gridDim.y - 1 && (gridDim.y & 1)) {
        const int c = threadIdx.x >> 1, h = threadIdx.x & 1;
        if (c0 + c < cols)
            *reinterpret_cast<uint16_t *>(st + scale_at(c0 + c, r0 / 32 + 4 + 2 * h, cols)) = 0;
    }
    if (threadIdx.x < 256 && blockIdx.x == gridDim.x - 1 && (gridDim.x & 1)) {
        const int r = threadIdx.x >> 1, h = threadIdx.x & 1;
        if (r0 + r < rows)
            *reinterpret_cast<uint16_t *>(s + scale_at(r0 + r, c0 / 32 + 4 + 2 * h, rows)) = 0;
    }
}

// Eight codes per lane.
template <bool BF16>
__global__ __launch_bounds__(256) void mxfp4_dequant_kernel(const uint8_t *q, const uint8_t *s, int64_t rows,
                                                            int64_t cols, void *out, int64_t first)
{
    const int64_t at = ((first + blockIdx.x) * 256 + threadIdx.x) * 8;
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
    const int64_t steps = (cols + 255) / 256, tiles_m = (rows + 31) / 32, tiles = tiles_m * G;
    const int64_t most = steps < LAUNCH_BLOCKS ? LAUNCH_BLOCKS / steps : 1; // tiles of a launch
    for (int64_t first = 0; first < tiles; first += most) {
        const int64_t grid = steps * (tiles - first < most ? tiles - first : most);
        FGB_BY_TYPE_AND_RULE(mxfp4_quant_kernel, <<<(unsigned)grid, 256, 0, (hipStream_t)stream>>>(
                                                     x, rows, cols, ldx, q, s, (int)steps, (int)tiles_m, (int)first));
        FGB_LAUNCHED("mxfp4_quant_kernel");
    }
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
    hipStream_t hs = (hipStream_t)stream;
    if (x_dtype == FGB_BF16) {
        const int64_t tiles_n = (cols + TN - 1) / TN, tiles_m = (rows + TM - 1) / TM;
        const int64_t tiles = tiles_n * tiles_m * G, grid = tiles < 512 ? tiles : 512;
        if (rule == FGB_SCALE_CEIL)
            mxfp4_quant_t_bf16_kernel<RULE_CEIL><<<(unsigned)grid, 512, 0, hs>>>(x, rows, cols, ldx, q, s, qt, st,
                                                                                (int)tiles_n, (int)tiles_m, (int)tiles);
        else
            mxfp4_quant_t_bf16_kernel<RULE_OCP_FLOOR><<<(unsigned)grid, 512, 0, hs>>>(x, rows, cols, ldx, q, s, qt, st,
                                                                                     (int)tiles_n, (int)tiles_m, (int)tiles);
    } else {
        FGB_REQUIRE(cols <= (1ll << 30) - 256, FGB_EINVAL, "mxfp4_quant_t: cols of an FP32 x must be below 2^30 - 255");
        const dim3 grid((unsigned)((cols + QT - 1) / QT), (unsigned)gy, (unsigned)G);
        if (rule == FGB_SCALE_CEIL)
            mxfp4_quant_t_f32_kernel<RULE_CEIL><<<grid, 512, 0, hs>>>(x, rows, cols, ldx, q, s, qt, st);
        else
            mxfp4_quant_t_f32_kernel<RULE_OCP_FLOOR><<<grid, 512, 0, hs>>>(x, rows, cols, ldx, q, s, qt, st);
    }
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
    FGB_REQUIRE(aligned16(q) && aligned16(out), FGB_EINVAL, "mxfp4_dequant: q and out must be 16-byte aligned");
    FGB_REQUIRE(rows < (1ll << 31) && cols < (1ll << 31) && rows * (cols / 32) < (1ll << 33), FGB_EINVAL,
                "mxfp4_dequant: too many elements");
    const int64_t blocks = (rows * cols / 8 + 255) / 256;
    for (int64_t first = 0; first < blocks; first += LAUNCH_BLOCKS) {
        const unsigned grid = (unsigned)(blocks - first < LAUNCH_BLOCKS ? blocks - first : LAUNCH_BLOCKS);
        if (out_dtype == FGB_BF16)
            mxfp4_dequant_kernel<true><<<grid, 256, 0, (hipStream_t)stream>>>(q, s, rows, cols, out, first);
        else
            mxfp4_dequant_kernel<false><<<grid, 256, 0, (hipStream_t)stream>>>(q, s, rows, cols, out, first);
        FGB_LAUNCHED("mxfp4_dequant_kernel");
    }
    return FGB_OK;
}
