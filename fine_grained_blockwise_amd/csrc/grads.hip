// grads.hip -- the global norm of many gradients, and their clipping.
//
//   S = sum over all tensors of g^2, norm = scale sqrt(S),
//   out = g scale min(1, max_norm / norm); a norm that is infinite or NaN in FP32, as it is
//   returned, clips nothing.
//
// Squares and sums are FP64: the square of a BF16 or FP32 value is exact and neither over- nor
// underflows.  Every sum has a fixed order: a thread's values, the workgroup's threads, the
// workgroups.
//
// Bound by memory: the gradients are read twice, the clipped ones written once.  The
// tensors' addresses travel in the kernel's arguments (4 KB hold LIST of them), so that a
// captured launch has them and nothing is copied; a longer list takes several launches.
// FP32 gradients of 1.41 G elements into BF16: squares 0.91 ms (6.2 TB/s), scaling 1.49 ms
// (5.7 TB/s).
#include <algorithm>
#include <new>

#include "fgb_internal.h"

namespace fgb {

constexpr int LIST = 166;   // tensors of one launch
constexpr int CHUNK = 8192; // elements of one tensor that a workgroup takes at a time

// Workgroups of the squares' launches: eight a CU take the chunks in turn, so that few partial
// sums are left.  The scaling's take a chunk each: the ones that run together then write one
// stretch of memory (1.41 G elements: 1.49 ms, 2048 workgroups in turn 1.65 ms).
constexpr uint32_t SUM_BLOCKS = 2048;

struct GradList {
    const void *p[LIST];
    void *o[LIST];
    uint32_t upto[LIST]; // chunks of this and the tensors before
    uint32_t info[LIST]; // elements of the last chunk, 2^16 for a BF16 gradient, 2^17 for a BF16 output
    int count;
};
// (Entries are whole dwords: for narrower ones beside addresses the compiler formed scalar
// loads whose base and offset are aligned in their sum only, and the card drops the low two
// bits of each.)
static_assert(sizeof(GradList) <= 4096 - 64, "the arguments of a launch are at most 4 KB");

// The tensor that chunk c belongs to, its first element there and its elements.  A lane holds
// every 64th of the tensors' ends, so that finding the tensor costs a comparison a lane and not
// a chain of loads.
struct Piece {
    const void *p;
    void *o;
    int64_t from;
    int n, kind; // kind: 1 for a BF16 gradient, 2 for a BF16 output
};
struct Ends {
    static constexpr int N = (LIST + 63) / 64;
    uint32_t upto[N];
    __device__ __forceinline__ explicit Ends(const GradList &l)
    {
#pragma unroll
        for (int k = 0; k < N; k++) {
            const int i = 64 * k + lane_id();
            const uint32_t v = l.upto[min(i, LIST - 1)];
            upto[k] = i < l.count ? v : 0xFFFFFFFFu;
        }
    }
    __device__ __forceinline__ Piece piece(const GradList &l, uint32_t c) const // c: the same in all lanes
    {
        int t = 0;
#pragma unroll
        for (int k = 0; k < N; k++)
            t += __builtin_popcountll(__ballot(upto[k] <= c));
        const uint32_t info = l.info[t];
        return {l.p[t], l.o[t], (int64_t)(c - (t ? l.upto[t - 1] : 0u)) * CHUNK,
                c + 1 == l.upto[t] ? (int)(info & 0xFFFF) : CHUNK, (int)(info >> 16)};
    }
};

// Eight neighbouring gradients (the addresses are aligned to one element only: the card's
// loads and stores need no more).
template <bool BF16> __device__ __forceinline__ void load8g(const void *p, int64_t at, float (&f)[8])
{
    if constexpr (BF16) {
        uint32_t u[4];
        __builtin_memcpy(u, (const uint16_t *)p + at, 16);
#pragma unroll
        for (int i = 0; i < 4; i++) {
            f[2 * i] = bf16lo(u[i]);
            f[2 * i + 1] = bf16hi(u[i]);
        }
    } else {
        __builtin_memcpy(f, (const float *)p + at, 32);
    }
}
template <bool BF16> __device__ __forceinline__ float load1g(const void *p, int64_t at)
{
    return BF16 ? __uint_as_float((uint32_t)((const uint16_t *)p)[at] << 16) : ((const float *)p)[at];
}
// (BF16 outputs are written past the caches: clipping 72 M elements took 136 and 145 us, before
// other steps)
template <bool BF16> __device__ __forceinline__ void store8g(void *p, int64_t at, const float (&f)[8])
{
    if constexpr (BF16) {
        typedef uint32_t words __attribute__((ext_vector_type(4), aligned(2)));
        const words u = {pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7])};
        __builtin_nontemporal_store(u, reinterpret_cast<words *>((uint16_t *)p + at));
    } else {
        __builtin_memcpy((float *)p + at, f, 32);
    }
}
template <bool BF16> __device__ __forceinline__ void store1g(void *p, int64_t at, float f)
{
    if constexpr (BF16)
        ((__bf16 *)p)[at] = (__bf16)f;
    else
        ((float *)p)[at] = f;
}

// The eights of a piece and the elements left over: eight(at, values) and one(at, value).  A
// thread's loads go out together, those past the end for the last eight once more (squares of
// 122 tensors of 7168: 6.2 us with a loop over what a piece holds, 5.2 so).
template <bool BF16, class Eight, class One>
__device__ __forceinline__ void over_piece(const void *p, int64_t from, int n, Eight eight, One one)
{
    constexpr int STEP = 8 * 256, U = CHUNK / STEP;
    const int whole = n & ~7, rest = whole + (int)threadIdx.x;
    float f[U][8], last = 0.0f;
    if (whole) {
#pragma unroll
        for (int u = 0; u < U; u++)
            load8g<BF16>(p, from + min(8 * (int)threadIdx.x + u * STEP, whole - 8), f[u]);
    }
    if (rest < n)
        last = load1g<BF16>(p, from + rest);
#pragma unroll
    for (int u = 0; u < U; u++) {
        const int at = 8 * (int)threadIdx.x + u * STEP;
        if (at < whole)
            eight(from + at, f[u]);
    }
    if (rest < n)
        one(from + rest, last);
}

// The workgroup's sum of v, in every thread.
template <int THREADS> __device__ __forceinline__ double block_sum(double v)
{
    __shared__ double red[THREADS / 64];
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1)
        v += __shfl_xor(v, d);
    if (lane_id() == 0)
        red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int i = 1; i < THREADS / 64; i++)
        v += red[i];
    return v;
}

template <bool BF16> __device__ __forceinline__ double piece_squares(const void *p, int64_t from, int n)
{
    double sum = 0.0;
    over_piece<BF16>(
        p, from, n,
        [&](int64_t, const float (&f)[8]) {
#pragma unroll
            for (int j = 0; j < 8; j++)
                sum = fma((double)f[j], (double)f[j], sum);
        },
        [&](int64_t, float f) { sum = fma((double)f, (double)f, sum); });
    return sum;
}

__global__ __launch_bounds__(256) void grad_squares_kernel(GradList l, double *part)
{
    double sum = 0.0;
    const uint32_t chunks = l.upto[l.count - 1];
    const Ends ends(l);
    for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
        const Piece k = ends.piece(l, c);
        sum += k.kind & 1 ? piece_squares<true>(k.p, k.from, k.n) : piece_squares<false>(k.p, k.from, k.n);
    }
    sum = block_sum<256>(sum);
    if (threadIdx.x == 0)
        part[blockIdx.x] = sum;
}

__global__ __launch_bounds__(1024) void grad_total_kernel(const double *part, int n, double *out, int accumulate)
{
    double sum = 0.0;
    for (int i = threadIdx.x; i < n; i += 2 * 1024) { // two loads together
        const double a = part[i], b = i + 1024 < n ? part[i + 1024] : 0.0;
        sum += a;
        sum += b;
    }
    sum = block_sum<1024>(sum);
    if (threadIdx.x == 0)
        *out = accumulate ? *out + sum : sum;
}

template <bool IN, bool OUT, class Times> __device__ __forceinline__ void piece_scale(const Piece &k, Times times)
{
    over_piece<IN>(
        k.p, k.from, k.n,
        [&](int64_t at, float (&v)[8]) {
#pragma unroll
            for (int j = 0; j < 8; j++)
                v[j] = times(v[j]);
            store8g<OUT>(k.o, at, v);
        },
        [&](int64_t at, float v) { store1g<OUT>(k.o, at, times(v)); });
}
template <class Times> __device__ __forceinline__ void scale_kind(const Piece &k, Times times)
{
    if (k.kind == 3)
        piece_scale<true, true>(k, times);
    else if (k.kind == 2)
        piece_scale<false, true>(k, times);
    else if (k.kind == 1)
        piece_scale<true, false>(k, times);
    else
        piece_scale<false, false>(k, times);
}

// squares: the sum (parts = 0), or up to FEW_PARTS parts of it, which every workgroup adds
// itself, in grad_total_kernel's order (122 tensors of 7168: 20 us a call, 16.5 without that
// launch).  A list's last chunks come first: the sums' pass left them in the cache.  (The lists of a
// longer one come in the order in which they were summed.)
constexpr int FEW_PARTS = 256;
__global__ __launch_bounds__(256) void grad_scale_kernel(GradList l, const double *squares, int parts, double max_norm,
                                                         double scale, float *norm_out)
{
    double sum = *squares;
    if (parts > 0) // uniform
        sum = block_sum<256>((int)threadIdx.x < parts ? squares[threadIdx.x] : 0.0);
    const double norm = scale * sqrt(sum);
    const bool clip = norm > max_norm && (float)norm < __builtin_inff();
    const double factor = clip ? scale * (max_norm / norm) : scale;
    const float f = (float)factor;
    const bool beyond = factor < 0x1p-126 || factor > 0x1.fffffep127; // FP32 holds fewer than 24 bits of it
    if (norm_out && blockIdx.x == 0 && threadIdx.x == 0)
        *norm_out = (float)norm;
    if (l.count == 0)
        return;
    const uint32_t chunks = l.upto[l.count - 1];
    const Ends ends(l);
    for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
        const Piece k = ends.piece(l, chunks - 1 - c);
        if (f == 1.0f && k.p == k.o)
            continue; // in place and unchanged
        if (beyond) // uniform
            scale_kind(k, [&](float v) { return (float)(v * factor); });
        else
            scale_kind(k, [&](float v) { return v * f; });
    }
}

static unsigned grad_grid(const GradList &l, uint32_t most)
{
    const uint32_t chunks = l.count ? l.upto[l.count - 1] : 1;
    return chunks < most ? chunks : most;
}

static int64_t chunks_of(int64_t n) { return (n + CHUNK - 1) / CHUNK; }

// The tensors from `at` on that one launch takes; empty ones are passed over.
static int next_list(GradList &l, int at, int n, const void *const *grads, void *const *outs, const int64_t *numel,
                     const int *dtypes, const int *out_dtypes)
{
    l.count = 0;
    uint32_t upto = 0;
    for (; at < n && l.count < LIST; at++) {
        if (numel[at] == 0)
            continue;
        const int k = l.count++;
        l.p[k] = grads[at];
        l.o[k] = outs ? outs[at] : nullptr;
        l.info[k] = (uint32_t)((numel[at] - 1) % CHUNK + 1) | (dtypes[at] == FGB_BF16 ? 1u << 16 : 0u) |
                    (outs && out_dtypes[at] == FGB_BF16 ? 2u << 16 : 0u);
        l.upto[k] = upto += (uint32_t)chunks_of(numel[at]);
    }
    return at;
}

static int check_grads(const char *name, int n, const void *const *grads, const int64_t *numel, const int *dtypes)
{
    FGB_REQUIRE(n >= 0 && (n == 0 || (grads && numel && dtypes)), FGB_EINVAL, "%s: null list", name);
    int64_t chunks = 0;
    for (int i = 0; i < n; i++) {
        FGB_REQUIRE(dtypes[i] == FGB_F32 || dtypes[i] == FGB_BF16, FGB_EUNSUPPORTED,
                    "%s: gradient %d must be FGB_F32 or FGB_BF16", name, i);
        FGB_REQUIRE(numel[i] >= 0 && numel[i] < (1ll << 40), FGB_EINVAL, "%s: gradient %d has a bad length", name, i);
        FGB_REQUIRE(numel[i] == 0 || (grads[i] && ((uintptr_t)grads[i] & (dtypes[i] == FGB_BF16 ? 1 : 3)) == 0),
                    FGB_EINVAL, "%s: gradient %d is null or misaligned", name, i);
        chunks += chunks_of(numel[i]);
    }
    FGB_REQUIRE(chunks < (1ll << 31), FGB_EINVAL, "%s: too many elements", name);
    return FGB_OK;
}

// No output may lie over another one, or over a gradient that is not its own.
static int check_outputs(int n, const void *const *grads, void *const *outs, const int64_t *numel, const int *dtypes,
                         const int *out_dtypes)
{
    struct Span {
        uintptr_t from, to;
        int of, out;
    };
    Span *const spans = new (std::nothrow) Span[2 * (size_t)n];
    FGB_REQUIRE(spans, FGB_ENOMEM, "grad_clip: no host memory to compare the places of %d tensors", n);
    int m = 0;
    for (int i = 0; i < n; i++) {
        if (numel[i] == 0)
            continue;
        const uintptr_t p = (uintptr_t)grads[i], o = (uintptr_t)outs[i];
        if (!(p == o && dtypes[i] == out_dtypes[i])) // in place: one span for both
            spans[m++] = {p, p + (size_t)numel[i] * (dtypes[i] == FGB_BF16 ? 2 : 4), i, 0};
        spans[m++] = {o, o + (size_t)numel[i] * (out_dtypes[i] == FGB_BF16 ? 2 : 4), i, 1};
    }
    std::sort(spans, spans + m, [](const Span &a, const Span &b) { return a.from < b.from; });
    bool bad = false;
    uintptr_t out_end = 0, any_end = 0; // ends of the outputs and of all spans so far
    for (int i = 0; i < m && !bad; i++) {
        bad = spans[i].from < (spans[i].out ? any_end : out_end);
        any_end = std::max(any_end, spans[i].to);
        if (spans[i].out)
            out_end = std::max(out_end, spans[i].to);
    }
    delete[] spans;
    FGB_REQUIRE(!bad, FGB_EINVAL, "grad_clip: an output lies over another one or over a gradient that is not its own");
    return FGB_OK;
}

// Partial sums of all launches of a list: its non-empty tensors in runs of LIST.
static int64_t partials(int n, const int64_t *numel)
{
    int64_t total = 0, chunks = 0;
    int count = 0;
    for (int i = 0; i < n; i++) {
        if (numel[i] <= 0)
            continue;
        chunks += chunks_of(numel[i]);
        if (++count == LIST) {
            total += chunks < SUM_BLOCKS ? chunks : SUM_BLOCKS;
            chunks = count = 0;
        }
    }
    return total + (chunks < SUM_BLOCKS ? chunks : SUM_BLOCKS);
}

// The parts of the sum of squares; *parts: how many.
static int sum_squares(int n, const void *const *grads, const int64_t *numel, const int *dtypes, double *part,
                       int *parts, hipStream_t st)
{
    GradList l;
    int64_t done = 0;
    for (int at = 0; at < n;) {
        at = next_list(l, at, n, grads, nullptr, numel, dtypes, nullptr);
        if (l.count == 0)
            break;
        const unsigned grid = grad_grid(l, SUM_BLOCKS);
        grad_squares_kernel<<<grid, 256, 0, st>>>(l, part + done);
        FGB_LAUNCHED("grad_squares_kernel");
        done += grid;
    }
    *parts = (int)done;
    return FGB_OK;
}

static int total_of(const double *part, int parts, double *out, int accumulate, hipStream_t st)
{
    grad_total_kernel<<<1, 1024, 0, st>>>(part, parts, out, accumulate);
    FGB_LAUNCHED("grad_total_kernel");
    return FGB_OK;
}

} // namespace fgb

using namespace fgb;

extern "C" size_t grad_sumsq_workspace_size(const int64_t *numel, int n)
{
    return n < 0 || (n > 0 && !numel) ? 0 : 8 * (size_t)(partials(n, numel) + 1);
}

extern "C" int grad_sumsq(const void *const *grads, const int64_t *numel, const int *dtypes, int n, double *sumsq,
                          int accumulate, void *workspace, size_t ws_bytes, void *stream)
{
    clear_error();
    const int rc = check_grads("grad_sumsq", n, grads, numel, dtypes);
    if (rc != FGB_OK)
        return rc;
    FGB_REQUIRE(sumsq && ((uintptr_t)sumsq & 7) == 0, FGB_EINVAL, "grad_sumsq: sumsq null or misaligned");
    const size_t need = grad_sumsq_workspace_size(numel, n);
    FGB_REQUIRE(workspace && ws_bytes >= need, FGB_EWORKSPACE, "grad_sumsq: workspace of %zu bytes needed", need);
    FGB_REQUIRE(((uintptr_t)workspace & 7) == 0, FGB_EINVAL, "grad_sumsq: workspace must be 8-byte aligned");
    int parts;
    const int failed = sum_squares(n, grads, numel, dtypes, (double *)workspace, &parts, (hipStream_t)stream);
    return failed != FGB_OK ? failed : total_of((double *)workspace, parts, sumsq, accumulate, (hipStream_t)stream);
}

extern "C" int grad_clip(const void *const *grads, void *const *outs, const int64_t *numel, const int *dtypes,
                         const int *out_dtypes, int n, double max_norm, double scale, const double *sumsq, float *norm,
                         void *workspace, size_t ws_bytes, void *stream)
{
    clear_error();
    int rc = check_grads("grad_clip", n, grads, numel, dtypes);
    if (rc != FGB_OK)
        return rc;
    FGB_REQUIRE(n == 0 || (outs && out_dtypes), FGB_EINVAL, "grad_clip: null list");
    for (int i = 0; i < n; i++) {
        FGB_REQUIRE(out_dtypes[i] == FGB_F32 || out_dtypes[i] == FGB_BF16, FGB_EUNSUPPORTED,
                    "grad_clip: output %d must be FGB_F32 or FGB_BF16", i);
        FGB_REQUIRE(numel[i] == 0 || (outs[i] && ((uintptr_t)outs[i] & (out_dtypes[i] == FGB_BF16 ? 1 : 3)) == 0),
                    FGB_EINVAL, "grad_clip: output %d is null or misaligned", i);
    }
    FGB_REQUIRE(max_norm > 0.0 && scale > 0.0 && scale < __builtin_inf(), FGB_EINVAL,
                "grad_clip: max_norm and scale must be positive");
    if ((rc = check_outputs(n, grads, outs, numel, dtypes, out_dtypes)) != FGB_OK)
        return rc;
    FGB_REQUIRE(((uintptr_t)sumsq & 7) == 0 && norm && ((uintptr_t)norm & 3) == 0, FGB_EINVAL,
                "grad_clip: sumsq misaligned, or norm null or misaligned");
    const hipStream_t st = (hipStream_t)stream;
    int parts = 0;
    if (!sumsq) {
        const size_t need = grad_sumsq_workspace_size(numel, n);
        FGB_REQUIRE(workspace && ws_bytes >= need, FGB_EWORKSPACE, "grad_clip: workspace of %zu bytes needed", need);
        FGB_REQUIRE(((uintptr_t)workspace & 7) == 0, FGB_EINVAL, "grad_clip: workspace must be 8-byte aligned");
        double *const part = (double *)workspace + 1;
        if ((rc = sum_squares(n, grads, numel, dtypes, part, &parts, st)) != FGB_OK)
            return rc;
        sumsq = part;
        if (parts == 0 || parts > FEW_PARTS) {
            sumsq = (double *)workspace;
            if ((rc = total_of(part, parts, (double *)workspace, 0, st)) != FGB_OK)
                return rc;
            parts = 0;
        }
    }
    GradList l;
    int at = 0;
    do { // (an empty list still gives the norm)
        at = next_list(l, at, n, grads, outs, numel, dtypes, out_dtypes);
        if (l.count == 0 && norm == nullptr)
            break;
        grad_scale_kernel<<<grad_grid(l, (uint32_t)LAUNCH_BLOCKS), 256, 0, st>>>(l, sumsq, parts, max_norm, scale, norm);
        FGB_LAUNCHED("grad_scale_kernel");
        norm = nullptr;
    } while (at < n);
    return FGB_OK;
}
