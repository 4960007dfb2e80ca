// router_grouped.hip -- the router whose choice a bias and groups of experts decide, and the
// bias's update (scores, weights, counts, loss and gradient: router_device.h).
//
// With a bias experts are chosen by c = s + b, the score rounded to FP32 once and the sum once
// more (so that any correct implementation compares the same numbers; scores are therefore
// formed in FP64), without one by c = z.  A group's value is the sum of its two largest c with
// a bias, its largest c without; experts outside the topk_groups groups of largest value (equal
// values: the lowest id) cannot be chosen.
//
// L lanes take a token and hold its experts as in router_device.h.  Bound by instruction issue:
// 16384 x 256 logits are 17 MB, and choosing 8 in 4 of 8 groups with the loss takes 20 us (28
// under a trace), of which the FP64 scores 4, the groups 3, the rounds of the choice 4.
#include "router_device.h"

namespace fgb {

struct GroupedArgs : RouterArgs {
    const float *bias;           // [E] or NULL
    int groups, topk_groups, of; // groups of `of` experts
    int lanes;                   // of a group, see group_lanes
};

// The two largest keys of P neighbouring lanes (a power of two up to 16; uniform).
template <int CTRL> __device__ __forceinline__ void join_two(uint32_t &first, uint32_t &second)
{
    const uint32_t f = dpp<CTRL>(first), s = dpp<CTRL>(second);
    second = max(max(second, s), min(first, f));
    first = max(first, f);
}
__device__ __forceinline__ void lanes_two(int P, uint32_t &first, uint32_t &second)
{
    if (P >= 2)
        join_two<FGB_DPP_QUAD_XOR1>(first, second);
    if (P >= 4)
        join_two<FGB_DPP_QUAD_XOR2>(first, second);
    if (P >= 8)
        join_two<FGB_DPP_HALF_MIRROR>(first, second);
    if (P >= 16)
        join_two<FGB_DPP_ROW_ROR8>(first, second);
}

// e^x, x in [-200, 200], to a relative 2^-50: x log2 e = n + r, |r| <= 1/2, and 2^r by its
// Taylor polynomial (the first term left out is below 2^-52).  log2 e is two numbers: one alone
// is off by 2^-55.4, which x and ln 2 make 2^-48.2.
__device__ __forceinline__ double exp64(double x)
{
    constexpr double LOG2E = 1.4426950408889634, LOG2E_REST = 2.0355273740931033e-17;
    const double n = __builtin_rint(x * LOG2E), r = fma(x, LOG2E_REST, fma(x, LOG2E, -n));
    // ln(2)^k / k!
    double p = 2.5678435993488205e-11;
    p = fma(p, r, 4.4455382718708116e-10);
    p = fma(p, r, 7.0549116208011233e-09);
    p = fma(p, r, 1.0178086009239699e-07);
    p = fma(p, r, 1.3215486790144309e-06);
    p = fma(p, r, 1.5252733804059840e-05);
    p = fma(p, r, 1.5403530393381610e-04);
    p = fma(p, r, 1.3333558146428443e-03);
    p = fma(p, r, 9.6181291076284772e-03);
    p = fma(p, r, 5.5504108664821580e-02);
    p = fma(p, r, 2.4022650695910072e-01);
    p = fma(p, r, 6.9314718055994531e-01);
    p = fma(p, r, 1.0);
    return ldexp(p, (int)n);
}
// 1 / d for a normal d: the card's estimate and two Newton steps.
__device__ __forceinline__ double inverse64(double d)
{
    double r = __builtin_amdgcn_rcp(d);
    r = fma(r, fma(-d, r, 1.0), r);
    return fma(r, fma(-d, r, 1.0), r);
}

// Lanes that look for a group's two largest keys.  A group that is a power of two of quads,
// up to 16 lanes', finds them in the lanes' registers (positive); any other through LDS, by as
// many lanes of the token as there are (negative).
static int group_lanes(int E, int groups, int L)
{
    const int of = E / groups, P = of / 4;
    if (of % 4 == 0 && P <= 16 && P <= L && (P & (P - 1)) == 0)
        return P;
    int n = 1;
    while (2 * n * groups <= L && n < 16)
        n *= 2;
    return -n;
}
// LDS words of the groups' values and (the LDS way) of the keys of a workgroup's tokens; 3
// more for the alignment.
static size_t group_words(int E, int groups, int L, int lanes)
{
    return groups == 1 ? 0 : (size_t)256 / L * ((groups + 3) / 4 * 4 + (lanes < 0 ? E : 0)) + 3;
}

// The keys of c from those of the logits (0: unusable); most: the largest usable logit.
template <int SCORE, int L, int R>
__device__ __forceinline__ void biased_keys(const float (&z)[R], const float (&bias)[R], float most, uint32_t (&key)[R])
{
    if constexpr (SCORE == FGB_ROUTER_SOFTMAX) {
        double s[R], sum = 0.0;
#pragma unroll
        for (int j = 0; j < R; j++) { // (equal: an infinite one has the score 1, not NaN)
            s[j] = !key[j] ? 0.0 : z[j] == most ? 1.0 : exp64(fmax((double)z[j] - (double)most, -200.0));
            sum += s[j];
        }
#pragma unroll
        for (int d = 1; d < L; d <<= 1)
            sum += __shfl_xor(sum, d);
        const double inv = inverse64(sum);
#pragma unroll
        for (int j = 0; j < R; j++)
            key[j] = key[j] ? logit_key<false>((float)(s[j] * inv) + bias[j], 0) : 0u;
    } else {
#pragma unroll
        for (int j = 0; j < R; j++) { // (past 200 the score is 0 or 1 in FP32)
            const double t = exp64(-(double)fminf(fmaxf(z[j], -200.0f), 200.0f));
            key[j] = key[j] ? logit_key<false>((float)inverse64(1.0 + t) + bias[j], 0) : 0u;
        }
    }
}

// Takes the keys of experts outside the best groups.  values: [groups] words of LDS, a multiple
// of 16 bytes, the last ones 0; keys: [E]; of: the experts' groups, a byte each.
template <int L, int Q>
__device__ __forceinline__ void close_groups(const GroupedArgs &a, uint32_t (&key)[4 * Q], const uint32_t (&of)[Q], int l,
                                             int e0, uint32_t *values, uint32_t *keys)
{
    constexpr int R = 4 * Q;
    // (Keys > 0 are neither -inf nor NaN.  The sum of two of them can be -inf, whose key is 0: it
    // gets the key below the finite ones, as 0 is a group's that has nothing to choose.)
    const auto value = [&](uint32_t first, uint32_t second) {
        return a.bias && second ? max(logit_key<false>(key_logit<false>(first) + key_logit<false>(second), 0), 1u) : first;
    };
    if (a.lanes > 0) { // uniform
#pragma unroll
        for (int q = 0; q < Q; q++) {
            const uint32_t *k = key + 4 * q;
            uint32_t first = max(k[0], k[1]), second = min(k[0], k[1]);
            const uint32_t f = max(k[2], k[3]), s = min(k[2], k[3]);
            second = max(max(second, s), min(first, f));
            first = max(first, f);
            lanes_two(a.lanes, first, second);
            if ((l & (a.lanes - 1)) == 0 && e0 + 4 * L * q < a.E)
                values[of[q] & 255] = value(first, second);
        }
    } else {
#pragma unroll
        for (int j = 0; j < R; j++)
            if (e0 + at_quad<L>(j) < a.E)
                keys[e0 + at_quad<L>(j)] = key[j];
        wave_sync();
        const int n = -a.lanes;
        for (int g0 = 0; g0 < a.groups; g0 += L / n) { // (the token's lanes together)
            const int g = g0 + l / n;
            uint32_t first = 0, second = 0;
            if (g < a.groups) {
#pragma unroll 4
                for (int i = l % n; i < a.of; i += n) {
                    const uint32_t k = keys[g * a.of + i];
                    second = max(second, min(first, k));
                    first = max(first, k);
                }
            }
            lanes_two(n, first, second);
            if (g < a.groups && l % n == 0)
                values[g] = value(first, second);
        }
    }
    wave_sync();
    uint64_t open = 0; // a bit a group
    for (int g0 = 0; g0 < a.groups; g0 += L) {
        const int g = g0 + l;
        const uint32_t own = g < a.groups ? values[g] : 0u;
        int before = 0;
        for (int h = 0; h < a.groups; h += 4) {
            const uint4 v = *reinterpret_cast<const uint4 *>(values + h);
            before += (v.x > own || (v.x == own && h < g)) + (v.y > own || (v.y == own && h + 1 < g)) +
                      (v.z > own || (v.z == own && h + 2 < g)) + (v.w > own || (v.w == own && h + 3 < g));
        }
        const uint64_t b = __ballot(own && before < a.topk_groups) >> ((threadIdx.x & 63) & ~(L - 1));
        open |= (L == 64 ? b : b & ((1ull << (L & 63)) - 1)) << g0;
    }
    wave_sync();
#pragma unroll
    for (int j = 0; j < R; j++)
        key[j] = open >> (of[j / 4] >> (8 * (j % 4)) & 255) & 1 ? key[j] : 0u;
}

template <bool BF16, int SCORE, int L, int Q>
__global__ __launch_bounds__(256) void router_grouped_kernel(GroupedArgs a)
{
    extern __shared__ float red[]; // [groups][E] floats (the loss's sums), E + 1 ints, close_groups's
    constexpr int GROUPS = 256 / L, R = 4 * Q;
    const int group = threadIdx.x / L;
    int l = threadIdx.x % L, e0 = 4 * l;
    int *cnt = reinterpret_cast<int *>(red + (a.loss ? GROUPS * a.E : 0));
    uint32_t *values = reinterpret_cast<uint32_t *>(cnt + a.E + 1);
    const int padded = (a.groups + 3) / 4 * 4;
    values += -(reinterpret_cast<uintptr_t>(values) >> 2) & 3;
    uint32_t *keys = values + GROUPS * padded + group * a.E;
    values += group * padded;
    __shared__ int ids[256]; // [groups][L]
    for (int e = threadIdx.x; e <= a.E; e += 256)
        cnt[e] = 0;
    if (a.groups > 1)
        for (int g = l; g < padded; g += L)
            values[g] = 0;
    float psum[R], bias[R];
    uint32_t of[Q];
#pragma unroll
    for (int q = 0; q < Q; q++) {
        of[q] = 0;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int e = min(e0 + 4 * L * q + i, a.E - 1);
            psum[4 * q + i] = 0.0f;
            bias[4 * q + i] = a.bias ? a.bias[e] : 0.0f;
            of[q] |= (uint32_t)(e / a.of) << (8 * i);
        }
    }
    __syncthreads();
    int live_n = 0;
    for (int64_t t0 = (int64_t)blockIdx.x * GROUPS; t0 < a.T; t0 += (int64_t)gridDim.x * GROUPS) {
        const int64_t t = t0 + group;
        // Addresses, comparisons and shifts by these are formed anew for each token: kept over the
        // loop they take 40 registers and a wave a SIMD (16384 x 256: 33.6 us, 27.2 so).
        asm volatile("" : "+v"(l), "+v"(e0));
#pragma unroll
        for (int q = 0; q < Q; q++)
            asm volatile("" : "+v"(of[q]));
        const bool on = t < a.T && (!a.mask || a.mask[t] != 0);
        float z[R];
        uint32_t key[R], best = 0, usable = 0;
        load_logits<BF16, L, Q>(a, min(t, a.T - 1), e0, z);
#pragma unroll
        for (int j = 0; j < R; j++) {
            key[j] = on ? logit_key<false>(z[j], 0) : 0u;
            best = max(best, key[j]);
            usable |= key[j] && bias[j] > NEG_INF ? 1u : 0u; // (c > -inf as a score is in [0, 1])
        }
        const float most = key_logit<false>(group_max<L>(best));
        const bool live = group_max<L>(usable) != 0;
        // the scores' normalisation and the loss's sums
        Norm n{fminf(most, 0.0f), 1.0f};
        if (SCORE == FGB_ROUTER_SOFTMAX || a.loss) { // uniform
            float num[R], p[R];
            Sig sg[R];
            n = probabilities<SCORE, L, R>(z, most, num, p, sg);
            if (live) {
                live_n++;
#pragma unroll
                for (int j = 0; j < R; j++)
                    psum[j] += p[j];
            }
        } else {
            uint32_t nan = 0;
#pragma unroll
            for (int j = 0; j < R; j++)
                nan |= z[j] == z[j] ? 0u : 1u;
            n.inv = group_max<L>(nan) ? __builtin_nanf("") : 1.0f;
            live_n += live;
        }
        if (a.bias) // uniform
            biased_keys<SCORE, L, R>(z, bias, most, key);
        if (a.groups > 1) // uniform
            close_groups<L, Q>(a, key, of, l, e0, values, keys);
        // topk rounds; lane r keeps the r-th choice.  A quad's largest key is kept beside it, so a
        // round looks through one quad of the lane.
        uint32_t quad[Q], mine = 0;
#pragma unroll
        for (int q = 0; q < Q; q++)
            quad[q] = max(max(key[4 * q], key[4 * q + 1]), max(key[4 * q + 2], key[4 * q + 3]));
        for (int r = 0; r < a.k; r++) {
            best = quad[0];
#pragma unroll
            for (int q = 1; q < Q; q++)
                best = max(best, quad[q]);
            const uint32_t top = group_max<L>(best);
            mine = l == r ? top : mine;
            // the lane's lowest id with this key: its quad, and there its place
            int at = Q - 1;
#pragma unroll
            for (int q = Q - 2; q >= 0; q--)
                at = quad[q] == top ? q : at;
            uint32_t k[4];
#pragma unroll
            for (int i = 0; i < 4; i++) {
                k[i] = key[4 * (Q - 1) + i];
#pragma unroll
                for (int q = Q - 2; q >= 0; q--)
                    k[i] = at == q ? key[4 * q + i] : k[i];
            }
            const int i = k[0] == top ? 0 : k[1] == top ? 1 : k[2] == top ? 2 : 3;
            int id = e0 + 4 * L * at + i;
            bool win = top != 0 && best == top;
            const uint64_t some = __ballot(top != 0), hits = __ballot(win);
            if (__builtin_popcountll(hits) * L > __builtin_popcountll(some)) { // equal values in several lanes of a token
                const int lowest = ~(int)group_max<L>(win ? ~(uint32_t)id : 0u);
                win = win && id == lowest;
            }
            if (win)
                ids[group * L + r] = id;
            k[0] = win && i == 0 ? 0u : k[0];
            k[1] = win && i == 1 ? 0u : k[1];
            k[2] = win && i == 2 ? 0u : k[2];
            k[3] = win && i == 3 ? 0u : k[3];
            const uint32_t left = max(max(k[0], k[1]), max(k[2], k[3]));
#pragma unroll
            for (int q = 0; q < Q; q++) {
                quad[q] = at == q ? left : quad[q];
#pragma unroll
                for (int j = 0; j < 4; j++)
                    key[4 * q + j] = at == q ? k[j] : key[4 * q + j];
            }
        }
        // lane r: slot r, its expert, logit (read again: its line is near) and weight
        int expert = -1;
        float zr = NEG_INF;
        wave_sync();
        if (mine) {
            expert = ids[threadIdx.x];
            zr = BF16 ? __uint_as_float((uint32_t)((const uint16_t *)a.z)[t * a.ldz + expert] << 16)
                      : ((const float *)a.z)[t * a.ldz + expert];
            atomicAdd(&cnt[expert], 1); // integers: any order gives the same counts
        }
        wave_sync();
        float w;
        if (a.renorm) { // from the largest chosen logit: a larger one need not be among them
            const float m = key_logit<false>(group_max<L>(mine ? logit_key<false>(zr, 0) : 0u));
            w = mine ? numerator<SCORE>(zr, SCORE == FGB_ROUTER_SIGMOID ? fminf(m, 0.0f) : m) : 0.0f;
            w = w / group_sum<L>(w);
            // (a NaN logit is not chosen, but must not go unseen either)
            w = n.inv == n.inv ? w : n.inv;
        } else {
            w = SCORE == FGB_ROUTER_SIGMOID ? sigmoid(zr).s : numerator<SCORE>(zr, n.m) * n.inv;
        }
        if (t < a.T && l < a.k) {
            a.idx[t * a.k + l] = expert;
            a.w[t * a.k + l] = expert < 0 ? 0.0f : a.scale * w;
        }
    }
    finish_workgroup<L, R>(a, red, cnt, psum, live_n);
}

template <bool BF16, int SCORE> static void launch_grouped(GroupedArgs a, int lanes, hipStream_t st)
{
    const unsigned grid = (unsigned)router_blocks(a.T, lanes);
    const int L = at_least_slots(lanes, a.k), groups = 256 / L;
    const int Q = (a.E + 4 * L - 1) / (4 * L);
    a.lanes = group_lanes(a.E, a.groups, L);
    const size_t lds = 4 * ((a.loss ? groups * a.E : 0) + a.E + 1 + group_words(a.E, a.groups, L, a.lanes));
#define FGB_R(LANES, PER)                                                                                              \
    if (L == LANES && Q == PER)                                                                                        \
        router_grouped_kernel<BF16, SCORE, LANES, PER><<<grid, 256, lds, st>>>(a);
#define FGB_L(LANES) FGB_R(LANES, 1) FGB_R(LANES, 2) FGB_R(LANES, 3) FGB_R(LANES, 4)
    FGB_L(8)
    FGB_L(16)
    FGB_L(32)
    FGB_L(64)
#undef FGB_L
#undef FGB_R
}

// b + rate sign(mean - counts): whole numbers are compared, counts_e E against their sum.
__global__ __launch_bounds__(1024) void moe_bias_kernel(const float *b, const int32_t *counts, int E, float rate, float *out)
{
    __shared__ long long red[16];
    const int e = threadIdx.x;
    const float before = e < E ? b[e] : 0.0f; // (all of it before anything is written: out may lie over it)
    long long c = e < E ? counts[e] : 0, sum = c;
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1)
        sum += __shfl_xor(sum, d);
    if (lane_id() == 0)
        red[e >> 6] = sum;
    __syncthreads();
    sum = 0;
    for (int i = 0; i < (int)(blockDim.x >> 6); i++)
        sum += red[i];
    c *= E;
    if (e < E)
        out[e] = before + (c < sum ? rate : c > sum ? -rate : 0.0f);
}

} // namespace fgb

using namespace fgb;

// The most workgroups of any T' <= T: with more than the plain router's lanes 65536 lanes at most,
// with 64 lanes four tokens a workgroup.  (router_blocks(T, grouped_lanes(T, E)) itself falls where
// a token's lanes halve.)
extern "C" size_t moe_router_grouped_workspace_size(int64_t T, int E)
{
    if (T < 0 || E < 1 || E > 1024)
        return 0;
    const int64_t plain = router_blocks(T, router_lanes(E)), spread = T < 1024 ? (T + 3) / 4 : 256;
    return router_workspace(plain == 1 || plain > spread ? plain : spread, E);
}

extern "C" int moe_router_grouped(const void *logits, int dtype, int64_t T, int E, int64_t ld, int topk,
                                  const uint8_t *token_mask, const float *bias, int groups, int topk_groups, int score,
                                  int renorm, float scale, float loss_coef, int32_t *topk_idx, float *weights,
                                  int32_t *counts, float *loss, void *workspace, size_t ws_bytes, void *stream)
{
    clear_error();
    const char *name = "moe_router_grouped";
    FGB_REQUIRE(groups >= 1 && groups <= 64 && E % groups == 0, FGB_EINVAL,
                "%s: groups must be in [1, 64] and divide E (groups=%d E=%d)", name, groups, E);
    FGB_REQUIRE(topk_groups >= 1 && topk_groups <= groups && topk <= topk_groups * (E / groups), FGB_EINVAL,
                "%s: topk_groups must be in [1, groups] and hold topk experts (topk_groups=%d topk=%d)", name,
                topk_groups, topk);
    FGB_REQUIRE(((uintptr_t)bias & 3) == 0, FGB_EINVAL, "%s: bias must be 4-byte aligned", name);
    GroupedArgs a{};
    // (A workspace for the plain router's workgroups only: its lanes.  1000 x 256 FP32: 18.6 us, 13.4
    // with its own.)
    int lanes = grouped_lanes(T, E);
    const size_t own = router_workspace(router_blocks(T, lanes), E);
    if (own > 0 && (!workspace || ws_bytes < own))
        lanes = router_lanes(E);
    const int64_t blocks = router_blocks(T, lanes);
    const int rc = router_forward_args(name, a, blocks, logits, dtype, T, E, ld, topk, token_mask, score, renorm, scale, loss_coef,
                                 topk_idx, weights, counts, loss, workspace, ws_bytes);
    if (rc != FGB_OK)
        return rc;
    a.bias = bias; a.groups = groups; a.topk_groups = topk_groups; a.of = E / groups;
    const hipStream_t st = (hipStream_t)stream;
    if (dtype == FGB_BF16)
        score == FGB_ROUTER_SOFTMAX ? launch_grouped<true, FGB_ROUTER_SOFTMAX>(a, lanes, st)
                                    : launch_grouped<true, FGB_ROUTER_SIGMOID>(a, lanes, st);
    else
        score == FGB_ROUTER_SOFTMAX ? launch_grouped<false, FGB_ROUTER_SOFTMAX>(a, lanes, st)
                                    : launch_grouped<false, FGB_ROUTER_SIGMOID>(a, lanes, st);
    FGB_LAUNCHED("router_grouped_kernel");
    return router_finish(a, blocks, st);
}

extern "C" int moe_bias_update(const float *bias, const int32_t *counts, int E, float rate, float *out, void *stream)
{
    clear_error();
    FGB_REQUIRE(E >= 1 && E <= 1024, FGB_EINVAL, "moe_bias_update: need 1 <= E <= 1024 (E=%d)", E);
    FGB_REQUIRE(bias && counts && out && (((uintptr_t)bias | (uintptr_t)counts | (uintptr_t)out) & 3) == 0, FGB_EINVAL,
                "moe_bias_update: null or misaligned pointer");
    moe_bias_kernel<<<1, (E + 63) / 64 * 64, 0, (hipStream_t)stream>>>(bias, counts, E, rate, out);
    FGB_LAUNCHED("moe_bias_kernel");
    return FGB_OK;
}
