// router.hip -- the MoE router: the experts of each token, their weights, the
// slots per expert, the balance loss, and the gradient of the logits.
//
// For logits z [T, E] and a token t that is live (its mask is set and it has an
// expert with z > -inf):
//   s_e = softmax(z)_e, p = s          (softmax scores), or
//   s_e = sigmoid(z_e), p = s / sum s   (sigmoid scores);
//   the experts i_1 .. i_k with the largest z (equal logits: the lowest id; -inf
//   and NaN are never chosen, a slot left over gets id -1 and weight 0);
//   w_j = scale * s_{i_j}, divided by sum_j s_{i_j} where renorm is set;
//   counts_e = the slots that chose e, n = the live tokens,
//   loss = coef * E / (k n^2) * sum_e counts_e sum_t p_te.
// Gradient, with g_e = dloss * coef * E / (k n^2) * counts_e, v_j = w_j / scale and
// D_j = scale * dw_j:
//   the loss's part  p_e (g_e - sum g p), times (1 - s_e) for sigmoid scores;
//   the weights' part, at the chosen experts,
//     renorm:   v_j (D_j - sum D v), times (1 - s) for sigmoid scores;
//     softmax:  s_j D_j, and - p_e sum_j s_j D_j at every expert;
//     sigmoid:  s_j D_j (1 - s_j).
// A renormed sigmoid weight is formed from exp(z - m) / (1 + exp(z)), m =
// min(0, max z), so that logits far below zero do not divide zero by zero.
//
// A wave takes one token at a time: lane l holds experts l R .. l R + R - 1.  All
// sums are fp32 in a fixed order (the last, over workgroups, in fp64): results do
// not depend on timing.
#include "fgb_internal.h"

namespace fgb {

constexpr float NEG_INF = -__builtin_inff();

struct RouterArgs {
    const void *z;
    int64_t T, ldz;
    int E, k;
    const uint8_t *mask;
    int renorm;
    float scale, coef;
    int32_t *idx;
    float *w;
    int32_t *counts; // [E + 1]
    float *loss;     // or NULL
    int32_t *pcnt;   // [blocks][E + 1]
    float *psum;     // [blocks][E]
    // backward
    const float *dw;
    const float *dloss;
    void *dz;
    int64_t lddz;
};

template <bool BF16> __device__ __forceinline__ float load_logit(const void *z, int64_t at)
{
    return BF16 ? __uint_as_float((uint32_t)((const uint16_t *)z)[at] << 16) : ((const float *)z)[at];
}

__device__ __forceinline__ float wave_sum(float v)
{
#pragma unroll
    for (int d = 1; d < 64; d <<= 1)
        v += __shfl_xor(v, d);
    return v;
}
__device__ __forceinline__ float wave_max(float v)
{
#pragma unroll
    for (int d = 1; d < 64; d <<= 1)
        v = fmaxf(v, __shfl_xor(v, d));
    return v;
}

// Order-preserving map of a logit to an unsigned key; 0 for -inf and NaN, which
// are never chosen.  -0 and +0 are equal logits and get one key.
__device__ __forceinline__ uint32_t logit_key(float z)
{
    const uint32_t u = __float_as_uint(z == 0.0f ? 0.0f : z);
    const uint32_t key = (u >> 31) ? ~u : (u | 0x80000000u);
    return z > NEG_INF ? key : 0u;
}

// Scores of a live token: s (and for sigmoid scores the stable numerators t of
// the renormed weights), and 1 / sum for p.
template <int SCORE, int R>
__device__ __forceinline__ void scores(const float (&z)[R], float (&s)[R], float (&p)[R], float (&t)[R])
{
    float m = NEG_INF;
#pragma unroll
    for (int j = 0; j < R; j++) {
        m = fmaxf(m, z[j]);
    }
    m = wave_max(m);
    float sum = 0.0f;
    if constexpr (SCORE == FGB_ROUTER_SOFTMAX) {
#pragma unroll
        for (int j = 0; j < R; j++) {
            s[j] = expf(z[j] - m);
            sum += s[j];
        }
        sum = wave_sum(sum);
#pragma unroll
        for (int j = 0; j < R; j++)
            t[j] = p[j] = s[j] = s[j] / sum;
    } else {
        const float m0 = fminf(m, 0.0f);
#pragma unroll
        for (int j = 0; j < R; j++) {
            // z <= 0: exp(z) / (1 + exp(z)); z > 0: 1 / (1 + exp(-z)).
            const float a = expf(-fabsf(z[j])), d = 1.0f + a;
            s[j] = (z[j] > 0.0f ? 1.0f : a) / d;
            t[j] = z[j] > 0.0f ? s[j] : expf(z[j] - m0) / d;
            sum += t[j];
        }
        sum = wave_sum(sum);
#pragma unroll
        for (int j = 0; j < R; j++)
            p[j] = t[j] / sum;
    }
}

template <bool BF16, int SCORE, int R>
__global__ __launch_bounds__(256) void router_fwd_kernel(RouterArgs a)
{
    extern __shared__ float red[]; // [4][E] floats, then [4][E + 1] ints
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    float psum[R];
    int cnt[R];
    int live_n = 0;
#pragma unroll
    for (int j = 0; j < R; j++) {
        psum[j] = 0.0f;
        cnt[j] = 0;
    }
    for (int64_t t = (int64_t)blockIdx.x * 4 + wave; t < a.T; t += (int64_t)gridDim.x * 4) {
        float z[R];
        uint32_t key[R];
        uint32_t any = 0;
        const bool on = !a.mask || a.mask[t] != 0;
#pragma unroll
        for (int j = 0; j < R; j++) {
            const int e = lane * R + j;
            z[j] = e < a.E ? load_logit<BF16>(a.z, t * a.ldz + e) : NEG_INF;
            key[j] = logit_key(z[j]);
            any |= key[j];
        }
        const bool live = on && __ballot(any != 0) != 0;
        if (!live) { // uniform
            if (lane < a.k) {
                a.idx[t * a.k + lane] = -1;
                a.w[t * a.k + lane] = 0.0f;
            }
            continue;
        }
        live_n++;
        float s[R], p[R], num[R];
        scores<SCORE, R>(z, s, p, num);
#pragma unroll
        for (int j = 0; j < R; j++)
            psum[j] += p[j];
        // top-k: the largest key over the wave, lowest lane and position first
        float mine = 0.0f, total = 0.0f;
        int mine_e = -1;
        for (int r = 0; r < a.k; r++) {
            uint32_t best = 0;
            int at = 0;
#pragma unroll
            for (int j = 0; j < R; j++)
                if (key[j] > best) {
                    best = key[j];
                    at = j;
                }
            const uint32_t top = group_max_u32<64>(best);
            if (top == 0)
                break; // uniform: nothing left to choose
            const int win = (int)__builtin_ctzll(__ballot(best == top));
            float val = 0.0f;
#pragma unroll
            for (int j = 0; j < R; j++)
                if (j == at) {
                    val = a.renorm ? num[j] : s[j];
                    if (lane == win) {
                        key[j] = 0;
                        cnt[j]++;
                    }
                }
            const float v = __shfl(val, win);
            const int e = __shfl(lane * R + at, win);
            total += v;
            if (lane == r) {
                mine = v;
                mine_e = e;
            }
        }
        if (lane < a.k) {
            a.idx[t * a.k + lane] = mine_e;
            a.w[t * a.k + lane] = mine_e < 0 ? 0.0f : a.scale * (a.renorm ? mine / total : mine);
        }
    }
    // the workgroup's counts and sums, waves in order
    float *fs = red;
    int *is = reinterpret_cast<int *>(red + 4 * a.E);
#pragma unroll
    for (int j = 0; j < R; j++) {
        const int e = lane * R + j;
        if (e < a.E) {
            fs[wave * a.E + e] = psum[j];
            is[wave * (a.E + 1) + e] = cnt[j];
        }
    }
    if (lane == 0)
        is[wave * (a.E + 1) + a.E] = live_n;
    __syncthreads();
    for (int e = threadIdx.x; e <= a.E; e += 256) {
        int c = 0;
        for (int w = 0; w < 4; w++)
            c += is[w * (a.E + 1) + e];
        a.pcnt[(int64_t)blockIdx.x * (a.E + 1) + e] = c;
        if (e < a.E) {
            float f = 0.0f;
            for (int w = 0; w < 4; w++)
                f += fs[w * a.E + e];
            a.psum[(int64_t)blockIdx.x * a.E + e] = f;
        }
    }
}

// One workgroup: counts over the workgroups' partial results, and the loss.
__global__ __launch_bounds__(256) void router_reduce_kernel(RouterArgs a, int blocks)
{
    __shared__ double part[256];
    __shared__ int live_n;
    double acc = 0.0;
    for (int e = threadIdx.x; e <= a.E; e += 256) {
        int c = 0;
        double f = 0.0;
        for (int b = 0; b < blocks; b++) {
            c += a.pcnt[(int64_t)b * (a.E + 1) + e];
            if (e < a.E)
                f += a.psum[(int64_t)b * a.E + e];
        }
        a.counts[e] = c;
        if (e == a.E)
            live_n = c;
        else
            acc += (double)c * f;
    }
    part[threadIdx.x] = acc;
    __syncthreads();
    if (threadIdx.x == 0 && a.loss) {
        double sum = 0.0;
        for (int i = 0; i < 256; i++)
            sum += part[i];
        const double n = live_n > 0 ? live_n : 1;
        *a.loss = (float)((double)a.coef * a.E / (a.k * n * n) * sum);
    }
}

template <bool BF16, int SCORE, int R>
__global__ __launch_bounds__(256) void router_bwd_kernel(RouterArgs a)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int n = a.counts[a.E];
    const float dl = a.dloss ? *a.dloss : 0.0f;
    const float f = n > 0 ? (float)((double)dl * a.coef * a.E / ((double)a.k * n * n)) : 0.0f;
    float g[R];
#pragma unroll
    for (int j = 0; j < R; j++) {
        const int e = lane * R + j;
        g[j] = e < a.E ? f * (float)a.counts[e] : 0.0f;
    }
    for (int64_t t = (int64_t)blockIdx.x * 4 + wave; t < a.T; t += (int64_t)gridDim.x * 4) {
        const int slot = lane < a.k ? a.idx[t * a.k + lane] : -1;
        float dz[R];
#pragma unroll
        for (int j = 0; j < R; j++)
            dz[j] = 0.0f;
        if (__ballot(slot >= 0) != 0) { // the token was live
            float z[R], s[R], p[R], num[R];
#pragma unroll
            for (int j = 0; j < R; j++) {
                const int e = lane * R + j;
                z[j] = e < a.E ? load_logit<BF16>(a.z, t * a.ldz + e) : NEG_INF;
            }
            scores<SCORE, R>(z, s, p, num);
            const float D = slot >= 0 && a.dw ? a.scale * a.dw[t * a.k + lane] : 0.0f;
            // the chosen experts' scores: slot r's D at its expert
            float d[R];
            bool on[R];
#pragma unroll
            for (int j = 0; j < R; j++) {
                d[j] = 0.0f;
                on[j] = false;
            }
            for (int r = 0; r < a.k; r++) {
                const int e = __shfl(slot, r);
                const float Dr = __shfl(D, r);
#pragma unroll
                for (int j = 0; j < R; j++)
                    if (e == lane * R + j) {
                        d[j] = Dr;
                        on[j] = true;
                    }
            }
            float gp = 0.0f, chosen = 0.0f, dv = 0.0f;
#pragma unroll
            for (int j = 0; j < R; j++) {
                gp += g[j] * p[j];
                const float v = on[j] ? (a.renorm ? num[j] : s[j]) : 0.0f;
                chosen += v;
                dv += d[j] * v;
            }
            gp = wave_sum(gp);
            chosen = wave_sum(chosen);
            dv = wave_sum(dv);
            const float mean = a.renorm ? dv / chosen : 0.0f;
#pragma unroll
            for (int j = 0; j < R; j++) {
                const float v = !on[j] ? 0.0f : a.renorm ? num[j] / chosen : s[j];
                float w = v * (d[j] - mean);
                float l = p[j] * (g[j] - gp);
                if constexpr (SCORE == FGB_ROUTER_SOFTMAX) {
                    if (!a.renorm)
                        l -= p[j] * dv;
                } else {
                    const float slope = 1.0f / (1.0f + expf(z[j])); // 1 - s, without cancellation
                    w *= slope;
                    l *= slope;
                }
                dz[j] = on[j] ? l + w : l;
            }
        }
#pragma unroll
        for (int j = 0; j < R; j++) {
            const int e = lane * R + j;
            if (e < a.E) {
                if constexpr (BF16)
                    ((__bf16 *)a.dz)[t * a.lddz + e] = (__bf16)dz[j];
                else
                    ((float *)a.dz)[t * a.lddz + e] = dz[j];
            }
        }
    }
}

// Workgroups of the forward pass: four tokens each and pass, at most two per CU.
static int64_t router_blocks(int64_t T) { return T < 4 ? 1 : T < 2048 ? (T + 3) / 4 : 512; }

static int check_router(const char *name, const void *z, int dtype, int64_t T, int E, int64_t ldz, int k, int score)
{
    FGB_REQUIRE(T >= 0 && E >= 1 && E <= 1024 && T < (1ll << 31), FGB_EINVAL,
                "%s: need T >= 0 and 1 <= E <= 1024 (T=%lld E=%d)", name, (long long)T, E);
    FGB_REQUIRE(k >= 1 && k <= E && k <= 64, FGB_EINVAL, "%s: need 1 <= topk <= min(E, 64) (topk=%d)", name, k);
    FGB_REQUIRE(dtype == FGB_F32 || dtype == FGB_BF16, FGB_EUNSUPPORTED, "%s: dtype must be FGB_F32 or FGB_BF16", name);
    FGB_REQUIRE(score == FGB_ROUTER_SOFTMAX || score == FGB_ROUTER_SIGMOID, FGB_EUNSUPPORTED,
                "%s: score must be FGB_ROUTER_SOFTMAX or FGB_ROUTER_SIGMOID", name);
    FGB_REQUIRE(ldz >= E, FGB_EINVAL, "%s: the row stride must be >= E", name);
    FGB_REQUIRE(T == 0 || (z && ((uintptr_t)z & (dtype == FGB_BF16 ? 1 : 3)) == 0), FGB_EINVAL,
                "%s: logits null or misaligned", name);
    return FGB_OK;
}

template <bool BF16, int SCORE, bool FWD> static void launch_router(const RouterArgs &a, int64_t grid, hipStream_t st)
{
    const size_t lds = FWD ? (size_t)4 * (2 * a.E + 1) * 4 : 0;
#define FGB_R(N)                                                                                                       \
    if constexpr (FWD)                                                                                                 \
        router_fwd_kernel<BF16, SCORE, N><<<(unsigned)grid, 256, lds, st>>>(a);                                        \
    else                                                                                                               \
        router_bwd_kernel<BF16, SCORE, N><<<(unsigned)grid, 256, lds, st>>>(a);
    if (a.E <= 64) {
        FGB_R(1)
    } else if (a.E <= 128) {
        FGB_R(2)
    } else if (a.E <= 256) {
        FGB_R(4)
    } else if (a.E <= 512) {
        FGB_R(8)
    } else {
        FGB_R(16)
    }
#undef FGB_R
}

template <bool FWD> static void dispatch_router(const RouterArgs &a, int dtype, int score, int64_t grid, hipStream_t st)
{
    if (dtype == FGB_BF16)
        score == FGB_ROUTER_SOFTMAX ? launch_router<true, FGB_ROUTER_SOFTMAX, FWD>(a, grid, st)
                                    : launch_router<true, FGB_ROUTER_SIGMOID, FWD>(a, grid, st);
    else
        score == FGB_ROUTER_SOFTMAX ? launch_router<false, FGB_ROUTER_SOFTMAX, FWD>(a, grid, st)
                                    : launch_router<false, FGB_ROUTER_SIGMOID, FWD>(a, grid, st);
}

} // namespace fgb

using namespace fgb;

extern "C" size_t moe_router_workspace_size(int64_t T, int E)
{
    if (T < 0 || E < 1 || E > 1024)
        return 0;
    return (size_t)router_blocks(T) * (2 * (size_t)E + 1) * 4;
}

extern "C" int moe_router(const void *logits, int dtype, int64_t T, int E, int64_t ld, int topk,
                          const uint8_t *token_mask, int score, int renorm, float scale, float loss_coef,
                          int32_t *topk_idx, float *weights, int32_t *counts, float *loss, void *workspace,
                          size_t ws_bytes, void *stream)
{
    clear_error();
    const int rc = check_router("moe_router", logits, dtype, T, E, ld, topk, score);
    if (rc != FGB_OK)
        return rc;
    FGB_REQUIRE(counts && (T == 0 || (topk_idx && weights)), FGB_EINVAL, "moe_router: null pointer");
    FGB_REQUIRE((((uintptr_t)topk_idx | (uintptr_t)weights | (uintptr_t)counts | (uintptr_t)loss) & 3) == 0, FGB_EINVAL,
                "moe_router: outputs must be 4-byte aligned");
    FGB_REQUIRE(workspace && ws_bytes >= moe_router_workspace_size(T, E), FGB_EWORKSPACE,
                "moe_router: workspace of %zu bytes needed", moe_router_workspace_size(T, E));
    FGB_REQUIRE(((uintptr_t)workspace & 3) == 0, FGB_EINVAL, "moe_router: workspace must be 4-byte aligned");
    const int64_t blocks = router_blocks(T);
    RouterArgs a{};
    a.z = logits; a.T = T; a.ldz = ld; a.E = E; a.k = topk; a.mask = token_mask;
    a.renorm = renorm; a.scale = scale; a.coef = loss_coef;
    a.idx = topk_idx; a.w = weights; a.counts = counts; a.loss = loss;
    a.psum = (float *)workspace;
    a.pcnt = (int32_t *)((float *)workspace + blocks * E);
    dispatch_router<true>(a, dtype, score, blocks, (hipStream_t)stream);
    FGB_LAUNCHED("router_fwd_kernel");
    router_reduce_kernel<<<1, 256, 0, (hipStream_t)stream>>>(a, (int)blocks);
    FGB_LAUNCHED("router_reduce_kernel");
    return FGB_OK;
}

extern "C" int moe_router_backward(const void *logits, int dtype, int64_t T, int E, int64_t ld, int topk,
                                   const int32_t *topk_idx, const int32_t *counts, const float *dweights,
                                   const float *dloss, int score, int renorm, float scale, float loss_coef,
                                   void *dlogits, int64_t ldd, void *stream)
{
    clear_error();
    const int rc = check_router("moe_router_backward", logits, dtype, T, E, ld, topk, score);
    if (rc != FGB_OK)
        return rc;
    if (T == 0)
        return FGB_OK;
    FGB_REQUIRE(topk_idx && counts && dlogits, FGB_EINVAL, "moe_router_backward: null pointer");
    FGB_REQUIRE((((uintptr_t)topk_idx | (uintptr_t)counts | (uintptr_t)dweights | (uintptr_t)dloss) & 3) == 0 &&
                    ((uintptr_t)dlogits & (dtype == FGB_BF16 ? 1 : 3)) == 0,
                FGB_EINVAL, "moe_router_backward: misaligned pointer");
    FGB_REQUIRE(ldd >= E, FGB_EINVAL, "moe_router_backward: the row stride of dlogits must be >= E");
    RouterArgs a{};
    a.z = logits; a.T = T; a.ldz = ld; a.E = E; a.k = topk;
    a.renorm = renorm; a.scale = scale; a.coef = loss_coef;
    a.idx = (int32_t *)topk_idx; a.counts = (int32_t *)counts; a.dw = dweights; a.dloss = dloss;
    a.dz = dlogits; a.lddz = ldd;
    dispatch_router<false>(a, dtype, score, T < 8192 ? (T + 3) / 4 : 2048, (hipStream_t)stream);
    FGB_LAUNCHED("router_bwd_kernel");
    return FGB_OK;
}
