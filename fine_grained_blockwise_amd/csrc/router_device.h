// router_device.h -- the MoE router: the experts of each token, their weights, the
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
// L lanes (8, 16, 32 or 64, at least topk: lane j ends with slot j) take a token, so a
// wave of a 32-expert router handles eight tokens at once.  A lane holds Q <= 4 quads of
// experts, quad q of lane l being 4 (q L + l) .. + 3: a load, a store and an access to LDS
// each touch one run of memory (4999 x 257 bf16: forward with loss 19.4 us with a lane's
// experts in one run of 16, 16.3 us so; 32768 x 1024 backward 75 and 49 us).  A choice is
// a maximum over the L lanes; its logit is read back from the winning key.  All sums are
// fp32 in a fixed order (the last, over workgroups, in fp64): results do not depend on
// timing.  Launches and instruction issue bound it: 16384 x 32 logits are 2 MB.
#pragma once
#include "fgb_internal.h"

namespace fgb {

constexpr float NEG_INF = -__builtin_inff();
constexpr int NOWHERE = 0x7FFFFFF;

// Expert of a lane's j-th logit, less the lane's first (four times the lane).
template <int L> constexpr __device__ int at_quad(int j) { return j / 4 * 4 * L + j % 4; }

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
    // workspace: parts of the loss [reducing workgroups], the ticket (8 bytes), then
    double *lpart;
    int32_t *ticket;
    float *psum;   // [blocks][E]
    int32_t *pcnt; // [blocks][E + 1]
    // backward
    const float *dw;
    const float *dloss;
    void *dz;
    int64_t lddz;
};

// The lane's logits of token t, -inf past the last expert.  Only the last quad can
// reach past it (4 L (Q - 1) < E): it is read from where four experts are left and
// moved up.  (Rows need no alignment beyond the type's: the card's loads do not.)
template <bool BF16, int L, int Q>
__device__ __forceinline__ void load_logits(const RouterArgs &a, int64_t t, int e0, float (&z)[4 * Q])
{
    const int64_t row = t * a.ldz;
    if (a.E < 4) { // uniform
#pragma unroll
        for (int i = 0; i < 4; i++) {
            z[i] = NEG_INF;
            if (e0 + i < a.E)
                z[i] = BF16 ? __uint_as_float((uint32_t)((const uint16_t *)a.z)[row + e0 + i] << 16)
                            : ((const float *)a.z)[row + e0 + i];
        }
        return;
    }
#pragma unroll
    for (int q = 0; q < Q; q++) {
        const int e = q < Q - 1 ? e0 + 4 * L * q : min(e0 + 4 * L * q, a.E - 4);
        if constexpr (BF16) {
            uint2 u;
            __builtin_memcpy(&u, (const uint16_t *)a.z + row + e, 8);
            z[4 * q] = bf16lo(u.x);
            z[4 * q + 1] = bf16hi(u.x);
            z[4 * q + 2] = bf16lo(u.y);
            z[4 * q + 3] = bf16hi(u.y);
        } else {
            __builtin_memcpy(&z[4 * q], (const float *)a.z + row + e, 16);
        }
    }
    constexpr int j = 4 * (Q - 1);
    const int past = e0 + 4 * L * (Q - 1) - (a.E - 4); // experts of the lane's last quad past the last one
    if (a.E & 3) {                                     // uniform
#pragma unroll
        for (int n = 0; n < 3; n++) { // move up by one, past times
            const bool move = past > n;
            z[j] = move ? z[j + 1] : z[j];
            z[j + 1] = move ? z[j + 2] : z[j + 1];
            z[j + 2] = move ? z[j + 3] : z[j + 2];
            z[j + 3] = move ? NEG_INF : z[j + 3];
        }
    }
    if (past >= 4) {
#pragma unroll
        for (int i = 0; i < 4; i++)
            z[j + i] = NEG_INF;
    }
}

// Sum and maximum over aligned groups of L lanes; every lane gets the result.  Rows of
// 16 lanes are joined by swapping them between two copies (VALU, no LDS round trip).
template <int L> __device__ __forceinline__ float group_sum(float v)
{
#define FGB_ADD(CTRL) v += __uint_as_float(dpp<CTRL>(__float_as_uint(v)))
    FGB_ADD(FGB_DPP_QUAD_XOR1);
    FGB_ADD(FGB_DPP_QUAD_XOR2);
    FGB_ADD(FGB_DPP_HALF_MIRROR);
    if constexpr (L >= 16)
        FGB_ADD(FGB_DPP_ROW_ROR8);
#undef FGB_ADD
    if constexpr (L >= 32) {
        const auto w = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(w[0]) + __uint_as_float(w[1]);
    }
    if constexpr (L >= 64) {
        const auto w = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(w[0]) + __uint_as_float(w[1]);
    }
    return v;
}
template <int L> __device__ __forceinline__ uint32_t group_max(uint32_t v)
{
    v = group_max_u32<(L < 16 ? L : 16)>(v);
    if constexpr (L >= 32) {
        const auto w = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        v = max(w[0], w[1]);
    }
    if constexpr (L >= 64) {
        const auto w = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        v = max(w[0], w[1]);
    }
    return v;
}

// Orders a wave's LDS accesses before and after it (other lanes' among them).
__device__ __forceinline__ void wave_sync()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// Order-preserving map of expert e's logit to an unsigned key and back; 0 for -inf and
// NaN, which are never chosen.  -0 and +0 are equal logits and get one key.  A bf16
// logit's key needs 16 bits; the 16 below them hold the id, the lowest as the largest,
// so that one maximum chooses and names the expert.
template <bool BF16> __device__ __forceinline__ uint32_t logit_key(float z, int e)
{
    const uint32_t u = __float_as_uint(z == 0.0f ? 0.0f : z);
    uint32_t key = (u >> 31) ? ~u : (u | 0x80000000u);
    if constexpr (BF16)
        key = (key | 0xFFFFu) - (uint32_t)e;
    return z > NEG_INF ? key : 0u;
}
template <bool BF16> __device__ __forceinline__ float key_logit(uint32_t key)
{
    const uint32_t u = (key >> 31) ? key & 0x7FFFFFFFu : ~key;
    return __uint_as_float(BF16 ? u & 0xFFFF0000u : u);
}
__device__ __forceinline__ int key_expert_bf16(uint32_t key) { return (int)(~key & 0xFFFFu); }

// What a token's scores are formed with: for softmax m = max z and inv = 1 / sum
// exp(z - m), for sigmoid m = min(0, max z) and inv = 1 / sum t.
struct Norm {
    float m, inv;
};

// Sigmoid s and its complement, from one exponential and one reciprocal (of a number
// in [1, 2], to one unit in the last place).
struct Sig {
    float s, one_minus, r; // r = 1 / (1 + exp(-|z|))
};
__device__ __forceinline__ Sig sigmoid(float z)
{
    const float a = expf(-fabsf(z)), r = __builtin_amdgcn_rcpf(1.0f + a);
    return z > 0.0f ? Sig{r, a * r, r} : Sig{a * r, r, r};
}
// exp(z - m) (softmax: s before its division), or the sigmoid's numerator
// t = exp(z - m) / (1 + exp(z)), in the form that neither over- nor underflows:
// s itself where a logit of the token is above 0.
template <int SCORE> __device__ __forceinline__ float numerator(float z, float m)
{
    if constexpr (SCORE == FGB_ROUTER_SOFTMAX)
        return expf(z - m);
    const Sig g = sigmoid(z);
    return m < 0.0f ? expf(z - m) * g.r : g.s;
}

// The loss from sum_e counts_e sum_t p_te.
__device__ __forceinline__ void write_loss(const RouterArgs &a, double sum, int live_n)
{
    const double n = live_n > 0 ? live_n : 1;
    *a.loss = (float)((double)a.coef * a.E / (a.k * n * n) * sum);
}

// p of the lane's experts (num: the numerators; sg: the sigmoids, for that score), m
// the largest logit of the group.
template <int SCORE, int L, int R>
__device__ __forceinline__ Norm probabilities(const float (&z)[R], float m, float (&num)[R], float (&p)[R], Sig (&sg)[R])
{
    Norm n;
    n.m = m;
    float sum = 0.0f;
    if constexpr (SCORE == FGB_ROUTER_SIGMOID) {
        n.m = fminf(m, 0.0f);
#pragma unroll
        for (int j = 0; j < R; j++) {
            sg[j] = sigmoid(z[j]);
            num[j] = sg[j].s;
        }
        if (__any(n.m < 0.0f)) { // a token of the wave without a logit above 0
#pragma unroll
            for (int j = 0; j < R; j++)
                num[j] = n.m < 0.0f ? expf(z[j] - n.m) * sg[j].r : num[j];
        }
    } else {
#pragma unroll
        for (int j = 0; j < R; j++)
            num[j] = expf(z[j] - n.m);
    }
#pragma unroll
    for (int j = 0; j < R; j++)
        sum += num[j];
    n.inv = 1.0f / group_sum<L>(sum);
#pragma unroll
    for (int j = 0; j < R; j++)
        p[j] = num[j] * n.inv;
    return n;
}

// The end of a forward workgroup: its counts and sums over tokens (a group's psum and live
// tokens), groups in order; a lone workgroup finishes.  red: [groups][E], where the loss is
// wanted; cnt: [E + 1], the choices so far.
template <int L, int R>
__device__ __forceinline__ void finish_workgroup(const RouterArgs &a, float *red, int *cnt, const float (&psum)[R],
                                                 int live_n)
{
    constexpr int GROUPS = 256 / L;
    const int l = threadIdx.x % L, group = threadIdx.x / L, e0 = 4 * l;
    if (l == 0)
        atomicAdd(&cnt[a.E], live_n);
    if (a.loss) {
#pragma unroll
        for (int j = 0; j < R; j++)
            if (e0 + at_quad<L>(j) < a.E)
                red[group * a.E + e0 + at_quad<L>(j)] = psum[j];
    }
    __syncthreads();
    const bool lone = gridDim.x == 1;
    if (!lone && a.loss && blockIdx.x == 0 && threadIdx.x == 0)
        *a.ticket = 0;
    double part = 0.0;
    for (int e = threadIdx.x; e <= a.E; e += 256) {
        const int c = cnt[e];
        if (lone)
            a.counts[e] = c;
        else
            a.pcnt[(int64_t)blockIdx.x * (a.E + 1) + e] = c;
        if (a.loss && e < a.E) {
            float f = 0.0f;
            for (int g = 0; g < GROUPS; g++)
                f += red[g * a.E + e];
            if (!lone)
                a.psum[(int64_t)blockIdx.x * a.E + e] = f;
            part += (double)c * f;
        }
    }
    if (lone && a.loss) {
        __shared__ double parts[256];
        parts[threadIdx.x] = part;
        __syncthreads();
        if (threadIdx.x == 0) {
            double sum = 0.0;
            for (int i = 0; i < 256 && i < a.E; i++)
                sum += parts[i];
            write_loss(a, sum, cnt[a.E]);
        }
    }
}

// Lanes per token, by what was measured: a round of the choice costs about 10 Q + 20
// instructions for 64 / L tokens, so fewer lanes with more experts each are faster
// (forward, 16384 x 256 FP32 with the loss: 16 lanes 24 us, 32 lanes 26 us; 32768 x 512:
// 32 lanes 51 us, 64 lanes 61 us); the backward pass is level (14.7 and 13.8, 32 and 34).
static int router_lanes(int E) { return E <= 128 ? 8 : E <= 256 ? 16 : E <= 512 ? 32 : 64; }
// ... with lane j taking slot j.
static int at_least_slots(int L, int k)
{
    const int need = k <= 8 ? 8 : k <= 16 ? 16 : k <= 32 ? 32 : 64;
    return L > need ? L : need;
}

// Workgroups of the forward pass, at most three per CU (four: 16384 x 256 24 against
// 22 us, more partial results to add); one alone needs no second launch.
static int64_t router_blocks(int64_t T, int L)
{
    const int64_t per = 256 / L, n = (T + per - 1) / per;
    return n < 1 ? 1 : n < 768 ? n : 768;
}
// Lanes per token where a bias or groups choose, a longer work of a token's: as many more as
// keep every workgroup on a CU of its own (65536 lanes), or all of them in a lone one, which
// needs no second launch.  Forward kernel and reduction, 1000 x 256 FP32: 64 lanes 8.6 + 4.8
// us, 16 lanes 14.0 + 4.6; 2047 x 64: 32 lanes 8.1 + 4.8, 64 lanes 10.2 + 5.0, 8 lanes 10.9 +
// 4.4; 4000 x 256: 16 lanes 14.6 + 4.5, 64 lanes 13.2 + 6.7.
static int grouped_lanes(int64_t T, int E)
{
    int L = router_lanes(E);
    const int64_t most = T * L <= 256 ? 256 : 65536;
    while (L < 64 && 2 * L * T <= most)
        L *= 2;
    return L;
}

static int reduce_blocks(int E) { return E <= 32 ? 1 : (E + 15) / 16; }
// Bytes of workspace for the partial results of that many workgroups.
static size_t router_workspace(int64_t blocks, int E)
{
    return blocks == 1 ? 0 : (size_t)(reduce_blocks(E) + 1) * 8 + (size_t)blocks * (2 * (size_t)E + 1) * 4;
}

// What both entry points of the forward pass check, and their arguments (router.hip).
int check_router(const char *name, const void *z, int dtype, int64_t T, int E, int64_t ldz, int k, int score);
int router_forward_args(const char *name, RouterArgs &a, int64_t blocks, const void *logits, int dtype, int64_t T, int E, int64_t ld,
                        int topk, const uint8_t *token_mask, int score, int renorm, float scale, float loss_coef,
                        int32_t *topk_idx, float *weights, int32_t *counts, float *loss, void *workspace,
                        size_t ws_bytes);
// Adds the workgroups' partial results, where there are several.
int router_finish(const RouterArgs &a, int64_t blocks, hipStream_t st);

} // namespace fgb
