// router_kernel.h -- the MoE router: the experts of each token, their weights, the
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
    const float *bias;           // [E] or NULL
    int groups, topk_groups, of; // groups of `of` experts
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

// The choice by other values than the logits: with a bias c = s + b, the score rounded to
// FP32 once and the sum once more (so that any correct implementation compares the same
// numbers), without one c = z.  A group's value is the sum of its two largest c with a bias,
// its largest c without; experts outside the topk_groups groups of largest value (equal
// values: the lowest id) lose their keys.
template <int L, int Q> struct Choice {
    static constexpr int R = 4 * Q;
    float bias[R];
    int of[R];      // the experts' groups
    uint32_t *keys; // [E] of the token, then its groups' values and whether they are open
    uint32_t *values, *open;

    // `lds`: GROUPS * (E + 2 groups) words, where groups > 1.
    __device__ __forceinline__ void begin(const RouterArgs &a, int e0, uint32_t *lds, int group, int groups)
    {
#pragma unroll
        for (int j = 0; j < R; j++) {
            const int e = min(e0 + at_quad<L>(j), a.E - 1);
            bias[j] = a.bias ? a.bias[e] : 0.0f;
            of[j] = e / a.of;
        }
        keys = lds + group * a.E;
        values = lds + groups * a.E + 2 * group * a.groups;
        open = values + a.groups;
    }

    // key: the logits' keys (0: unusable), most: the largest usable logit -> the keys of c.
    template <int SCORE>
    __device__ __forceinline__ void choose(const RouterArgs &a, const float (&z)[R], float most, int l, int e0,
                                           uint32_t (&key)[R])
    {
        if (a.bias) { // uniform
            double s[R], inv = 1.0;
            if constexpr (SCORE == FGB_ROUTER_SOFTMAX) {
                double sum = 0.0;
#pragma unroll
                for (int j = 0; j < R; j++) { // (equal: an infinite one has the score 1, not NaN)
                    s[j] = !key[j] ? 0.0 : z[j] == most ? 1.0 : exp((double)z[j] - (double)most);
                    sum += s[j];
                }
#pragma unroll
                for (int d = 1; d < L; d <<= 1)
                    sum += __shfl_xor(sum, d);
                inv = 1.0 / sum;
            } else {
#pragma unroll
                for (int j = 0; j < R; j++)
                    s[j] = 1.0 / (1.0 + exp(-(double)z[j]));
            }
#pragma unroll
            for (int j = 0; j < R; j++) {
                const float c = (float)(SCORE == FGB_ROUTER_SOFTMAX ? s[j] * inv : s[j]) + bias[j];
                key[j] = key[j] ? logit_key<false>(c, 0) : 0u;
            }
        }
        if (a.groups == 1) // uniform
            return;
#pragma unroll
        for (int j = 0; j < R; j++)
            if (e0 + at_quad<L>(j) < a.E)
                keys[e0 + at_quad<L>(j)] = key[j];
        wave_sync();
        for (int g = l; g < a.groups; g += L) {
            uint32_t first = 0, second = 0;
            for (int i = 0; i < a.of; i++) {
                const uint32_t k = keys[g * a.of + i];
                second = max(second, min(first, k));
                first = max(first, k);
            }
            if (a.bias && second) // (both > 0, so neither is -inf or NaN)
                first = logit_key<false>(key_logit<false>(first) + key_logit<false>(second), 0);
            values[g] = first;
        }
        wave_sync();
        for (int g = l; g < a.groups; g += L) {
            const uint32_t own = values[g];
            int before = 0;
            for (int h = 0; h < a.groups; h++) {
                const uint32_t v = values[h];
                before += v > own || (v == own && h < g);
            }
            open[g] = before < a.topk_groups;
        }
        wave_sync();
#pragma unroll
        for (int j = 0; j < R; j++)
            key[j] = open[of[j]] ? key[j] : 0u;
        wave_sync();
    }
};

template <bool BF16, int SCORE, int L, int Q, bool CHOICE>
__global__ __launch_bounds__(256) void router_fwd_kernel(RouterArgs a)
{
    extern __shared__ float red[]; // [groups][E] floats (the loss's sums), then E + 1 ints; CHOICE: choose()'s
    constexpr int GROUPS = 256 / L, R = 4 * Q;
    constexpr bool NAMED = BF16 && !CHOICE; // a key names its expert
    const int l = threadIdx.x % L, group = threadIdx.x / L, e0 = 4 * l;
    int *cnt = reinterpret_cast<int *>(red + (a.loss ? GROUPS * a.E : 0));
    __shared__ int ids[NAMED ? 1 : 256];      // [groups][L]
    __shared__ float chosen[CHOICE ? 256 : 1]; // their logits
    Choice<L, Q> how;
    if constexpr (CHOICE)
        how.begin(a, e0, reinterpret_cast<uint32_t *>(cnt + a.E + 1), group, GROUPS);
    for (int e = threadIdx.x; e <= a.E; e += 256)
        cnt[e] = 0;
    __syncthreads();
    float psum[R];
    int live_n = 0;
#pragma unroll
    for (int j = 0; j < R; j++)
        psum[j] = 0.0f;
    for (int64_t t0 = (int64_t)blockIdx.x * GROUPS; t0 < a.T; t0 += (int64_t)gridDim.x * GROUPS) {
        const int64_t t = t0 + group;
        const bool on = t < a.T && (!a.mask || a.mask[t] != 0);
        float z[R];
        uint32_t key[R], best = 0;
        load_logits<BF16, L, Q>(a, min(t, a.T - 1), e0, z);
#pragma unroll
        for (int j = 0; j < R; j++) {
            key[j] = on ? logit_key<NAMED>(z[j], e0 + at_quad<L>(j)) : 0u;
            best = max(best, key[j]);
        }
        float most = NEG_INF; // the token's largest logit
        if constexpr (CHOICE) {
            most = key_logit<false>(group_max<L>(best));
            how.template choose<SCORE>(a, z, most, l, e0, key);
            best = 0;
#pragma unroll
            for (int j = 0; j < R; j++)
                best = max(best, key[j]);
        }
        uint32_t top = group_max<L>(best);
        const uint32_t first = top; // 0: the token is not live
        // topk rounds; lane r keeps the r-th choice's key (and, through LDS, its id)
        uint32_t mine = 0;
        for (int r = 0; r < a.k; r++) {
            mine = l == r ? top : mine;
            best = 0;
            if constexpr (NAMED) { // one expert has this key (no expert: all have 0)
#pragma unroll
                for (int j = 0; j < R; j++) {
                    key[j] = key[j] == top ? 0u : key[j];
                    best = max(best, key[j]);
                }
            } else {
                int at = NOWHERE; // the lane's lowest id with the largest key, less e0
#pragma unroll
                for (int j = R - 1; j >= 0; j--)
                    at = key[j] == top ? at_quad<L>(j) : at;
                const uint64_t some = __ballot(top != 0), hits = some & __ballot(at != NOWHERE);
                if constexpr (Q == 1) { // ids grow with the lane: the lowest lane's
                    const int win = L == 64 ? __builtin_ctzll(hits | (1ull << 63))
                                            : __builtin_ctz((uint32_t)(hits >> ((threadIdx.x & 63) & ~(L - 1))) |
                                                            (L == 32 ? 0x80000000u : 1u << (L & 31)));
                    at = l == win ? at : NOWHERE;
                } else if (__builtin_popcountll(hits) * L > __builtin_popcountll(some)) {
                    // equal logits in several lanes of a token
                    const int lowest = ~(int)group_max<L>(at == NOWHERE ? 0u : ~(uint32_t)(e0 + at));
                    at = e0 + at == lowest ? at : NOWHERE;
                }
                if (at != NOWHERE) {
                    ids[group * L + r] = e0 + at;
                    if constexpr (CHOICE) {
                        float zr = 0.0f;
#pragma unroll
                        for (int j = 0; j < R; j++)
                            zr = at == at_quad<L>(j) ? z[j] : zr;
                        chosen[group * L + r] = zr;
                    }
                }
#pragma unroll
                for (int j = 0; j < R; j++) {
                    key[j] = at == at_quad<L>(j) ? 0u : key[j];
                    best = max(best, key[j]);
                }
            }
            top = group_max<L>(best);
        }
        int mine_e = -1;
        float zr = key_logit<NAMED>(mine);
        if constexpr (NAMED) {
            mine_e = mine ? key_expert_bf16(mine) : -1;
        } else {
            wave_sync();
            if (mine) {
                mine_e = ids[threadIdx.x];
                if constexpr (CHOICE)
                    zr = chosen[threadIdx.x];
            }
            wave_sync();
        }
        if (mine)
            atomicAdd(&cnt[mine_e], 1); // integers: any order gives the same counts
        float num[R], p[R];
        Sig sg[R];
        const Norm n = probabilities<SCORE, L, R>(z, CHOICE ? most : key_logit<NAMED>(first), num, p, sg);
        // lane r: the weight of slot r
        float nr = mine ? numerator<SCORE>(zr, n.m) : 0.0f;
        float w = nr * n.inv;
        if (a.renorm) {
            if constexpr (CHOICE) { // the largest logit need not be among the chosen
                const float m = key_logit<false>(group_max<L>(mine ? logit_key<false>(zr, 0) : 0u));
                nr = mine ? numerator<SCORE>(zr, SCORE == FGB_ROUTER_SIGMOID ? fminf(m, 0.0f) : m) : 0.0f;
            }
            w = nr / group_sum<L>(nr);
            // (a NaN logit is not chosen, but must not go unseen either)
            w = n.inv == n.inv ? w : n.inv;
        } else if (SCORE == FGB_ROUTER_SIGMOID) {
            w = sigmoid(zr).s;
        }
        if (t < a.T && l < a.k) {
            a.idx[t * a.k + l] = mine_e;
            a.w[t * a.k + l] = mine_e < 0 ? 0.0f : a.scale * w;
        }
        if (first != 0) {
            live_n++;
#pragma unroll
            for (int j = 0; j < R; j++)
                psum[j] += p[j];
        }
    }
    if (l == 0)
        atomicAdd(&cnt[a.E], live_n);
    if (a.loss) {
#pragma unroll
        for (int j = 0; j < R; j++)
            if (e0 + at_quad<L>(j) < a.E)
                red[group * a.E + e0 + at_quad<L>(j)] = psum[j];
    }
    __syncthreads();
    // the workgroup's counts and sums, groups in order; a lone workgroup finishes
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
static int64_t router_blocks(int64_t T, int E)
{
    const int64_t per = 256 / router_lanes(E), n = (T + per - 1) / per;
    return n < 1 ? 1 : n < 768 ? n : 768;
}

static int reduce_blocks(int E) { return E <= 32 ? 1 : (E + 15) / 16; }

template <bool BF16, int SCORE, bool CHOICE> static void launch_router_fwd(const RouterArgs &a, hipStream_t st)
{
    const int L = at_least_slots(router_lanes(a.E), a.k), groups = 256 / L;
    const int Q = (a.E + 4 * L - 1) / (4 * L);
    const unsigned grid = (unsigned)router_blocks(a.T, a.E);
    const size_t words = (size_t)(a.loss ? groups * a.E : 0) + a.E + 1 +
                         (CHOICE && a.groups > 1 ? (size_t)groups * (a.E + 2 * a.groups) : 0);
#define FGB_R(LANES, PER)                                                                                              \
    if (L == LANES && Q == PER)                                                                                        \
        router_fwd_kernel<BF16, SCORE, LANES, PER, CHOICE><<<grid, 256, 4 * words, st>>>(a);
#define FGB_L(LANES) FGB_R(LANES, 1) FGB_R(LANES, 2) FGB_R(LANES, 3) FGB_R(LANES, 4)
    FGB_L(8)
    FGB_L(16)
    FGB_L(32)
    FGB_L(64)
#undef FGB_L
#undef FGB_R
}

// The forward pass by the arguments' types.
template <bool CHOICE> static void dispatch_router_fwd(const RouterArgs &a, int dtype, int score, hipStream_t st)
{
    if (dtype == FGB_BF16)
        score == FGB_ROUTER_SOFTMAX ? launch_router_fwd<true, FGB_ROUTER_SOFTMAX, CHOICE>(a, st)
                                    : launch_router_fwd<true, FGB_ROUTER_SIGMOID, CHOICE>(a, st);
    else
        score == FGB_ROUTER_SOFTMAX ? launch_router_fwd<false, FGB_ROUTER_SOFTMAX, CHOICE>(a, st)
                                    : launch_router_fwd<false, FGB_ROUTER_SIGMOID, CHOICE>(a, st);
}

// What both entry points of the forward pass check, and their arguments (router.hip).
int check_router(const char *name, const void *z, int dtype, int64_t T, int E, int64_t ldz, int k, int score);
int router_forward_args(const char *name, RouterArgs &a, const void *logits, int dtype, int64_t T, int E, int64_t ld,
                        int topk, const uint8_t *token_mask, int score, int renorm, float scale, float loss_coef,
                        int32_t *topk_idx, float *weights, int32_t *counts, float *loss, void *workspace,
                        size_t ws_bytes);
// Adds the workgroups' partial results, where there are several.
int router_finish(const RouterArgs &a, hipStream_t st);

} // namespace fgb
