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
// L lanes (8, 16, 32 or 64, at least topk: lane j ends with slot j) take a token, so a
// wave of a 32-expert router handles eight tokens at once.  A lane holds Q <= 4 quads of
// experts, quad q of lane l being 4 (q L + l) .. + 3: a load, a store and an access to LDS
// each touch one run of memory (4999 x 257 bf16: forward with loss 19.4 us with a lane's
// experts in one run of 16, 16.3 us so; 32768 x 1024 backward 75 and 49 us).  A choice is
// a maximum over the L lanes; its logit is read back from the winning key.  All sums are
// fp32 in a fixed order (the last, over workgroups, in fp64): results do not depend on
// timing.  Launches and instruction issue bound it: 16384 x 32 logits are 2 MB.
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

template <bool BF16, int SCORE, int L, int Q>
__global__ __launch_bounds__(256) void router_fwd_kernel(RouterArgs a)
{
    extern __shared__ float red[]; // [groups][E] floats (the loss's sums), then E + 1 ints
    constexpr int GROUPS = 256 / L, R = 4 * Q;
    const int l = threadIdx.x % L, group = threadIdx.x / L, e0 = 4 * l;
    int *cnt = reinterpret_cast<int *>(red + (a.loss ? GROUPS * a.E : 0));
    __shared__ int ids[BF16 ? 1 : 256]; // [groups][L]
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
            key[j] = on ? logit_key<BF16>(z[j], e0 + at_quad<L>(j)) : 0u;
            best = max(best, key[j]);
        }
        uint32_t top = group_max<L>(best);
        const uint32_t first = top; // 0: the token is not live
        // topk rounds; lane r keeps the r-th choice's key (and, through LDS, its id)
        uint32_t mine = 0;
        for (int r = 0; r < a.k; r++) {
            mine = l == r ? top : mine;
            best = 0;
            if constexpr (BF16) { // one expert has this key (no expert: all have 0)
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
                if (at != NOWHERE)
                    ids[group * L + r] = e0 + at;
#pragma unroll
                for (int j = 0; j < R; j++) {
                    key[j] = at == at_quad<L>(j) ? 0u : key[j];
                    best = max(best, key[j]);
                }
            }
            top = group_max<L>(best);
        }
        int mine_e = -1;
        if constexpr (BF16) {
            mine_e = mine ? key_expert_bf16(mine) : -1;
        } else {
            wave_sync();
            if (mine)
                mine_e = ids[threadIdx.x];
            wave_sync();
        }
        if (mine)
            atomicAdd(&cnt[mine_e], 1); // integers: any order gives the same counts
        float num[R], p[R];
        Sig sg[R];
        const Norm n = probabilities<SCORE, L, R>(z, key_logit<BF16>(first), num, p, sg);
        // lane r: the weight of slot r
        const float zr = key_logit<BF16>(mine);
        const float nr = mine ? numerator<SCORE>(zr, n.m) : 0.0f;
        float w = nr * n.inv;
        if (a.renorm) {
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

// Counts and loss from the workgroups' partial results: COLS experts a workgroup, 1024 /
// COLS threads to an expert, added in a fixed order; the first workgroup takes the live
// tokens too.  Up to 32 experts one workgroup writes the loss; beyond, the one that comes
// last (the ticket, zeroed by the forward kernel) adds the workgroups' parts, a lane each,
// in a fixed order too.  The ticket costs about 2 us, so 32 experts go to one workgroup
// (512 x 32 with the loss: 7.7 us, two workgroups 9.0 us); beyond, a CU's rate over its
// columns counts (4999 x 257: 15.8 us with 32 experts each, 15.2 us with 16).
constexpr int RED_WAVES = 16;
template <int COLS> __global__ __launch_bounds__(64 * RED_WAVES) void router_reduce_kernel(RouterArgs a, int blocks)
{
    constexpr int SLICES = 64 * RED_WAVES / COLS;
    __shared__ double fsum[RED_WAVES][COLS];
    __shared__ int csum[RED_WAVES][COLS], lsum[RED_WAVES];
    const int col = threadIdx.x % COLS, slice = threadIdx.x / COLS;
    const int e = blockIdx.x * COLS + col;
    const bool on = e < a.E;
    const int ec = on ? e : a.E - 1;
    int c = 0, live = 0;
    double f = 0.0;
    // eight partial results in flight at a time: loads without branches, the last one
    // again past the end
    for (int b0 = slice; b0 < blocks; b0 += 8 * SLICES) {
        int ci[8], li[8] = {};
        float fi[8] = {};
#pragma unroll
        for (int i = 0; i < 8; i++)
            ci[i] = a.pcnt[(int64_t)min(b0 + i * SLICES, blocks - 1) * (a.E + 1) + ec];
        if (a.loss) {
#pragma unroll
            for (int i = 0; i < 8; i++)
                fi[i] = a.psum[(int64_t)min(b0 + i * SLICES, blocks - 1) * a.E + ec];
        }
        if (blockIdx.x == 0) {
#pragma unroll
            for (int i = 0; i < 8; i++)
                li[i] = a.pcnt[(int64_t)min(b0 + i * SLICES, blocks - 1) * (a.E + 1) + a.E];
        }
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const bool in = b0 + i * SLICES < blocks;
            c += in ? ci[i] : 0;
            live += in ? li[i] : 0;
            f += in ? fi[i] : 0.0f;
        }
    }
    // a wave's slices, then the waves in order
#pragma unroll
    for (int d = COLS; d < 64; d <<= 1) {
        c += __shfl_xor(c, d);
        f += __shfl_xor(f, d);
        live += __shfl_xor(live, d);
    }
    if ((threadIdx.x & 63) < COLS) {
        const int wave = threadIdx.x >> 6;
        csum[wave][col] = c;
        fsum[wave][col] = f;
        if (col == 0)
            lsum[wave] = live;
    }
    __syncthreads();
    if (threadIdx.x >= 64)
        return;
    c = live = 0;
    f = 0.0;
#pragma unroll
    for (int s = 0; s < RED_WAVES; s++) {
        c += csum[s][col];
        live += lsum[s];
        f += fsum[s][col];
    }
    const int lane = threadIdx.x;
    const bool mine = on && lane < COLS;
    if (mine)
        a.counts[e] = c;
    double part = mine ? (double)c * f : 0.0;
#pragma unroll
    for (int d = COLS / 2; d >= 1; d >>= 1)
        part += __shfl_xor(part, d);
    if (lane == 0 && blockIdx.x == 0)
        __hip_atomic_store(&a.counts[a.E], live, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (!a.loss)
        return;
    if (gridDim.x == 1) {
        if (lane == 0)
            write_loss(a, part, live);
        return;
    }
    int before = 0;
    if (lane == 0) {
        __hip_atomic_store(&a.lpart[blockIdx.x], part, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        before = __hip_atomic_fetch_add(a.ticket, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
    }
    if (__builtin_amdgcn_readfirstlane(before) != (int)gridDim.x - 1)
        return;
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
    double sum = 0.0; // (at most 1024 / 16 workgroups)
    live = __hip_atomic_load(&a.counts[a.E], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (lane < (int)gridDim.x)
        sum = __hip_atomic_load(&a.lpart[lane], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1)
        sum += __shfl_xor(sum, d);
    if (lane == 0)
        write_loss(a, sum, live);
}

template <bool BF16, int SCORE, int L, int Q>
__global__ __launch_bounds__(256) void router_bwd_kernel(RouterArgs a)
{
    extern __shared__ uint4 lds[]; // [groups][4 L Q]: D of the chosen experts
    constexpr int GROUPS = 256 / L, R = 4 * Q;
    constexpr uint32_t NOT_CHOSEN = 0xFFFFFFFFu; // a NaN that D is never left as
    const int l = threadIdx.x % L, group = threadIdx.x / L, e0 = 4 * l;
    uint4 *quads = lds + group * (L * Q);
    uint32_t *mine = reinterpret_cast<uint32_t *>(quads);
    const int n = a.counts[a.E];
    const float dl = a.dloss ? *a.dloss : 0.0f;
    const float f = n > 0 ? (float)((double)dl * a.coef * a.E / ((double)a.k * n * n)) : 0.0f;
    float g[R];
#pragma unroll
    for (int j = 0; j < R; j++)
        g[j] = f * (float)a.counts[min(e0 + at_quad<L>(j), a.E)]; // (past the last expert p is 0)
    for (int64_t t0 = (int64_t)blockIdx.x * GROUPS; t0 < a.T; t0 += (int64_t)gridDim.x * GROUPS) {
        const int64_t t = t0 + group;
        const int slot = t < a.T && l < a.k ? a.idx[t * a.k + l] : -1;
        float z[R];
        load_logits<BF16, L, Q>(a, min(t, a.T - 1), e0, z);
        float D = slot >= 0 && a.dw ? a.scale * a.dw[t * a.k + l] : 0.0f;
        D = D == D ? D : __builtin_nanf("");
        // to the lanes of the chosen experts, through LDS (one wave's accesses are in order)
#pragma unroll
        for (int q = 0; q < Q; q++)
            quads[q * L + l] = make_uint4(NOT_CHOSEN, NOT_CHOSEN, NOT_CHOSEN, NOT_CHOSEN);
        wave_sync();
        if (slot >= 0 && slot < a.E)
            mine[slot] = __float_as_uint(D);
        wave_sync();
        uint32_t u[R];
#pragma unroll
        for (int q = 0; q < Q; q++) {
            const uint4 w = quads[q * L + l];
            u[4 * q] = w.x;
            u[4 * q + 1] = w.y;
            u[4 * q + 2] = w.z;
            u[4 * q + 3] = w.w;
        }
        float d[R];
        bool on[R];
        uint32_t best = 0;
#pragma unroll
        for (int j = 0; j < R; j++) {
            on[j] = u[j] != NOT_CHOSEN;
            d[j] = on[j] ? __uint_as_float(u[j]) : 0.0f;
            best = max(best, logit_key<false>(z[j], 0));
        }
        const bool live = group_max<L>(slot >= 0 ? 1u : 0u) != 0;
        float num[R], p[R], dz[R];
        Sig sg[R];
        probabilities<SCORE, L, R>(z, key_logit<false>(group_max<L>(best)), num, p, sg);
        float gp = 0.0f, chosen = 0.0f, dv = 0.0f, v[R];
#pragma unroll
        for (int j = 0; j < R; j++) {
            gp += g[j] * p[j];
            v[j] = !on[j] ? 0.0f : a.renorm ? num[j] : SCORE == FGB_ROUTER_SIGMOID ? sg[j].s : p[j];
            chosen += v[j];
            dv += d[j] * v[j];
        }
        gp = group_sum<L>(gp);
        dv = group_sum<L>(dv);
        float mean = 0.0f, inv = 1.0f;
        if (a.renorm) {
            inv = 1.0f / group_sum<L>(chosen);
            mean = dv * inv;
        }
#pragma unroll
        for (int j = 0; j < R; j++) {
            float w = v[j] * inv * (d[j] - mean);
            float q = p[j] * (g[j] - gp);
            if constexpr (SCORE == FGB_ROUTER_SOFTMAX) {
                if (!a.renorm)
                    q -= p[j] * dv;
            } else {
                w *= sg[j].one_minus;
                q *= sg[j].one_minus;
            }
            dz[j] = !live ? 0.0f : on[j] ? q + w : q;
        }
        if (t >= a.T)
            continue;
        const int64_t row = t * a.lddz;
#pragma unroll
        for (int q = 0; q < Q; q++) {
            const int e = e0 + 4 * L * q, j = 4 * q;
            if (e + 4 <= a.E) {
                if constexpr (BF16) {
                    const uint2 w = make_uint2(pack_bf16x2(dz[j], dz[j + 1]), pack_bf16x2(dz[j + 2], dz[j + 3]));
                    __builtin_memcpy((uint16_t *)a.dz + row + e, &w, 8);
                } else {
                    __builtin_memcpy((float *)a.dz + row + e, &dz[j], 16);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 3; i++)
                    if (e + i < a.E) {
                        if constexpr (BF16)
                            ((__bf16 *)a.dz)[row + e + i] = (__bf16)dz[j + i];
                        else
                            ((float *)a.dz)[row + e + i] = dz[j + i];
                    }
            }
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

template <bool BF16, int SCORE, bool FWD> static void launch_router(RouterArgs a, hipStream_t st)
{
    const int L = at_least_slots(router_lanes(a.E), a.k), groups = 256 / L;
    const int Q = (a.E + 4 * L - 1) / (4 * L);
    const int64_t n = (a.T + groups - 1) / groups;
    const unsigned grid = (unsigned)(FWD ? router_blocks(a.T, a.E) : n < 2048 ? n : 2048);
    const size_t lds = FWD ? (size_t)4 * ((a.loss ? groups * a.E : 0) + a.E + 1) : (size_t)16 * 256 * Q;
#define FGB_R(LANES, PER)                                                                                              \
    if (L == LANES && Q == PER) {                                                                                      \
        if constexpr (FWD)                                                                                             \
            router_fwd_kernel<BF16, SCORE, LANES, PER><<<grid, 256, lds, st>>>(a);                                     \
        else                                                                                                           \
            router_bwd_kernel<BF16, SCORE, LANES, PER><<<grid, 256, lds, st>>>(a);                                     \
    }
#define FGB_L(LANES) FGB_R(LANES, 1) FGB_R(LANES, 2) FGB_R(LANES, 3) FGB_R(LANES, 4)
    FGB_L(8)
    FGB_L(16)
    FGB_L(32)
    FGB_L(64)
#undef FGB_L
#undef FGB_R
}

template <bool FWD> static void dispatch_router(const RouterArgs &a, int dtype, int score, hipStream_t st)
{
    const bool bf16 = dtype == FGB_BF16;
    if (bf16)
        score == FGB_ROUTER_SOFTMAX ? launch_router<true, FGB_ROUTER_SOFTMAX, FWD>(a, st)
                                    : launch_router<true, FGB_ROUTER_SIGMOID, FWD>(a, st);
    else
        score == FGB_ROUTER_SOFTMAX ? launch_router<false, FGB_ROUTER_SOFTMAX, FWD>(a, st)
                                    : launch_router<false, FGB_ROUTER_SIGMOID, FWD>(a, st);
}

} // namespace fgb

using namespace fgb;

extern "C" size_t moe_router_workspace_size(int64_t T, int E)
{
    if (T < 0 || E < 1 || E > 1024)
        return 0;
    const int64_t blocks = router_blocks(T, E);
    return blocks == 1 ? 0 : (size_t)(reduce_blocks(E) + 1) * 8 + (size_t)blocks * (2 * (size_t)E + 1) * 4;
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
    const size_t need = moe_router_workspace_size(T, E);
    FGB_REQUIRE(need == 0 || (workspace && ws_bytes >= need), FGB_EWORKSPACE, "moe_router: workspace of %zu bytes needed",
                need);
    FGB_REQUIRE(((uintptr_t)workspace & 7) == 0, FGB_EINVAL, "moe_router: workspace must be 8-byte aligned");
    const int64_t blocks = router_blocks(T, E);
    RouterArgs a{};
    a.z = logits; a.T = T; a.ldz = ld; a.E = E; a.k = topk; a.mask = token_mask;
    a.renorm = renorm; a.scale = scale; a.coef = loss_coef;
    a.idx = topk_idx; a.w = weights; a.counts = counts; a.loss = loss;
    if (blocks > 1) {
        a.lpart = (double *)workspace;
        a.ticket = (int32_t *)(a.lpart + reduce_blocks(E));
        a.psum = (float *)(a.lpart + reduce_blocks(E) + 1);
        a.pcnt = (int32_t *)(a.psum + blocks * E);
    }
    dispatch_router<true>(a, dtype, score, (hipStream_t)stream);
    FGB_LAUNCHED("router_fwd_kernel");
    if (blocks > 1) {
        const int n = reduce_blocks(E);
        if (n == 1)
            router_reduce_kernel<32><<<n, 64 * RED_WAVES, 0, (hipStream_t)stream>>>(a, (int)blocks);
        else
            router_reduce_kernel<16><<<n, 64 * RED_WAVES, 0, (hipStream_t)stream>>>(a, (int)blocks);
        FGB_LAUNCHED("router_reduce_kernel");
    }
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
    dispatch_router<false>(a, dtype, score, (hipStream_t)stream);
    FGB_LAUNCHED("router_bwd_kernel");
    return FGB_OK;
}
