// router.hip -- the MoE router's kernels and entry points (the mathematics and what it shares
// with the choice by a bias and groups: router_device.h).
#include "router_device.h"

namespace fgb {

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
    finish_workgroup<L, R>(a, red, cnt, psum, live_n);
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

// Tokens whose chosen experts lie far below the largest logit, as a bias or groups can choose
// them: beside it their numerators vanish, so a renormed weight's part is formed from the
// largest chosen logit.  (Where the largest logit is chosen the numerators sum to at least
// 1/2.)  The pass over the tokens leaves them to this one, which reads the logits again for
// each step: it is rare, and in the usual pass its registers cost 3% (32768 x 512 forward and
// backward: 82.5 us, 79.6 without).  It takes tokens up to twice the limit, so that none falls
// between the two roundings of the sum.
constexpr float FAR = 0x1p-60f;

template <bool BF16, int SCORE, int L>
__device__ __forceinline__ void router_bwd_far(const RouterArgs &a, float *part, float f)
{
    constexpr int GROUPS = 256 / L;
    const int l = threadIdx.x % L, group = threadIdx.x / L;
#pragma unroll 1
    for (int64_t t0 = (int64_t)blockIdx.x * GROUPS; t0 < a.T; t0 += (int64_t)gridDim.x * GROUPS) {
        const int64_t t = min(t0 + group, a.T - 1);
        const auto logit = [&](int e) {
            return BF16 ? __uint_as_float((uint32_t)((const uint16_t *)a.z)[t * a.ldz + e] << 16)
                        : ((const float *)a.z)[t * a.ldz + e];
        };
        const int slot = t0 + group < a.T && l < a.k ? a.idx[t * a.k + l] : -1;
        const bool on = slot >= 0 && slot < a.E;
        uint32_t best = 0;
#pragma unroll 1
        for (int e = l; e < a.E; e += L)
            best = max(best, logit_key<false>(logit(e), 0));
        float m = key_logit<false>(group_max<L>(best));
        m = SCORE == FGB_ROUTER_SIGMOID ? fminf(m, 0.0f) : m;
        const float zr = on ? logit(slot) : NEG_INF;
        const float total = group_sum<L>(on ? numerator<SCORE>(zr, m) : 0.0f);
        const bool live = group_max<L>(slot >= 0 ? 1u : 0u) != 0, far = live && total < 2.0f * FAR; // as that pass has it
        if (!__any(far))
            continue;
        // the slots' parts, to their experts
        float mc = key_logit<false>(group_max<L>(logit_key<false>(zr, 0)));
        mc = SCORE == FGB_ROUTER_SIGMOID ? fminf(mc, 0.0f) : mc;
        const float D = on && a.dw ? a.scale * a.dw[t * a.k + l] : 0.0f;
        const float n = on ? numerator<SCORE>(zr, mc) : 0.0f;
        const float share = n / group_sum<L>(n);
        const float mean = group_sum<L>(on ? D * share : 0.0f);
        wave_sync();
#pragma unroll 1
        for (int e = l; e < a.E; e += L)
            part[e] = 0.0f;
        wave_sync();
        if (on)
            part[slot] = share * (D - mean);
        wave_sync();
        // the loss's part
        float sum = 0.0f, gp = 0.0f;
#pragma unroll 1
        for (int e = l; e < a.E; e += L) {
            const float v = numerator<SCORE>(logit(e), m);
            sum += v;
            gp += f * (float)a.counts[e] * v;
        }
        const float inv = 1.0f / group_sum<L>(sum);
        gp = group_sum<L>(gp) * inv;
#pragma unroll 1
        for (int e = l; e < a.E; e += L) {
            const float z = logit(e), p = numerator<SCORE>(z, m) * inv;
            float dz = p * (f * (float)a.counts[e] - gp) + part[e];
            if constexpr (SCORE == FGB_ROUTER_SIGMOID)
                dz *= sigmoid(z).one_minus;
            if (far) {
                if constexpr (BF16)
                    ((__bf16 *)a.dz)[t * a.lddz + e] = (__bf16)dz;
                else
                    ((float *)a.dz)[t * a.lddz + e] = dz;
            }
        }
    }
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
    bool any_far = false;
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
        bool far = false;
        if (a.renorm) {
            const float total = group_sum<L>(chosen);
            inv = 1.0f / total;
            mean = dv * inv;
            // A lone expert's weight is constant: its part is 0, not what v (1 / v) D - D leaves,
            // which can outweigh the loss's part.
            const uint64_t slots = __ballot(slot >= 0) >> ((threadIdx.x & 63) & ~(L - 1));
            const bool lone = __builtin_popcountll(L == 64 ? slots : slots & ((1ull << (L & 63)) - 1)) == 1;
            inv = lone ? 0.0f : inv;
            mean = lone ? 0.0f : mean;
            far = live && total < FAR;
            any_far |= __any(far) != 0;
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
        if (t >= a.T || far)
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
    if (any_far)
        router_bwd_far<BF16, SCORE, L>(a, reinterpret_cast<float *>(quads), f);
}

template <bool BF16, int SCORE> static void launch_router_fwd(const RouterArgs &a, hipStream_t st)
{
    const int L = at_least_slots(router_lanes(a.E), a.k), groups = 256 / L;
    const int Q = (a.E + 4 * L - 1) / (4 * L);
    const unsigned grid = (unsigned)router_blocks(a.T, router_lanes(a.E));
    const size_t lds = (size_t)4 * ((a.loss ? groups * a.E : 0) + a.E + 1);
#define FGB_R(LANES, PER)                                                                                              \
    if (L == LANES && Q == PER)                                                                                        \
        router_fwd_kernel<BF16, SCORE, LANES, PER><<<grid, 256, lds, st>>>(a);
#define FGB_L(LANES) FGB_R(LANES, 1) FGB_R(LANES, 2) FGB_R(LANES, 3) FGB_R(LANES, 4)
    FGB_L(8)
    FGB_L(16)
    FGB_L(32)
    FGB_L(64)
#undef FGB_L
#undef FGB_R
}

template <bool BF16, int SCORE> static void launch_router_bwd(const RouterArgs &a, hipStream_t st)
{
    const int L = at_least_slots(router_lanes(a.E), a.k), groups = 256 / L;
    const int Q = (a.E + 4 * L - 1) / (4 * L);
    const int64_t n = (a.T + groups - 1) / groups;
    const unsigned grid = (unsigned)(n < 2048 ? n : 2048);
#define FGB_R(LANES, PER)                                                                                              \
    if (L == LANES && Q == PER)                                                                                        \
        router_bwd_kernel<BF16, SCORE, LANES, PER><<<grid, 256, (size_t)16 * 256 * Q, st>>>(a);
#define FGB_L(LANES) FGB_R(LANES, 1) FGB_R(LANES, 2) FGB_R(LANES, 3) FGB_R(LANES, 4)
    FGB_L(8)
    FGB_L(16)
    FGB_L(32)
    FGB_L(64)
#undef FGB_L
#undef FGB_R
}

int check_router(const char *name, const void *z, int dtype, int64_t T, int E, int64_t ldz, int k, int score)
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

int router_forward_args(const char *name, RouterArgs &a, int64_t blocks, const void *logits, int dtype, int64_t T, int E, int64_t ld,
                        int topk, const uint8_t *token_mask, int score, int renorm, float scale, float loss_coef,
                        int32_t *topk_idx, float *weights, int32_t *counts, float *loss, void *workspace,
                        size_t ws_bytes)
{
    const int rc = check_router(name, logits, dtype, T, E, ld, topk, score);
    if (rc != FGB_OK)
        return rc;
    FGB_REQUIRE(counts && (T == 0 || (topk_idx && weights)), FGB_EINVAL, "%s: null pointer", name);
    FGB_REQUIRE((((uintptr_t)topk_idx | (uintptr_t)weights | (uintptr_t)counts | (uintptr_t)loss) & 3) == 0, FGB_EINVAL,
                "%s: outputs must be 4-byte aligned", name);
    const size_t need = router_workspace(blocks, E);
    FGB_REQUIRE(need == 0 || (workspace && ws_bytes >= need), FGB_EWORKSPACE, "%s: workspace of %zu bytes needed", name,
                need);
    FGB_REQUIRE(((uintptr_t)workspace & 7) == 0, FGB_EINVAL, "%s: workspace must be 8-byte aligned", name);
    a.z = logits; a.T = T; a.ldz = ld; a.E = E; a.k = topk; a.mask = token_mask;
    a.renorm = renorm; a.scale = scale; a.coef = loss_coef;
    a.idx = topk_idx; a.w = weights; a.counts = counts; a.loss = loss;
    if (blocks > 1) {
        a.lpart = (double *)workspace;
        a.ticket = (int32_t *)(a.lpart + reduce_blocks(E));
        a.psum = (float *)(a.lpart + reduce_blocks(E) + 1);
        a.pcnt = (int32_t *)(a.psum + blocks * E);
    }
    return FGB_OK;
}

int router_finish(const RouterArgs &a, int64_t blocks, hipStream_t st)
{
    const int n = reduce_blocks(a.E);
    if (blocks == 1)
        return FGB_OK;
    if (n == 1)
        router_reduce_kernel<32><<<n, 64 * RED_WAVES, 0, st>>>(a, (int)blocks);
    else
        router_reduce_kernel<16><<<n, 64 * RED_WAVES, 0, st>>>(a, (int)blocks);
    FGB_LAUNCHED("router_reduce_kernel");
    return FGB_OK;
}

} // namespace fgb

using namespace fgb;

extern "C" size_t moe_router_workspace_size(int64_t T, int E)
{
    if (T < 0 || E < 1 || E > 1024)
        return 0;
    return router_workspace(router_blocks(T, router_lanes(E)), E);
}

extern "C" int moe_router(const void *logits, int dtype, int64_t T, int E, int64_t ld, int topk,
                          const uint8_t *token_mask, int score, int renorm, float scale, float loss_coef,
                          int32_t *topk_idx, float *weights, int32_t *counts, float *loss, void *workspace,
                          size_t ws_bytes, void *stream)
{
    clear_error();
    RouterArgs a{};
    const int64_t blocks = router_blocks(T, router_lanes(E));
    const int rc = router_forward_args("moe_router", a, blocks, logits, dtype, T, E, ld, topk, token_mask, score, renorm, scale,
                                       loss_coef, topk_idx, weights, counts, loss, workspace, ws_bytes);
    if (rc != FGB_OK)
        return rc;
    const hipStream_t st = (hipStream_t)stream;
    if (dtype == FGB_BF16)
        score == FGB_ROUTER_SOFTMAX ? launch_router_fwd<true, FGB_ROUTER_SOFTMAX>(a, st)
                                    : launch_router_fwd<true, FGB_ROUTER_SIGMOID>(a, st);
    else
        score == FGB_ROUTER_SOFTMAX ? launch_router_fwd<false, FGB_ROUTER_SOFTMAX>(a, st)
                                    : launch_router_fwd<false, FGB_ROUTER_SIGMOID>(a, st);
    FGB_LAUNCHED("router_fwd_kernel");
    return router_finish(a, blocks, st);
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
    const hipStream_t st = (hipStream_t)stream;
    if (dtype == FGB_BF16)
        score == FGB_ROUTER_SOFTMAX ? launch_router_bwd<true, FGB_ROUTER_SOFTMAX>(a, st)
                                    : launch_router_bwd<true, FGB_ROUTER_SIGMOID>(a, st);
    else
        score == FGB_ROUTER_SOFTMAX ? launch_router_bwd<false, FGB_ROUTER_SOFTMAX>(a, st)
                                    : launch_router_bwd<false, FGB_ROUTER_SIGMOID>(a, st);
    FGB_LAUNCHED("router_bwd_kernel");
    return FGB_OK;
}
