// router_grouped.hip -- the router whose choice a bias and groups of experts decide, and the
// bias's update (the mathematics and the kernel: router_kernel.h).
#include "router_kernel.h"

namespace fgb {

// b + rate sign(mean - counts): whole numbers are compared, counts_e E against their sum.
__global__ __launch_bounds__(1024) void moe_bias_kernel(const float *b, const int32_t *counts, int E, float rate, float *out)
{
    __shared__ long long red[16];
    const int e = threadIdx.x;
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
        out[e] = b[e] + (c < sum ? rate : c > sum ? -rate : 0.0f);
}

} // namespace fgb

using namespace fgb;

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
    RouterArgs a{};
    const int rc = router_forward_args(name, a, logits, dtype, T, E, ld, topk, token_mask, score, renorm, scale, loss_coef,
                                 topk_idx, weights, counts, loss, workspace, ws_bytes);
    if (rc != FGB_OK)
        return rc;
    a.bias = bias; a.groups = groups; a.topk_groups = topk_groups; a.of = E / groups;
    dispatch_router_fwd<true>(a, dtype, score, (hipStream_t)stream);
    FGB_LAUNCHED("router_fwd_kernel");
    return router_finish(a, (hipStream_t)stream);
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
