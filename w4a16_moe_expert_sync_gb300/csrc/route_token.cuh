// route_token.cuh -- the router's arithmetic for one token, shared by the
// router, the fused alignment and (the weights) the few-token layer: bit-identical
// weights in all.
#pragma once

#include <cfloat>
#include <cstdint>

namespace w4 {

// The weights of a token's k chosen experts, by one warp: lane j < k has the j-th
// choice's logit and gets its weight, `top` is the first's.  In float64,
// rounded to fp32 once: exp(l_j - l_top) over the sum of the k selected, summed
// in slot order.  That is the renormalised softmax of the k (the full
// softmax's normaliser cancels), so the fp32 result is the float64 softmax's,
// bar a float64 rounding difference that lands on an fp32 rounding boundary.
__device__ __forceinline__ float chosen_weight(float logit, float top, int k, int lane)
{
    const double ex = lane < k ? exp(static_cast<double>(logit) - static_cast<double>(top)) : 0.0;
    double sum = 0.0;
    for (int j = 0; j < k; j++)
        sum += __shfl_sync(0xffffffffu, ex, j);
    return lane < k ? static_cast<float>(ex / sum) : 0.0f;
}

// The router for one token, computed by one warp: the k largest logits by k
// rounds of a warp arg-max (ties to the lower expert index), then softmax
// over them.  Lane j < k returns the j-th choice in id/w; other lanes return
// id -1, w 0.  EPL = logits per lane (E <= 32 EPL).
template <int EPL>
__device__ __forceinline__ void route_token(const float *__restrict__ row, int E, int k, int lane,
                                            int *id, float *w)
{
    float v[EPL];
    uint32_t taken = 0;
#pragma unroll
    for (int i = 0; i < EPL; i++) {
        const int e = lane + 32 * i;
        v[i] = e < E ? __ldg(row + e) : 0.0f;
        if (e >= E)
            taken |= 1u << i;
    }
    float my_val = 0.0f, top = 0.0f;
    int my_idx = -1;
    for (int j = 0; j < k; j++) {
        float bv = -FLT_MAX;
        int be = 0x7fffffff;
        bool have = false;
#pragma unroll
        for (int i = 0; i < EPL; i++) {
            const int e = lane + 32 * i;
            if (!(taken >> i & 1u) && (!have || v[i] > bv)) {   // e increases with i
                bv = v[i];
                be = e;
                have = true;
            }
        }
        // warp arg-max: larger value wins, equal values go to the lower index
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const float ov = __shfl_xor_sync(0xffffffffu, bv, o);
            const int oe = __shfl_xor_sync(0xffffffffu, be, o);
            const bool oh = __shfl_xor_sync(0xffffffffu, have ? 1 : 0, o) != 0;
            if (oh && (!have || ov > bv || (ov == bv && oe < be))) {
                bv = ov;
                be = oe;
                have = true;
            }
        }
        if ((be & 31) == lane)
            taken |= 1u << (be >> 5);
        if (j == 0)
            top = bv;
        if (lane == j) {
            my_val = bv;
            my_idx = be;
        }
    }
    *id = lane < k ? my_idx : -1;
    *w = chosen_weight(my_val, top, k, lane);
}

}  // namespace w4
