// rope.cu -- the norms of queries and keys for each head and the rotation by
// their position, in one pass over the projections' output; keys and values
// may go to their pages of a cache in the same pass.
//   u = x w / sqrt(mean(x^2) + eps)             over a head's D values
//   (a, b) -> A (a cos t - b sin t, a sin t + b cos t)   for the pairs of its
//                                               first `rot` values, t = pos f_i
// Arithmetic is fp32, each value is rounded once.
//
// Angles.  A frequency is held as the fraction of a turn per position, 64 bits
// after the point (a step).  pos * step modulo 2^64 is then the angle with its
// whole turns dropped exactly, whatever the position; its upper 32 bits are the
// argument of sincospif, 2^-32 of a turn from the product.  No table of
// cosines by position is kept, nothing is read but the rot / 2 steps.
//
// A CTA takes a few tokens.  Its threads first request their heads' values,
// then work out the tokens' cosines and sines once for all heads into shared
// memory.  A head is a group of 8, 16 or 32 lanes with 16 bytes each; the values
// of the other half that a pair needs come by shuffles.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/w4moe.h"
#include "checks.cuh"
#include "launch.h"
#include "ptx.cuh"

namespace w4 {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeTokens = 16;            // of a CTA at most
constexpr int kRopeBatch = 4;              // heads in flight a thread

template <bool BF16> __device__ __forceinline__ float2 unpack2(uint32_t v)
{
    if constexpr (BF16)
        return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
    else
        return __half22float2(*reinterpret_cast<const __half2 *>(&v));
}

template <bool BF16> __device__ __forceinline__ uint32_t round2(float lo, float hi)
{
    uint32_t r;
    if constexpr (BF16)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

template <bool BF16> __device__ __forceinline__ void unpack8(const uint4 &v, float (&f)[8])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const float2 p = unpack2<BF16>(w[i]);
        f[2 * i] = p.x;
        f[2 * i + 1] = p.y;
    }
}

// Where the tokens of a CTA go: their sequence's page, or nowhere.
struct Place {
    int pos;                               // position of the rotation
    int valid;                             // whether the token is of a sequence
    int page;                              // its page, or -1
    int slot;                              // and its place there
};

// The tokens' sequences, by all threads: each looks at its share of the offsets.  With
// offsets that do not ascend from 0 to T no token is of a sequence.
__device__ __forceinline__ void find_places(const RopeProblem &p, int t0, int n, Place *place)
{
    const int tid = threadIdx.x;
    bool bad = false;
    if (tid < n)
        place[tid].valid = 0;
    __syncthreads();
    for (int b = tid; b < p.B; b += kRopeThreads) {
        const int a = __ldg(p.q_offsets + b), e = __ldg(p.q_offsets + b + 1);
        if (a < 0 || e < a || e > p.T) {
            bad = true;
            continue;
        }
        for (int t = max(a, t0); t < min(e, t0 + n); t++) {
            const int at = max(p.lens[b], 0) - (e - t);
            const int entry = at >= 0 ? at / p.page : 0;
            const int id = at >= 0 && entry < p.W
                               ? __ldg(p.table + static_cast<int64_t>(b) * p.W + entry)
                               : -1;
            Place &out = place[t - t0];
            out.pos = p.positions ? p.positions[t] : at;
            out.page = id >= 0 && id < p.P ? id : -1;
            out.slot = at - entry * p.page;
            out.valid = 1;
            if (out.page < 0 && p.dev_status)
                atomicOr(p.dev_status, W4_DEV_BAD_PAGE);
        }
    }
    if (__syncthreads_or(bad)) {
        if (tid < n)
            place[tid].valid = 0;
        if (tid == 0 && blockIdx.x == 0 && p.dev_status)
            atomicOr(p.dev_status, W4_DEV_BAD_SLOT);
        __syncthreads();
    }
}

// Where pair f of a token stands in shared memory: a lane's pairs two by two, side by
// side with the other lanes' same two, so that 16-byte reads meet no bank twice.
__device__ __forceinline__ int turn_at(int f, int lane_pairs, int half)
{
    const int chunk = f / lane_pairs, i = f - chunk * lane_pairs;
    return ((i >> 1) * (half / lane_pairs) + chunk) * 2 + (i & 1);
}

// LANES: a head's lanes, 8 values each, D / 8 of them in use.
template <int LANES, bool BF16, bool APPEND>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeProblem p, int tokens)
{
    constexpr int kGroups = kRopeThreads / LANES;
    // [tokens][rot / 2]: A cos, A sin of a token's pairs in the order of turn_at
    extern __shared__ __align__(16) float2 turn[];
    __shared__ Place place[kRopeTokens];
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x, c = tid % LANES, group = tid / LANES;
    const int t0 = blockIdx.x * tokens, n = min(tokens, p.T - t0);
    const int rows = p.Hq + (APPEND ? 2 : 1) * p.Hkv, items = n * rows;
    const int half = p.rot / 2, chunks = p.D / 8;
    const int lane_pairs = p.interleaved ? 4 : 8;          // pairs that a lane has values of
    const bool in_head = c < chunks;

    // an item is one head of one token: queries, keys, values
    auto source = [&](int item) -> const uint4 * {
        const int t = item / rows, r = item - t * rows;
        const int64_t tok = t0 + t;
        const uint16_t *x;
        if (r < p.Hq)
            x = p.q + tok * p.q_tok + static_cast<int64_t>(r) * p.q_head;
        else if (!APPEND || r < p.Hq + p.Hkv)
            x = p.k + tok * p.k_tok + static_cast<int64_t>(r - p.Hq) * p.k_head;
        else
            x = p.v + tok * p.v_tok + static_cast<int64_t>(r - p.Hq - p.Hkv) * p.v_head;
        return reinterpret_cast<const uint4 *>(x + c * 8);
    };
    uint4 v[kRopeBatch];
    auto request = [&](int first) {
#pragma unroll
        for (int u = 0; u < kRopeBatch; u++) {
            const int item = first + u * kGroups;
            v[u] = make_uint4(0, 0, 0, 0);
            if (item < items && in_head)
                v[u] = __ldcs(source(item));
        }
    };
    request(group);

    if constexpr (APPEND)
        find_places(p, t0, n, place);
    for (int i = tid; i < n * half; i += kRopeThreads) {
        const int t = i / half, f = i - t * half;
        const int pos = APPEND ? place[t].pos : __ldg(p.positions + t0 + t);
        if (APPEND && !place[t].valid)
            continue;
        const uint64_t angle = static_cast<uint64_t>(static_cast<int64_t>(pos)) *
                               static_cast<uint64_t>(__ldg(p.steps + f));
        // half turns in [-1, 1)
        const float x = static_cast<float>(static_cast<int32_t>(angle >> 32)) * 0x1p-31f;
        float sn, cs;
        sincospif(x, &sn, &cs);
        turn[t * half + turn_at(f, lane_pairs, half)] =
            make_float2(cs * p.amplitude, sn * p.amplitude);
    }
    __syncthreads();

    // this lane's pairs: in halves its values are all first ones or all second ones of
    // pairs whose others the lane `other` holds
    const bool turned = c * 8 < p.rot, second = c * 8 >= half;
    const int other = p.interleaved || !turned ? c : second ? c - half / 8 : c + half / 8;
    for (int first = group; first < (items + kGroups - 1) / kGroups * kGroups;
         first += kRopeBatch * kGroups) {
        if (first != group)
            request(first);
#pragma unroll
        for (int u = 0; u < kRopeBatch; u++) {
            const int item = first + u * kGroups;
            if (item - group >= items)         // alike for the whole CTA
                break;
            const int t = min(item, items - 1) / rows, r = min(item, items - 1) - t * rows;
            const bool is_q = r < p.Hq, is_v = APPEND && r >= p.Hq + p.Hkv;
            uint4 out = v[u];
            float x[8], y[8];
            unpack8<BF16>(v[u], x);
            const uint16_t *weight = is_q ? p.q_weight : p.k_weight;
            float inv = 1.0f;
            if (p.q_weight || p.k_weight) {    // alike for the whole CTA
                float s = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; i++)
                    s = fmaf(x[i], x[i], s);
#pragma unroll
                for (int o = LANES / 2; o > 0; o >>= 1)
                    s += __shfl_xor_sync(0xffffffffu, s, o);
                if (weight && !is_v) {
                    inv = rsqrtf(s * p.inv_d + p.eps);
                    if (in_head) {
                        float w[8];
                        unpack8<BF16>(__ldg(reinterpret_cast<const uint4 *>(weight + c * 8)), w);
#pragma unroll
                        for (int i = 0; i < 8; i++)
                            x[i] *= inv * w[i];
                    }
                }
            }
            if (p.interleaved) {
#pragma unroll
                for (int i = 0; i < 8; i++)
                    y[i] = x[i ^ 1];
            } else {
#pragma unroll
                for (int i = 0; i < 8; i++)
                    y[i] = __shfl_sync(0xffffffffu, x[i], other, LANES);
            }
            if (item >= items || !in_head || (APPEND && !place[t].valid))
                continue;
            if (!is_v) {
                if (turned) {
                    const int stride = half / lane_pairs;
                    const float4 *tp = reinterpret_cast<const float4 *>(turn + t * half) +
                                       (p.interleaved ? c : second ? c - stride : c);
                    if (p.interleaved) {
#pragma unroll
                        for (int i = 0; i < 2; i++) {
                            const float4 cs = tp[i * stride];
                            x[4 * i] = fmaf(-y[4 * i], cs.y, x[4 * i] * cs.x);
                            x[4 * i + 1] = fmaf(y[4 * i + 1], cs.y, x[4 * i + 1] * cs.x);
                            x[4 * i + 2] = fmaf(-y[4 * i + 2], cs.w, x[4 * i + 2] * cs.z);
                            x[4 * i + 3] = fmaf(y[4 * i + 3], cs.w, x[4 * i + 3] * cs.z);
                        }
                    } else {
                        const float sign = second ? 1.0f : -1.0f;
#pragma unroll
                        for (int i = 0; i < 4; i++) {
                            const float4 cs = tp[i * stride];
                            x[2 * i] = fmaf(sign * y[2 * i], cs.y, x[2 * i] * cs.x);
                            x[2 * i + 1] = fmaf(sign * y[2 * i + 1], cs.w, x[2 * i + 1] * cs.z);
                        }
                    }
                }
                out = make_uint4(round2<BF16>(x[0], x[1]), round2<BF16>(x[2], x[3]),
                                 round2<BF16>(x[4], x[5]), round2<BF16>(x[6], x[7]));
            }
            const int64_t tok = t0 + t;
            uint16_t *to;
            if (is_q) {
                to = p.q_out + tok * p.q_out_tok + static_cast<int64_t>(r) * p.q_out_head;
            } else if constexpr (APPEND) {
                const Place at = place[t];
                if (at.page < 0)
                    continue;
                if (!W4_IN_BOUNDS(at.page < p.P && at.slot >= 0 && at.slot < p.page, p.dev_status))
                    continue;
                to = (is_v ? p.v_pages : p.k_pages) + at.page * p.page_stride +
                     at.slot * p.tok_stride +
                     static_cast<int64_t>(r - p.Hq - (is_v ? p.Hkv : 0)) * p.head_stride;
            } else {
                to = p.k_out + tok * p.k_out_tok + static_cast<int64_t>(r - p.Hq) * p.k_out_head;
            }
            *reinterpret_cast<uint4 *>(to + c * 8) = out;
        }
    }
}

template <int LANES>
cudaError_t launch_lanes(const RopeProblem &p, int tokens, cudaStream_t stream)
{
    const dim3 grid((p.T + tokens - 1) / tokens), block(kRopeThreads);
    const size_t smem = sizeof(float2) * tokens * (p.rot / 2);
    if (p.v_pages)
        return p.bf16 ? launch_pdl(rope_kernel<LANES, true, true>, grid, block, smem, stream, p, tokens)
                      : launch_pdl(rope_kernel<LANES, false, true>, grid, block, smem, stream, p,
                                   tokens);
    return p.bf16 ? launch_pdl(rope_kernel<LANES, true, false>, grid, block, smem, stream, p, tokens)
                  : launch_pdl(rope_kernel<LANES, false, false>, grid, block, smem, stream, p, tokens);
}

}  // namespace

cudaError_t launch_rope(const RopeProblem &q, cudaStream_t stream)
{
    RopeProblem p = q;
    p.inv_d = 1.0f / static_cast<float>(p.D);
    const int rows = p.Hq + (p.v_pages ? 2 : 1) * p.Hkv;
    const int lanes = p.D <= 64 ? 8 : p.D <= 128 ? 16 : 32;
    // as many tokens as give every group one batch
    const int tokens = std::min(std::max(kRopeThreads / lanes * kRopeBatch / rows, 1), kRopeTokens);
    return lanes == 8 ? launch_lanes<8>(p, tokens, stream)
           : lanes == 16 ? launch_lanes<16>(p, tokens, stream)
                         : launch_lanes<32>(p, tokens, stream);
}

}  // namespace w4
