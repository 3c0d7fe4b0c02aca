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
// whole turns dropped exactly, whatever the position; its upper 32 bits, rounded
// to fp32's 24 (2^-26 of a turn where that is near a half), are the argument of
// sincospif.  No table of cosines by position is kept, nothing is read but the
// rot / 2 steps.
//
// A group of 4, 8 or 16 lanes takes some heads of one token.  A lane has 16 of a
// head's values: 8 first ones of pairs and the 8 second ones (or 8 neighbouring pairs),
// so that it turns them by itself, with weights, cosines and sines multiplied together
// once for all its heads:
//   out = (x P + partner R) / rms,   P = w A cos t,  R = -+ w' A sin t
// kRopeBatch heads are in flight a lane.
//
// Bound by HBM, small calls by latency.  Measured on GB300 from a graph: 16387 tokens of
// 36 heads of 128, 302 MB, 54 us (45 at the copy bandwidth); 64,800 tokens of 32 heads into
// pages, 1.06 GB, 188 us (157); one token of 24 heads 2.9 us, 64 appended ones 4.1.  (2 heads
// in flight: 65 and 220 us, 8: 56 and 264 for the registers; a CTA of 256 threads 67 and 309;
// at most 16 heads a group 54 and 197.)
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

constexpr int kRopeThreads = 128;
constexpr int kRopeBatch = 4;              // heads in flight a lane
constexpr int kRopeHeads = 32;             // of a group at most
constexpr int kRopeOffsets = 4096;         // sequences whose offsets are staged in shared memory

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

template <bool BF16> __device__ __forceinline__ void unpack8(const uint4 &v, float *f)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const float2 p = unpack2<BF16>(w[i]);
        f[2 * i] = p.x;
        f[2 * i + 1] = p.y;
    }
}

template <bool BF16> __device__ __forceinline__ uint4 round8(const float *f)
{
    return make_uint4(round2<BF16>(f[0], f[1]), round2<BF16>(f[2], f[3]),
                      round2<BF16>(f[4], f[5]), round2<BF16>(f[6], f[7]));
}

// The sequence that token t is of, or -1; offsets ascend.
__device__ __forceinline__ int sequence_of(const int32_t *offsets, int B, int t)
{
    // one new token each: a step of decoding
    if (t < B && offsets[t] == t && offsets[t + 1] == t + 1)
        return t;
    if (t < offsets[0] || t >= offsets[B])
        return -1;
    int lo = 0, hi = B - 1;                // the last sequence that begins at t or before
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (offsets[mid] <= t)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// Whether the offsets ascend within [0, T], by the whole CTA; they are staged if they fit.
__device__ __forceinline__ bool offsets_ascend(const RopeProblem &p, int32_t *staged)
{
    bool bad = false;
    for (int b = threadIdx.x; b <= p.B; b += kRopeThreads) {
        const int a = p.q_offsets[b];
        bad |= a < 0 || a > p.T || (b > 0 && a < p.q_offsets[b - 1]);
        if (p.B <= kRopeOffsets)
            staged[b] = a;
    }
    return __syncthreads_or(bad) == 0;
}

// LANES: a head's lanes, 16 values each.
template <int LANES, bool BF16, bool APPEND>
__global__ void __launch_bounds__(kRopeThreads, 4) rope_kernel(const RopeProblem p, int heads)
{
    constexpr int kGroups = kRopeThreads / LANES;
    extern __shared__ int32_t staged[];
    pdl_wait();                            // (no load here is a non-coherent one: this kernel
    pdl_trigger();                         // begins while the one before still writes)
    const int lane = threadIdx.x & 31, l = threadIdx.x % LANES;
    const unsigned mates = (LANES == 32 ? ~0u : (1u << LANES) - 1u) << (lane / LANES * LANES);
    // a CTA's groups have neighbouring tokens and the same heads
    const int t = blockIdx.x * kGroups + threadIdx.x / LANES, part = blockIdx.y;
    const int all = p.Hq + (APPEND ? 2 : 1) * p.Hkv;
    const int row0 = part * heads, row1 = min(row0 + heads, all);

    // this lane's two 16-byte chunks of a head
    const int turned_lanes = p.rot / 16, chunks = p.D / 8;
    const bool turned = l < turned_lanes;
    int c0 = l, c1 = l + turned_lanes;
    if (!turned) {
        c0 = 2 * l;                        // 2 turned_lanes + 2 (l - turned_lanes)
        c1 = c0 + 1;
    }
    const bool has0 = c0 < chunks, has1 = c1 < chunks;

    bool valid = t < p.T;
    int pos = 0, page = -1, slot = 0;
    if constexpr (APPEND) {
        if (!offsets_ascend(p, staged)) {
            if (blockIdx.x == 0 && threadIdx.x == 0 && p.dev_status)
                atomicOr(p.dev_status, W4_DEV_BAD_SLOT);
            return;
        }
        if (valid) {
            const int32_t *offsets = p.B <= kRopeOffsets ? staged : p.q_offsets;
            const int b = sequence_of(offsets, p.B, t);
            valid = b >= 0;
            if (valid) {
                const int at = max(p.lens[b], 0) - (offsets[b + 1] - t);
                const int entry = at >= 0 ? at / p.page : 0;
                if (at >= 0 && entry < p.W)
                    page = p.table[static_cast<int64_t>(b) * p.W + entry];
                if (page >= p.P)
                    page = -1;
                slot = at - entry * p.page;
                pos = p.positions ? p.positions[t] : at;
                if (page < 0 && part == 0 && l == 0 && p.dev_status)
                    atomicOr(p.dev_status, W4_DEV_BAD_PAGE);
            }
        }
    } else if (valid) {
        pos = p.positions[t];
    }
    if (!valid)
        return;                            // its mates too

    float cs[8], sn[8];
#pragma unroll
    for (int i = 0; i < 8; i++) {
        cs[i] = 1.0f;
        sn[i] = 0.0f;
        if (turned) {
            // in neighbouring pairs chunk c has pairs 4 c .. 4 c + 3
            const int f = p.interleaved ? (i < 4 ? c0 * 4 + i : c1 * 4 + i - 4) : l * 8 + i;
            const uint64_t angle = static_cast<uint64_t>(static_cast<int64_t>(pos)) *
                                   static_cast<uint64_t>(p.steps[f]);
            // half turns in [-1, 1)
            const float x = static_cast<float>(static_cast<int32_t>(angle >> 32)) * 0x1p-31f;
            sincospif(x, &sn[i], &cs[i]);
            cs[i] *= p.amplitude;
            sn[i] *= p.amplitude;
        }
    }

    // Heads [h, h_end) of one kind, from and to memory with these strides.
    auto run = [&](const uint16_t *from, int64_t from_head, uint16_t *to, int64_t to_head, int n,
                   const uint16_t *weight) {
        float P[16], R[16];
        {
            float w[16];
#pragma unroll
            for (int i = 0; i < 16; i++)
                w[i] = 1.0f;
            if (weight) {
                if (has0)
                    unpack8<BF16>(*reinterpret_cast<const uint4 *>(weight + c0 * 8), w);
                if (has1)
                    unpack8<BF16>(*reinterpret_cast<const uint4 *>(weight + c1 * 8), w + 8);
            }
            if (p.interleaved) {
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    P[2 * i] = w[2 * i] * cs[i];
                    P[2 * i + 1] = w[2 * i + 1] * cs[i];
                    R[2 * i] = -w[2 * i + 1] * sn[i];
                    R[2 * i + 1] = w[2 * i] * sn[i];
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    P[i] = w[i] * cs[i];
                    P[8 + i] = w[8 + i] * cs[i];
                    R[i] = -w[8 + i] * sn[i];
                    R[8 + i] = w[i] * sn[i];
                }
            }
        }
        for (int h0 = 0; h0 < n; h0 += kRopeBatch) {
            uint4 v[kRopeBatch][2];
#pragma unroll
            for (int u = 0; u < kRopeBatch; u++) {
                const uint16_t *x = from + (h0 + u) * from_head;
                v[u][0] = v[u][1] = make_uint4(0, 0, 0, 0);
                if (h0 + u < n && has0)
                    v[u][0] = __ldcs(reinterpret_cast<const uint4 *>(x + c0 * 8));
                if (h0 + u < n && has1)
                    v[u][1] = __ldcs(reinterpret_cast<const uint4 *>(x + c1 * 8));
            }
#pragma unroll
            for (int u = 0; u < kRopeBatch; u++) {
                if (h0 + u >= n)
                    break;
                float x[16], y[16];
                unpack8<BF16>(v[u][0], x);
                unpack8<BF16>(v[u][1], x + 8);
                float inv = 1.0f;
                if (weight) {
                    float s[4] = {};
#pragma unroll
                    for (int i = 0; i < 16; i++)
                        s[i & 3] = fmaf(x[i], x[i], s[i & 3]);
                    float sum = (s[0] + s[1]) + (s[2] + s[3]);
#pragma unroll
                    for (int o = LANES / 2; o > 0; o >>= 1)
                        sum += __shfl_xor_sync(mates, sum, o);
                    inv = rsqrtf(fmaf(sum, p.inv_d, p.eps));
                }
#pragma unroll
                for (int i = 0; i < 16; i++)
                    y[i] = x[i] * P[i];
                if (turned) {              // (others' partners may be infinite: not times zero)
                    if (p.interleaved) {
#pragma unroll
                        for (int i = 0; i < 16; i++)
                            y[i] = fmaf(x[i ^ 1], R[i], y[i]);
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; i++)
                            y[i] = fmaf(x[i ^ 8], R[i], y[i]);
                    }
                }
#pragma unroll
                for (int i = 0; i < 16; i++)
                    y[i] *= inv;
                uint16_t *o = to + (h0 + u) * to_head;
                if (has0)
                    *reinterpret_cast<uint4 *>(o + c0 * 8) = round8<BF16>(y);
                if (has1)
                    *reinterpret_cast<uint4 *>(o + c1 * 8) = round8<BF16>(y + 8);
            }
        }
    };
    const int64_t tok = t;
    if (row0 < p.Hq)
        run(p.q + tok * p.q_tok + row0 * p.q_head, p.q_head,
            p.q_out + tok * p.q_out_tok + row0 * p.q_out_head, p.q_out_head,
            min(row1, p.Hq) - row0, p.q_weight);
    const int k0 = max(row0 - p.Hq, 0), k1 = min(row1 - p.Hq, p.Hkv);
    uint16_t *k_to;
    int64_t k_head;
    if constexpr (APPEND) {
        if (!(page >= 0 && W4_IN_BOUNDS(page < p.P && slot >= 0 && slot < p.page, p.dev_status)))
            return;
        k_to = p.k_pages + page * p.page_stride + slot * p.tok_stride;
        k_head = p.head_stride;
    } else {
        k_to = p.k_out + tok * p.k_out_tok;
        k_head = p.k_out_head;
    }
    if (k0 < k1)
        run(p.k + tok * p.k_tok + k0 * p.k_head, p.k_head, k_to + k0 * k_head, k_head, k1 - k0,
            p.k_weight);
    if constexpr (APPEND) {
        const int v0 = max(row0 - p.Hq - p.Hkv, 0), v1 = row1 - p.Hq - p.Hkv;
        const uint16_t *from = p.v + tok * p.v_tok;
        uint16_t *to = p.v_pages + page * p.page_stride + slot * p.tok_stride;
        for (int h0 = v0; h0 < v1; h0 += kRopeBatch) {
            uint4 v[kRopeBatch][2];
#pragma unroll
            for (int u = 0; u < kRopeBatch; u++) {
                const uint16_t *x = from + (h0 + u) * p.v_head;
                if (h0 + u < v1 && has0)
                    v[u][0] = __ldcs(reinterpret_cast<const uint4 *>(x + c0 * 8));
                if (h0 + u < v1 && has1)
                    v[u][1] = __ldcs(reinterpret_cast<const uint4 *>(x + c1 * 8));
            }
#pragma unroll
            for (int u = 0; u < kRopeBatch; u++) {
                uint16_t *o = to + (h0 + u) * p.head_stride;
                if (h0 + u < v1 && has0)
                    *reinterpret_cast<uint4 *>(o + c0 * 8) = v[u][0];
                if (h0 + u < v1 && has1)
                    *reinterpret_cast<uint4 *>(o + c1 * 8) = v[u][1];
            }
        }
    }
}

template <int LANES>
cudaError_t launch_lanes(const RopeProblem &p, int sms, cudaStream_t stream)
{
    const int rows = p.Hq + (p.v_pages ? 2 : 1) * p.Hkv;
    constexpr int kGroups = kRopeThreads / LANES;
    // a group's heads: few where there are few in all, so that every SM has some
    const int64_t fair = static_cast<int64_t>(p.T) * rows / (static_cast<int64_t>(sms) * 16 * kGroups);
    const int most = static_cast<int>(std::min<int64_t>(std::max<int64_t>(fair, 1), kRopeHeads));
    const int parts = (rows + most - 1) / most, heads = (rows + parts - 1) / parts;
    const dim3 grid((static_cast<unsigned>(p.T) + kGroups - 1) / kGroups, parts), block(kRopeThreads);
    const size_t smem = p.v_pages && p.B <= kRopeOffsets ? sizeof(int32_t) * (p.B + 1) : 0;
    if (p.v_pages)
        return p.bf16 ? launch_pdl(rope_kernel<LANES, true, true>, grid, block, smem, stream, p, heads)
                      : launch_pdl(rope_kernel<LANES, false, true>, grid, block, smem, stream, p, heads);
    return p.bf16 ? launch_pdl(rope_kernel<LANES, true, false>, grid, block, smem, stream, p, heads)
                  : launch_pdl(rope_kernel<LANES, false, false>, grid, block, smem, stream, p, heads);
}

}  // namespace

cudaError_t launch_rope(const RopeProblem &q, cudaStream_t stream)
{
    int dev = 0, sms = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err == cudaSuccess)
        err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (err != cudaSuccess)
        return err;
    RopeProblem p = q;
    p.inv_d = 1.0f / static_cast<float>(p.D);
    return p.D <= 64    ? launch_lanes<4>(p, sms, stream)
           : p.D <= 128 ? launch_lanes<8>(p, sms, stream)
                        : launch_lanes<16>(p, sms, stream);
}

}  // namespace w4
