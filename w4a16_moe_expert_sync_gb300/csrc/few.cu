// few.cu -- the whole routed-expert layer for a few tokens, in two kernels:
//   few_gate_up: (router,) jobs, h[a] = gelu_tanh(x_t . deq(Wg[e])^T) * (x_t . deq(Wu[e])^T)
//   few_down:    out_t = sum_j w_j (h[t k + j] . deq(Wd[e_j])^T)
//
// With a few tokens an expert sees one or two of them, so the layer is the
// stream of the touched experts' packed weights and every weight is used
// once or twice: a tensor-memory pipeline with 128-row tiles would spend its
// time on hand-overs.  Here a warp-level fp16 MMA (16 weight rows x 8 tokens
// x 16) takes the codes themselves: a nibble masked in place is the fp16
// subnormal q 2^-24 (low nibble of a byte) or 16 q 2^-24 (high nibble), both
// exact, and so is its product with an fp16 activation.  The group's scale
// and zero are applied to the fp32 sums,
//     sum_k s (q_k - z) x_k = s (2^24 (lo + hi / 16)) - s z sum_k x_k,
// so no weight is rounded at all.  The contraction order inside a group is
// free as long as codes and activations agree on it: a lane takes 8 codes at
// a time as they lie in a word, and the activations are stored permuted.
//
// A job is one expert with up to 8 of its assignments (the MMA's columns).
#include <algorithm>
#include <cuda_fp16.h>

#include "../../include/w4moe.h"
#include "launch.h"
#include "ptx.cuh"
#include "route_token.cuh"

namespace w4 {

namespace {

constexpr int kCols = 8;          // tokens per job: the MMA's N
constexpr int kMaxA = 256;        // assignments of a call
constexpr int kMaxM = 32;

// gate_up: 16 consumer warps in groups of four that share a task's
// contraction, and one producer warp.
constexpr int kGuGroups = 4, kGuSplit = 4;
constexpr int kGuThreads = 32 * (kGuGroups * kGuSplit + 1);
constexpr int kGuMaxSlots = 8;
// down: every warp on its own
constexpr int kDnWarps = 8, kDnThreads = 32 * kDnWarps, kDnMaxSlots = 2;
constexpr int kDnRows = 16;

struct FewArgs {
    const uint16_t *x;                 // [M, d] bf16
    const float *logits;               // [M, E], or NULL: ids and w are inputs
    int32_t *ids;                      // [M, k]
    float *w;                          // [M, k]
    const uint8_t *gu_q, *dn_q;
    const uint16_t *gu_s, *gu_z, *dn_s, *dn_z;
    uint16_t *h;                       // [M k, m] fp16, permuted
    uint16_t *out;                     // [M, d] bf16
    int32_t *dev_status;
    uint64_t wait_ns;
    int M, d, m, E, k;
    int slots, slot_bytes, x_stride;   // gate_up's ring; bytes between columns of x
    int dn_slots;                      // down's slots per warp
    bool routed;                       // ids and w come from gate_up
};

// ------------------------------------------------------------------- jobs
struct Jobs {
    int n;
    int16_t expert[kMaxA];
    int16_t count[kMaxA];
    int16_t a[kMaxA][kCols];
};

struct Shared {
    Jobs jobs;
    int heads[32];
    alignas(16) int ids[kMaxA];
    float w[kMaxA];
    int abort_flag;
};

// The routing in shared memory: the router for every token (one warp per
// token), or the caller's ids.  CTA 0 of gate_up also writes the router's
// results out.
__device__ void load_routing(const FewArgs &p, Shared &s, bool publish)
{
    const int tid = threadIdx.x, A = p.M * p.k, nt = blockDim.x;
    if (p.logits) {
        const int lane = tid & 31;
        for (int t = tid >> 5; t < p.M; t += nt >> 5) {
            int id;
            float w;
            const float *row = p.logits + static_cast<int64_t>(t) * p.E;
            if (p.E <= 128)
                route_token<4>(row, p.E, p.k, lane, &id, &w);
            else
                route_token<32>(row, p.E, p.k, lane, &id, &w);
            if (lane < p.k) {
                s.ids[t * p.k + lane] = id;
                s.w[t * p.k + lane] = w;
                if (publish) {
                    p.ids[t * p.k + lane] = id;
                    p.w[t * p.k + lane] = w;
                }
            }
        }
    } else {
        for (int a = tid; a < A; a += nt) {
            const int e = p.ids[a];
            const bool ok = e >= 0 && e < p.E;
            s.ids[a] = ok ? e : -1;
            s.w[a] = p.w[a];
            if (!ok && publish && p.dev_status)
                atomicOr(p.dev_status, kDevBadExpertId);
        }
    }
    for (int a = A + tid; a < ((A + 3) & ~3); a += nt)
        s.ids[a] = -2;
    __syncthreads();
}

// Assignments grouped into jobs, every CTA for itself: assignment a opens a
// job when the number of earlier assignments to its expert is a multiple of
// 8, and the job holds it and the next seven.  Jobs are numbered in order of
// their first assignment.
__device__ void build_jobs(Shared &s, int A)
{
    const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5;
    int base = 0;
    for (int a0 = 0; a0 < A; a0 += nt) {
        const int a = a0 + tid;
        bool head = false;
        int e = -1;
        if (a < A) {
            e = s.ids[a];
            int rank = 0;
            const int4 *v = reinterpret_cast<const int4 *>(s.ids);
            for (int i = 0; i < a; i += 4) {
                const int4 q = v[i >> 2];
                rank += (q.x == e) + (q.y == e && i + 1 < a) + (q.z == e && i + 2 < a) +
                        (q.w == e && i + 3 < a);
            }
            head = e >= 0 && rank % kCols == 0;
        }
        const unsigned bal = __ballot_sync(0xffffffffu, head);
        if (lane == 0)
            s.heads[warp] = __popc(bal);
        __syncthreads();
        int before = base + __popc(bal & ((1u << lane) - 1u)), total = base;
        for (int i = 0; i < nt >> 5; i++) {
            before += i < warp ? s.heads[i] : 0;
            total += s.heads[i];
        }
        if (head) {
            s.jobs.expert[before] = static_cast<int16_t>(e);
            int n = 0;
            for (int i = a; i < A && n < kCols; i++)
                if (s.ids[i] == e)
                    s.jobs.a[before][n++] = static_cast<int16_t>(i);
            s.jobs.count[before] = static_cast<int16_t>(n);
            for (int i = n; i < kCols; i++)       // unused columns repeat the first
                s.jobs.a[before][i] = static_cast<int16_t>(a);
        }
        base = total;
        __syncthreads();
    }
    if (tid == 0)
        s.jobs.n = base;
    __syncthreads();
}

// --------------------------------------------------------------- MMA core
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Eight codes of two weight rows (one word each) against eight activations
// (x0 x4 | x2 x6 | x1 x5 | x3 x7): the low nibbles into lo, the high into hi.
__device__ __forceinline__ void mma_word(float (&lo)[4], float (&hi)[4], uint32_t w0, uint32_t w1,
                                         const uint4 &b)
{
    const uint32_t v0 = w0 >> 8, v1 = w1 >> 8;
    mma16816(lo, w0 & 0x000F000Fu, w1 & 0x000F000Fu, v0 & 0x000F000Fu, v1 & 0x000F000Fu, b.x, b.y);
    mma16816(hi, w0 & 0x00F000F0u, w1 & 0x00F000F0u, v0 & 0x00F000F0u, v1 & 0x00F000F0u, b.z, b.w);
}

constexpr float kSub = 16777216.0f;            // 2^24: the codes' subnormal scale

__device__ __forceinline__ float half_bits(const uint16_t *p)
{
    return __half2float(__ushort_as_half(*p));
}

// Position of element e of 8 in the permuted order 0 4 2 6 1 5 3 7.
__device__ __forceinline__ int perm8(int e) { return ((e & 1) << 2) | (e & 2) | (e >> 2); }

__device__ __forceinline__ float gelu_tanh_f(float v)
{
    const float u = 0.7978845608028654f * fmaf(0.044715f * v, v * v, v);
    return __fdividef(v, 1.0f + __expf(-2.0f * u));
}

// fp16 with saturation to the finite range (NaN stays NaN).
__device__ __forceinline__ uint16_t to_half_sat(float v)
{
    return __half_as_ushort(__float2half_rn(fabsf(v) > 65504.0f ? copysignf(65504.0f, v) : v));
}

// ---------------------------------------------------------------- gate_up
// Tasks are (job, 8 intermediates): 8 gate rows and the 8 up rows beside
// them make the MMA's 16 rows, so g and u of an intermediate end in the same
// lane.  CTA c takes an equal contiguous share of the tasks; its producer
// streams each task's rows (two contiguous blocks of 8 rows, and their
// scales and zeros) through a ring of slots.
__global__ void __launch_bounds__(kGuThreads, 1) few_gate_up_kernel(const __grid_constant__ FewArgs p)
{
    extern __shared__ __align__(128) uint8_t dyn[];
    __shared__ Shared s;
    __shared__ __align__(8) uint64_t full[kGuMaxSlots], empty[kGuMaxSlots];
    __shared__ float red[2][kGuGroups][kGuSplit][32][4];

    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int G = p.d / 128, A = p.M * p.k;
    uint8_t *ring = dyn;
    uint8_t *xbuf = ring + p.slots * p.slot_bytes;                       // 8 columns of x
    float *xs = reinterpret_cast<float *>(xbuf + kCols * p.x_stride);    // [G][8] group sums

    if (tid == 0) {
        for (int i = 0; i < p.slots; i++) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], kGuSplit);
        }
        s.abort_flag = 0;
        fence_mbar_init();
    }
    pdl_wait();
    pdl_trigger();
    load_routing(p, s, blockIdx.x == 0);
    build_jobs(s, A);

    const int per_job = p.m / 8;
    const int64_t total = static_cast<int64_t>(s.jobs.n) * per_job;
    const int t0 = static_cast<int>(total * blockIdx.x / gridDim.x);
    const int t1 = static_cast<int>(total * (blockIdx.x + 1) / gridDim.x);
    const int block = 4 * p.d;                 // bytes of 8 rows of codes
    const int sblock = 16 * G;                 // bytes of 8 rows of scales

    if (warp == kGuGroups * kGuSplit) {        // producer
        if (lane == 0) {
            int issued = 0;
            for (int t = t0; t < t1; t++) {
                const int i = t - t0, slot = i % p.slots;
                if (i >= p.slots && !mbar_wait(&empty[slot], (i / p.slots - 1) & 1, &s.abort_flag,
                                               p.dev_status, kDevPipelineTimeout, p.wait_ns))
                    break;
                const int e = s.jobs.expert[t / per_job];
                const int64_t gate = (static_cast<int64_t>(e) * 2 * p.m + (t % per_job) * 8);
                const int64_t up = gate + p.m;
                uint8_t *dst = ring + slot * p.slot_bytes;
                mbar_arrive_expect_tx(&full[slot], 2 * block + 4 * sblock);
                bulk_load_nohint(dst, p.gu_q + gate * (p.d / 2), block, &full[slot]);
                bulk_load_nohint(dst + block, p.gu_q + up * (p.d / 2), block, &full[slot]);
                dst += 2 * block;
                bulk_load_nohint(dst, p.gu_s + gate * G, sblock, &full[slot]);
                bulk_load_nohint(dst + sblock, p.gu_s + up * G, sblock, &full[slot]);
                bulk_load_nohint(dst + 2 * sblock, p.gu_z + gate * G, sblock, &full[slot]);
                bulk_load_nohint(dst + 3 * sblock, p.gu_z + up * G, sblock, &full[slot]);
                issued++;
            }
            // the CTA may not end while a copy into its memory is in flight
            for (int i = max(0, issued - p.slots); i < issued; i++)
                mbar_wait(&full[i % p.slots], (i / p.slots) & 1, &s.abort_flag, p.dev_status,
                          kDevPipelineTimeout, p.wait_ns);
        }
        return;
    }

    const int grp = warp / kGuSplit, part = warp % kGuSplit;
    const int g = lane >> 2, t4 = lane & 3;
    constexpr int kConsumers = 32 * kGuGroups * kGuSplit;
    int it = 0;                                // this group's tasks so far
    for (int seg = t0; seg < t1;) {            // the tasks of one job at a time
        const int job = seg / per_job;
        const int end = min(t1, (job + 1) * per_job);
        const int n = s.jobs.count[job];
        asm volatile("bar.sync 1, %0;" ::"n"(kConsumers) : "memory");   // xbuf is free
        // x rows of the job in fp16, permuted: word w of lane t4's 32 codes of
        // group gi at chunk (gi, w, t4); a warp takes one (column, group)
        bool range = false;
        for (int c = warp; c < kCols * G; c += kGuGroups * kGuSplit) {
            const int col = c / G, gi = c % G;
            if (col >= n)
                break;
            const int tok = s.jobs.a[job][col] / p.k;
            const uint2 v = *reinterpret_cast<const uint2 *>(
                p.x + static_cast<int64_t>(tok) * p.d + gi * 128 + lane * 4);
            float sum = 0.0f;
            uint8_t *dst = xbuf + col * p.x_stride +
                           ((gi * 4 + ((lane >> 1) & 3)) * 4 + (lane >> 3)) * 16;
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const uint32_t bits = i < 2 ? v.x : v.y;
                const float f = __uint_as_float(i & 1 ? bits & 0xFFFF0000u : bits << 16);
                range |= !(fabsf(f) <= 65504.0f);
                const uint16_t hb = to_half_sat(f);
                sum += __half2float(__ushort_as_half(hb));
                reinterpret_cast<uint16_t *>(dst)[perm8((lane & 1) * 4 + i)] = hb;
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (lane == 0)
                xs[gi * kCols + col] = sum;
        }
        if (range && p.dev_status)
            atomicOr(p.dev_status, kDevFp16Range);
        asm volatile("bar.sync 1, %0;" ::"n"(kConsumers) : "memory");

        const uint8_t *xcol = xbuf + (g < n ? g : 0) * p.x_stride + t4 * 16;
        for (int t = seg; t < end; t++) {
            const int i = t - t0;
            if (i % kGuGroups != grp)
                continue;
            const int slot = i % p.slots;
            mbar_wait_warp(&full[slot], (i / p.slots) & 1, &s.abort_flag, p.dev_status,
                           kDevPipelineTimeout, p.wait_ns);
            const uint8_t *base = ring + slot * p.slot_bytes;
            const uint8_t *c0 = base + g * (p.d / 2) + t4 * 16;
            const uint16_t *sc = reinterpret_cast<const uint16_t *>(base + 2 * block) + g * G;
            float acc[4] = {};
            for (int gi = part; gi < G; gi += kGuSplit) {
                const uint4 q0 = *reinterpret_cast<const uint4 *>(c0 + gi * 64);
                const uint4 q1 = *reinterpret_cast<const uint4 *>(c0 + block + gi * 64);
                const float s0 = half_bits(sc + gi), s1 = half_bits(sc + sblock / 2 + gi);
                const float z0 = half_bits(sc + sblock + gi);
                const float z1 = half_bits(sc + sblock / 2 * 3 + gi);
                const float2 sum = *reinterpret_cast<const float2 *>(xs + gi * kCols + 2 * t4);
                const uint4 *b = reinterpret_cast<const uint4 *>(xcol + gi * 256);
                float lo[4] = {}, hi[4] = {};
                mma_word(lo, hi, q0.x, q1.x, b[0]);
                mma_word(lo, hi, q0.y, q1.y, b[4]);
                mma_word(lo, hi, q0.z, q1.z, b[8]);
                mma_word(lo, hi, q0.w, q1.w, b[12]);
                acc[0] += s0 * fmaf(-z0, sum.x, kSub * fmaf(hi[0], 0.0625f, lo[0]));
                acc[1] += s0 * fmaf(-z0, sum.y, kSub * fmaf(hi[1], 0.0625f, lo[1]));
                acc[2] += s1 * fmaf(-z1, sum.x, kSub * fmaf(hi[2], 0.0625f, lo[2]));
                acc[3] += s1 * fmaf(-z1, sum.y, kSub * fmaf(hi[3], 0.0625f, lo[3]));
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&empty[slot]);
            float(*r)[32][4] = red[it & 1][grp];
            it++;
            *reinterpret_cast<float4 *>(r[part][lane]) =
                make_float4(acc[0], acc[1], acc[2], acc[3]);
            asm volatile("bar.sync %0, %1;" ::"r"(2 + grp), "n"(32 * kGuSplit) : "memory");
            const int o = part * 32 + lane;    // 64 outputs: (column, intermediate)
            if (o < 64 && (o >> 3) < n) {
                const int col = o >> 3, row = o & 7, src = row * 4 + (col >> 1);
                float gv = 0.0f, uv = 0.0f;
#pragma unroll
                for (int q = 0; q < kGuSplit; q++) {
                    gv += r[q][src][col & 1];
                    uv += r[q][src][2 + (col & 1)];
                }
                const float hv = gelu_tanh_f(gv) * uv;
                if (!(fabsf(hv) <= 65504.0f) && p.dev_status)
                    atomicOr(p.dev_status, kDevFp16Range);
                // down's order: 8 intermediates to a chunk, chunk (group of 64, w, t4)
                const int ch = t % per_job;
                const int pos = (ch >> 3) * 64 + ((ch & 1) * 4 + ((ch >> 1) & 3)) * 8 + perm8(row);
                p.h[static_cast<int64_t>(s.jobs.a[job][col]) * p.m + pos] = to_half_sat(hv);
            }
        }
        seg = end;
    }
}

// ------------------------------------------------------------------- down
// CTA b owns output columns [16 b, 16 b + 16) of every token, so the combine
// stays inside it: warps take the jobs in turn, each streaming the 16 weight
// rows of its jobs through its own slots, and leave y[a][16] in shared
// memory; then each token's terms are added in slot order.
__global__ void __launch_bounds__(kDnThreads, 2) few_down_kernel(const __grid_constant__ FewArgs p)
{
    extern __shared__ __align__(128) uint8_t dyn[];
    __shared__ Shared s;
    __shared__ __align__(8) uint64_t full[kDnWarps][kDnMaxSlots];

    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int G = p.m / 64, A = p.M * p.k;
    const int block = 8 * p.m, sblock = 32 * G;          // 16 rows of codes, of scales
    const int slot_bytes = block + 2 * sblock;
    uint8_t *ring = dyn + warp * p.dn_slots * slot_bytes;
    float *y = reinterpret_cast<float *>(dyn + kDnWarps * p.dn_slots * slot_bytes);   // [A][16]

    if (tid == 0)
        s.abort_flag = 0;
    if (lane == 0) {
        for (int i = 0; i < p.dn_slots; i++)
            mbar_init(&full[warp][i], 1);
        fence_mbar_init();
    }
    // A caller's routing and the weights are older than gate_up, which began
    // only after its predecessors had ended: they may be read before this
    // kernel waits for gate_up's h.
    if (p.routed)
        pdl_wait();
    load_routing(p, s, false);
    build_jobs(s, A);

    const int nj = s.jobs.n;
    auto issue = [&](int j, int slot) {
        const int64_t row = static_cast<int64_t>(s.jobs.expert[j]) * p.d + blockIdx.x * kDnRows;
        uint8_t *dst = ring + slot * slot_bytes;
        uint64_t *bar = &full[warp][slot];
        mbar_arrive_expect_tx(bar, slot_bytes);
        bulk_load_nohint(dst, p.dn_q + row * (p.m / 2), block, bar);
        bulk_load_nohint(dst + block, p.dn_s + row * G, sblock, bar);
        bulk_load_nohint(dst + block + sblock, p.dn_z + row * G, sblock, bar);
    };
    if (lane == 0)
        for (int i = 0; i < p.dn_slots; i++)
            if (warp + i * kDnWarps < nj)
                issue(warp + i * kDnWarps, i);
    if (!p.routed)
        pdl_wait();
    pdl_trigger();

    const int g = lane >> 2, t4 = lane & 3;
    int it = 0;
    for (int j = warp; j < nj; j += kDnWarps, it++) {
        const int n = s.jobs.count[j], slot = it % p.dn_slots;
        const uint8_t *hrow = reinterpret_cast<const uint8_t *>(
                                  p.h + static_cast<int64_t>(s.jobs.a[j][g < n ? g : 0]) * p.m) +
                              t4 * 16;
        mbar_wait_warp(&full[warp][slot], (it / p.dn_slots) & 1, &s.abort_flag, p.dev_status,
                       kDevPipelineTimeout, p.wait_ns);
        const uint8_t *base = ring + slot * slot_bytes;
        const uint8_t *c0 = base + g * (p.m / 2) + t4 * 8;
        const uint16_t *sc = reinterpret_cast<const uint16_t *>(base + block) + g * G;
        float acc[4] = {};
#pragma unroll 4
        for (int gi = 0; gi < G; gi++) {
            const uint4 b0 = __ldcg(reinterpret_cast<const uint4 *>(hrow + gi * 128));
            const uint4 b1 = __ldcg(reinterpret_cast<const uint4 *>(hrow + gi * 128 + 64));
            const uint2 q0 = *reinterpret_cast<const uint2 *>(c0 + gi * 32);
            const uint2 q1 = *reinterpret_cast<const uint2 *>(c0 + 4 * p.m + gi * 32);
            const float s0 = half_bits(sc + gi), s1 = half_bits(sc + 8 * G + gi);
            const float z0 = half_bits(sc + 16 * G + gi), z1 = half_bits(sc + 24 * G + gi);
            float lo[4] = {}, hi[4] = {}, sum[4] = {};
            mma_word(lo, hi, q0.x, q1.x, b0);
            mma_word(lo, hi, q0.y, q1.y, b1);
            constexpr uint32_t one = 0x3C003C00u;      // the sums of h, by rows of ones
            mma16816(sum, one, one, one, one, b0.x, b0.y);
            mma16816(sum, one, one, one, one, b0.z, b0.w);
            mma16816(sum, one, one, one, one, b1.x, b1.y);
            mma16816(sum, one, one, one, one, b1.z, b1.w);
            acc[0] += s0 * fmaf(-z0, sum[0], kSub * fmaf(hi[0], 0.0625f, lo[0]));
            acc[1] += s0 * fmaf(-z0, sum[1], kSub * fmaf(hi[1], 0.0625f, lo[1]));
            acc[2] += s1 * fmaf(-z1, sum[0], kSub * fmaf(hi[2], 0.0625f, lo[2]));
            acc[3] += s1 * fmaf(-z1, sum[1], kSub * fmaf(hi[3], 0.0625f, lo[3]));
        }
        __syncwarp();
        if (lane == 0 && j + p.dn_slots * kDnWarps < nj)
            issue(j + p.dn_slots * kDnWarps, slot);
#pragma unroll
        for (int c = 0; c < 2; c++) {
            if (2 * t4 + c < n) {
                float *yr = y + s.jobs.a[j][2 * t4 + c] * kDnRows;
                yr[g] = acc[c];
                yr[g + 8] = acc[2 + c];
            }
        }
    }
    __syncthreads();
    for (int o = tid; o < p.M * kDnRows; o += kDnThreads) {
        const int t = o / kDnRows, r = o % kDnRows;
        float v = 0.0f;
        for (int j = 0; j < p.k; j++) {
            const int a = t * p.k + j;
            if (s.ids[a] >= 0)
                v = fmaf(s.w[a], y[a * kDnRows + r], v);
        }
        const uint32_t u = __float_as_uint(v);           // bf16, nearest even
        const uint32_t b = v != v ? 0x7FFFu : (u + 0x7FFFu + ((u >> 16) & 1u)) >> 16;
        p.out[static_cast<int64_t>(t) * p.d + blockIdx.x * kDnRows + r] = static_cast<uint16_t>(b);
    }
}

struct FewPlan {
    int slots, slot_bytes, x_stride;
    int dn_slots;
    size_t gu_smem, dn_smem;
};

// Shared memory of both kernels; false when the shape does not fit.
bool few_plan(int M, int d, int m, int k, FewPlan *f)
{
    constexpr int kDynMax = 227 * 1024 - 25 * 1024;      // beside the static arrays
    f->slot_bytes = 8 * d + 64 * (d / 128);
    f->x_stride = 2 * d + 64;            // + 64 B: the columns' chunks fall in distinct banks
    const int fixed = kCols * f->x_stride + (d / 128) * kCols * 4;
    f->slots = std::min(kGuMaxSlots, (kDynMax - fixed) / f->slot_bytes);
    f->gu_smem = static_cast<size_t>(fixed) + static_cast<size_t>(f->slots) * f->slot_bytes;
    // down: two slots per warp where two CTAs then still fit an SM, else one
    const size_t dn_ring = static_cast<size_t>(kDnWarps) * (8 * m + 64 * (m / 64));
    const size_t y = static_cast<size_t>(M) * k * kDnRows * 4;
    f->dn_slots = 2 * dn_ring + y <= 104 * 1024 ? 2 : 1;
    f->dn_smem = f->dn_slots * dn_ring + y;
    return f->slots >= 2 && f->dn_smem <= kDynMax;
}

}  // namespace

bool few_supported(int M, int d, int m, int k)
{
    FewPlan f;
    return M <= kMaxM && M * k <= kMaxA && few_plan(M, d, m, k, &f);
}

cudaError_t launch_few(const FewProblem &q, cudaStream_t stream)
{
    FewPlan f;
    if (!few_plan(q.M, q.d, q.m, q.k, &f))
        return cudaErrorInvalidValue;
    int dev = 0, sms = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err == cudaSuccess)
        err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (err != cudaSuccess)
        return err;
    err = cudaFuncSetAttribute(few_gate_up_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               static_cast<int>(f.gu_smem));
    if (err == cudaSuccess)
        err = cudaFuncSetAttribute(few_down_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   static_cast<int>(f.dn_smem));
    if (err != cudaSuccess)
        return err;
    FewArgs a{};
    a.x = q.x;
    a.logits = q.logits;
    a.ids = q.ids;
    a.w = q.w;
    a.gu_q = q.gu_q;
    a.gu_s = q.gu_s;
    a.gu_z = q.gu_z;
    a.dn_q = q.dn_q;
    a.dn_s = q.dn_s;
    a.dn_z = q.dn_z;
    a.h = q.h;
    a.out = q.out;
    a.dev_status = q.dev_status;
    a.wait_ns = pipeline_test_hooks().wait_ns;
    a.M = q.M;
    a.d = q.d;
    a.m = q.m;
    a.E = q.E;
    a.k = q.k;
    a.slots = f.slots;
    a.slot_bytes = f.slot_bytes;
    a.x_stride = f.x_stride;
    a.dn_slots = f.dn_slots;
    err = launch_pdl(few_gate_up_kernel, dim3(sms), dim3(kGuThreads), f.gu_smem, stream, a);
    if (err != cudaSuccess)
        return err;
    a.routed = a.logits != nullptr;
    a.logits = nullptr;
    return launch_pdl(few_down_kernel, dim3(q.d / kDnRows), dim3(kDnThreads), f.dn_smem, stream, a);
}

}  // namespace w4
