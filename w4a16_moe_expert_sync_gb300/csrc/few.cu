// few.cu -- the whole routed-expert layer for a few tokens, in one kernel:
//   gate_up: h[a] = gelu_tanh(x_t . deq(Wg[e])^T) * (x_t . deq(Wu[e])^T)
//   down:    y[a] = h[a] . deq(Wd[e])^T
//   combine: out_t = sum_j w_j y[t k + j], j in order
// with a grid barrier between the steps (a cooperative launch, one CTA per SM).
//
// With a few tokens an expert sees one or two of them, so the layer is the
// stream of the touched experts' packed weights and every weight is used
// once or twice: a tensor-memory pipeline with 128-row tiles would spend its
// time on hand-overs.  Here a warp-level fp16 MMA (16 weight rows x 8 tokens
// x 16) takes the codes themselves: a nibble masked in place is the fp16
// subnormal q 2^-24 (low nibble of a byte) or 16 q 2^-24 (high nibble), both
// exact, and so is its product with an fp16 activation.  The group's scale
// and zero are applied to the fp32 sums,
//     sum_k s (q_k - z) x_k = s (2^24 (lo + hi / 16) - z sum_k x_k),
// so no weight is rounded at all.  The contraction order inside a group is
// free as long as codes and activations agree on it: a lane takes 8 codes at
// a time as they lie in a word, and the activations are stored permuted.
//
// A job is one expert with up to 8 of its assignments (the MMA's columns); a
// task is a job's 16 weight rows of one MMA (gate_up: 8 gate rows and the 8 up
// rows beside them, so g and u of an intermediate end in the same lane); a
// unit is 256 codes of a task's 16 rows, one 2 KB TMA box.  A CTA takes an
// equal contiguous share of the tasks and its warps equal shares of those
// tasks' units, so the bytes are spread evenly from one token to 32; a task
// that crosses warps is added up through shared memory, in warp order.  Every
// warp streams its own units through a private ring.  The first units of down
// are requested before the grid barrier that ends gate_up.
//
// Bound by HBM.  Measured at d = 2816, m = 704, E = 128, k = 8 (GB300, back to back in
// a graph): 1 token 19.0 us (25.8 MB, 3.8 us at the copy bandwidth), 7 tokens 44 us (150
// MB, 22 us), 32 tokens 87 us (360 MB, 53 us).  Clocks of one token: routing and jobs 2.5,
// first requests 1.8, staging 1, gate_up's units 2.3 and its end 1.7, barrier 2.6, down's
// staging 1.3, units 1.3 and end 1.3, barrier 2.4, the rest launch and combine.  At 32
// tokens gate_up streams at 6.4 TB/s after 9.4 us of routing and staging, down, with twice
// the scales, at 5.0; CTAs wait 2.4 to 8 us at the first barrier, 1 to 3.5 at the second.
#include <algorithm>
#include <atomic>
#include <cooperative_groups.h>
#include <cuda_fp16.h>
#include <type_traits>

#include "../../include/w4moe.h"
#include "checks.cuh"
#include "launch.h"
#include "ptx.cuh"
#include "route_token.cuh"

namespace w4 {

namespace {

constexpr int kCols = 8;          // tokens per job: the MMA's N
constexpr int kMaxA = 256;        // assignments of a call
constexpr int kMaxM = 32;

struct FewArgs {
    CUtensorMap gu_map;                // gu_q as [2 E][m][d/2] bytes, box 2 x 8 x 128
    CUtensorMap dn_map;                // dn_q as [E][d][m/2] bytes, box 1 x 16 x 128
    const uint16_t *x;                 // [M, d] bf16
    const float *logits;               // [M, E], or NULL: ids and w are inputs
    int32_t *ids;                      // [M, k]
    float *w;                          // [M, k]
    const uint16_t *gu_s, *gu_z, *dn_s, *dn_z;
    float *h;                          // [M k, m]
    float *y;                          // [M k, d] fp32
    uint16_t *out;                     // [M, d] bf16
    int32_t *dev_status;
    uint64_t wait_ns;
    int withhold;                      // test hook: the rings' first stages never complete
    int M, d, m, E, k;                 // M <= the grid
    int scale_bytes;                   // a warp's ring of scales
    int cols;                          // activation columns that fit
};

// ------------------------------------------------------------------- jobs
constexpr int kMaxE = 1024;
constexpr int kChunks = kMaxA / 32;
// An expert's assignments among each 32; lives where the activations' columns
// come later.
using Seen = uint8_t[kChunks][kMaxE];

struct Shared {
    int n;                             // jobs
    int scaled;                        // of a pass: whether a group is scaled (see Columns)
    int warp_sum[32];
    int16_t expert[kMaxA];
    int16_t count[kMaxA];
    int16_t a[kMaxA][kCols];
    int16_t col0[kMaxA];               // of a pass: each job's first column,
    int16_t col_a[kMaxA];              // each column's assignment
    int16_t base[kMaxE];               // an expert's first job
    alignas(16) int ids[kMaxA];
};

// The k experts of one token by one warp, ties to the lower index: the same
// ids as route_token's, for a row without NaN (with NaN: some ids in [0, E)).  Floats are compared as
// integers in the same order, a round is two warp reductions.  Lane j < k
// returns the j-th choice.
template <int EPL>
__device__ __forceinline__ int top_experts(const float *__restrict__ row, int E, int k, int lane)
{
    uint32_t key[EPL];
#pragma unroll
    for (int i = 0; i < EPL; i++) {
        const int e = lane + 32 * i;
        const uint32_t u = e < E ? __float_as_uint(__ldg(row + e) + 0.0f) : 0u;   // -0 -> +0
        key[i] = e < E ? (u & 0x80000000u ? ~u : u | 0x80000000u) : 0u;
    }
    int mine = -1;
    for (int j = 0; j < k; j++) {
        uint32_t best = key[0];
        int at = 0;
#pragma unroll
        for (int i = 1; i < EPL; i++)
            if (key[i] > best) {
                best = key[i];
                at = i;
            }
        const uint32_t top = __reduce_max_sync(0xffffffffu, best);
        const int e = __reduce_min_sync(0xffffffffu, best == top ? lane + 32 * at : 0x7fffffff);
#pragma unroll
        for (int i = 0; i < EPL; i++)
            if (lane + 32 * i == e)
                key[i] = 0;
        if (lane == j)
            mine = e;
    }
    return mine;
}

// The routing in shared memory: the router for every token (one warp per
// token), or the caller's ids.
__device__ void load_routing(const FewArgs &p, Shared &s, Seen &seen)
{
    const int tid = threadIdx.x, A = p.M * p.k, nt = blockDim.x;
    for (int i = tid; i < kChunks * kMaxE / 16; i += nt)
        reinterpret_cast<int4 *>(seen)[i] = make_int4(0, 0, 0, 0);
    if (p.logits) {
        const int lane = tid & 31;
        for (int t = tid >> 5; t < p.M; t += nt >> 5) {
            const float *row = p.logits + static_cast<int64_t>(t) * p.E;
            const int e = p.E <= 128 ? top_experts<4>(row, p.E, p.k, lane)
                                     : top_experts<32>(row, p.E, p.k, lane);
            if (lane < p.k)
                s.ids[t * p.k + lane] = e;
        }
    } else {
        for (int a = tid; a < A; a += nt) {
            const int e = p.ids[a];
            const bool ok = e >= 0 && e < p.E;
            s.ids[a] = ok ? e : -1;
            if (!ok && blockIdx.x == 0 && p.dev_status)
                atomicOr(p.dev_status, kDevBadExpertId);
        }
    }
    __syncthreads();
}

// The router's results of token t, by one warp: its ids and their weights.
__device__ void publish_routing(const FewArgs &p, const Shared &s, int t, int lane)
{
    const int e = lane < p.k ? s.ids[t * p.k + lane] : 0;
    const float v = lane < p.k ? __ldg(p.logits + static_cast<int64_t>(t) * p.E + e) : 0.0f;
    const float top = __shfl_sync(0xffffffffu, v, 0);
    const float w = chosen_weight(v, top, p.k, lane);
    if (lane < p.k) {
        p.ids[t * p.k + lane] = e;
        p.w[t * p.k + lane] = w;
    }
}

// Assignments grouped into jobs, every CTA for itself and all alike: jobs in
// the order of their experts, an expert's assignments in order, 8 to a job.
// An assignment's rank among its expert's is the number of earlier lanes of
// its 32 with the same expert, plus the counts of the earlier 32s.
__device__ void build_jobs(Shared &s, Seen &seen, int A, int E)
{
    const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5;
    const int chunks = (A + 31) / 32;
    for (int c = warp; c < chunks; c += nt >> 5) {
        const int a = c * 32 + lane, e = a < A ? s.ids[a] : -1;
        const unsigned same = __match_any_sync(0xffffffffu, e);
        if (e >= 0 && lane == __ffs(same) - 1)
            seen[c][e] = static_cast<uint8_t>(__popc(same));
    }
    __syncthreads();
    // exclusive scan of the experts' job counts, a run of experts per thread
    const int run = (E + nt - 1) / nt, e0 = min(E, tid * run), e1 = min(E, e0 + run);
    int mine = 0;
    for (int e = e0; e < e1; e++) {
        int n = 0;
        for (int c = 0; c < chunks; c++)
            n += seen[c][e];
        mine += (n + kCols - 1) / kCols;
    }
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        incl += lane >= o ? v : 0;
    }
    if (lane == 31)
        s.warp_sum[warp] = incl;
    __syncthreads();
    int job = incl - mine;
    for (int w = 0; w < warp; w++)
        job += s.warp_sum[w];
    if (tid == nt - 1)
        s.n = job + mine;
    for (int e = e0; e < e1; e++) {
        int n = 0;
        for (int c = 0; c < chunks; c++)
            n += seen[c][e];
        s.base[e] = static_cast<int16_t>(job);
        for (; n > 0; n -= kCols, job++) {
            s.expert[job] = static_cast<int16_t>(e);
            s.count[job] = static_cast<int16_t>(min(n, kCols));
        }
    }
    __syncthreads();
    for (int c = warp; c < chunks; c += nt >> 5) {
        const int a = c * 32 + lane, e = a < A ? s.ids[a] : -1;
        const unsigned same = __match_any_sync(0xffffffffu, e);
        if (e >= 0) {
            int rank = __popc(same & ((1u << lane) - 1u));
            for (int i = 0; i < c; i++)
                rank += seen[i][e];
            s.a[s.base[e] + rank / kCols][rank % kCols] = static_cast<int16_t>(a);
        }
    }
    __syncthreads();
}

// --------------------------------------------------------------- MMA core
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1, const float (&c)[4])
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%10, %11, %12, %13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]),
          "f"(c[3]));
}

// Eight codes of two weight rows (one word each) against eight activations
// (x0 x4 | x2 x6 | x1 x5 | x3 x7): the low nibbles into lo, the high into hi.
__device__ __forceinline__ void mma_word(float (&lo)[4], float (&hi)[4], uint32_t w0, uint32_t w1,
                                         const uint4 &b)
{
    const uint32_t v0 = w0 >> 8, v1 = w1 >> 8;
    mma16816(lo, w0 & 0x000F000Fu, w1 & 0x000F000Fu, v0 & 0x000F000Fu, v1 & 0x000F000Fu, b.x, b.y,
             lo);
    mma16816(hi, w0 & 0x00F000F0u, w1 & 0x00F000F0u, v0 & 0x00F000F0u, v1 & 0x00F000F0u, b.z, b.w,
             hi);
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

// Saturation to fp16's finite range (NaN stays NaN).
__device__ __forceinline__ float saturated(float v)
{
    return fabsf(v) > 65504.0f ? copysignf(65504.0f, v) : v;
}

// 2^n.
__device__ __forceinline__ float power(int n)
{
    return __uint_as_float(static_cast<uint32_t>(127 + n) << 23);
}

// Two values in fp16.
__device__ __forceinline__ uint32_t half_pair(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// By how many powers of two a group is scaled up, of which `lanes` lanes side by side
// hold 4 values each: to 2^14 .. 2^15 if they are all below 2^-7, else not at all.
__device__ __noinline__ int shift_of(float a, float b, float c, float d, int lanes)
{
    float top = fmaxf(fmaxf(fabsf(a), fabsf(b)), fmaxf(fabsf(c), fabsf(d)));   // NaN does not count
    for (int o = lanes / 2; o > 0; o >>= 1)
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    return top < 0.0078125f ? min(141 - static_cast<int>(__float_as_uint(top) >> 23), 100) : 0;
}

// ----------------------------------------------------------------- streams
// One of the two contractions: gate_up (UP: groups of 128, rows r and m + r)
// or down (groups of 64, rows r and r + 8).
template <bool UP> struct Step {
    static constexpr int kGroup = UP ? 128 : 64;
    static constexpr int kWords = kGroup / 32;          // a lane's words of a row's group
    static constexpr int kUnitGroups = 256 / kGroup;
};

constexpr int kUnitBytes = 2048;                        // 16 rows x 128 bytes

__host__ __device__ constexpr int units_of(int K) { return (K + 255) / 256; }
__host__ __device__ constexpr int scale_bufs(int depth, int K)
{
    return (depth + units_of(K) - 1) / units_of(K) + 1;
}
__host__ __device__ constexpr int col_stride(int K, int G)
{
    // fp16 values, then the groups' sums and their factors (fp32); an odd multiple of 64
    // so that neighbouring columns' chunks fall in distinct banks
    return (2 * K + 8 * G + 127) / 128 * 128 + 64;
}

// The rest of a wait that its first try did not end, out of the hot loop: for stage
// `stage` of a ring whose next request goes to `ask`.  Once it has given up, by its
// limit or because another warp's has, and what the ring has under way (all of it, if
// stage is ask) has landed or had its time to, the warp is `gone`: nothing is requested
// or awaited any more.  (Votes keep it uniform: a __syncwarp at its end, or the answer
// returned, makes the caller's loop 10 KB longer and the layer 4 to 6 us slower.)
__device__ __noinline__ void wait_long(uint64_t *full, int stage, int ask, uint32_t phase,
                                       int depth, volatile int *gone, volatile int *abort_flag,
                                       int32_t *status, uint64_t limit_ns)
{
    if (__any_sync(0xffffffffu, *gone != 0))
        return;
    if (mbar_wait_warp(full + stage, phase, abort_flag, status, kDevPipelineTimeout, limit_ns))
        return;
    const uint64_t t0 = global_timer_ns();
    for (int n = ask > stage ? ask - stage : ask - stage + depth; n > 0; n--) {
        while (!__all_sync(0xffffffffu, mbar_try_wait(full + stage, phase)))
            if (__any_sync(0xffffffffu, global_timer_ns() - t0 > 200000000ull))
                break;
        if (++stage == depth) {
            stage = 0;
            phase ^= 1;
        }
    }
    *gone = 1;
}

// NW warps, each with a ring of DEPTH units.
template <int NW, int DEPTH>
struct Layer {
    static constexpr int kRingBytes = DEPTH * kUnitBytes;

    struct Mem {
        alignas(8) uint64_t full[NW][DEPTH];
        int abort_flag;
        int gone[NW];                          // see wait_long
        int head_task[NW];
        alignas(16) float head[NW][32][4];
    };

    // A warp's place in its ring; it runs on through both steps.
    struct Ring {
        uint8_t *buf;
        uint64_t *full;
        int ask_stage, stage;
        uint32_t phase;
    };

    // Requests unit `unit` of a task into the ring's next stage (and, with a
    // task's first unit in this warp's share, the task's scales and zeros:
    // 8 rows of them are 16 G contiguous bytes).  One lane.
    template <bool UP>
    static __device__ __forceinline__ void request(const FewArgs &p, int e, int tile, int unit,
                                                   bool first, uint8_t *stage, uint64_t *bar,
                                                   uint8_t *scales)
    {
        const int K = UP ? p.d : p.m, G = K / Step<UP>::kGroup;
        mbar_arrive_expect_tx(bar, kUnitBytes + (first ? 64 * G : 0));
        tma_load_3d(stage, UP ? &p.gu_map : &p.dn_map, unit * 128, tile * (UP ? 8 : 16),
                    UP ? 2 * e : e, bar);
        if (first) {
            const uint16_t *sc = UP ? p.gu_s : p.dn_s, *zp = UP ? p.gu_z : p.dn_z;
            const int64_t r0 = UP ? static_cast<int64_t>(e) * 2 * p.m + tile * 8
                                  : static_cast<int64_t>(e) * p.d + tile * 16;
            const int64_t r1 = r0 + p.m;
            if constexpr (UP) {
                bulk_load_nohint(scales, sc + r0 * G, 16 * G, bar);
                bulk_load_nohint(scales + 16 * G, sc + r1 * G, 16 * G, bar);
                bulk_load_nohint(scales + 32 * G, zp + r0 * G, 16 * G, bar);
                bulk_load_nohint(scales + 48 * G, zp + r1 * G, 16 * G, bar);
            } else {                       // rows r0 .. r0 + 15 are one block
                bulk_load_nohint(scales, sc + r0 * G, 32 * G, bar);
                bulk_load_nohint(scales + 32 * G, zp + r0 * G, 32 * G, bar);
            }
        }
    }

    // A finished task's sums, times 2^-24: acc[0..1] weight row `row` (gate), acc[2..3]
    // row + 8 (up) of columns 2 t4 and 2 t4 + 1.
    template <bool UP>
    static __device__ __forceinline__ void finish(const FewArgs &p, const Shared &s, int task,
                                                  const float (&acc)[4], int row, int t4)
    {
        const int per_job = UP ? p.m / 8 : p.d / 16;
        const int job = task / per_job, tile = task - job * per_job;
#pragma unroll
        for (int c = 0; c < 2; c++) {
            if (2 * t4 + c >= s.count[job])
                continue;
            const int64_t a = s.a[job][2 * t4 + c];
            if constexpr (UP) {
                const float hv = gelu_tanh_f(acc[c] * kSub) * (acc[2 + c] * kSub);
                if (!(fabsf(hv) <= 65504.0f) && p.dev_status)
                    atomicOr(p.dev_status, kDevFp16Range);
                if (W4_IN_BOUNDS(a < p.M * p.k && tile * 8 + row < p.m, p.dev_status))
                    p.h[a * p.m + tile * 8 + row] = saturated(hv);
            } else {
                if (!W4_IN_BOUNDS(a < p.M * p.k && tile * 16 + row + 8 < p.d, p.dev_status))
                    continue;
                float *y = p.y + a * p.d + tile * 16 + row;
                y[0] = acc[c] * kSub;
                y[8] = acc[2 + c] * kSub;
            }
        }
    }

    // The activations of a pass's columns, fp16 in the MMA's order, and their
    // groups' sums times -2^-24.  A group whose values are all below 2^-7 is scaled up
    // by a power of two before it is rounded, so that it keeps fp16's 11 bits and h,
    // which goes with the square of x, does not vanish; the inverse is its factor.  (In
    // other groups what fp16 lacks is at most 2^-18 of the largest.)  Passes without such
    // a group run a loop that knows no factors: 32 tokens 89 us, 97 where every group
    // is small, 91 to 92 with the factors in one loop for all.
    // A warp takes one column's 128 elements at a time, kBatch of them per call: load
    // reads them, put stores them.
    template <bool UP> struct Columns {
        using T = Step<UP>;
        // (1, 7 and 32 tokens: 18.4, 45.5 and 88.8 us; 4 and 4: 19.1, 46.1, 89.1)
        static constexpr int kBatch = UP ? 3 : 2;
        const FewArgs &p;
        Shared &s;
        uint8_t *xbuf;
        int items, blocks, warp, lane;
        std::conditional_t<UP, uint2, float4> v[kBatch];

        __device__ __forceinline__ Columns(const FewArgs &p_, Shared &s_, uint8_t *xbuf_,
                                           int cols, int warp_, int lane_)
            : p(p_), s(s_), xbuf(xbuf_), warp(warp_), lane(lane_)
        {
            blocks = ((UP ? p.d : p.m) + 127) / 128;
            items = cols * blocks;
        }
        __device__ __forceinline__ bool more(int batch) const
        {
            return warp + batch * kBatch * NW < items;
        }
        __device__ __forceinline__ void load(int batch)
        {
            const int K = UP ? p.d : p.m;
#pragma unroll
            for (int u = 0; u < kBatch; u++) {
                const int c = warp + (batch * kBatch + u) * NW, col = c / blocks;
                const int el = (c - col * blocks) * 128 + lane * 4;
                v[u] = {};
                if (c < items && el < K) {
                    const int64_t a = s.col_a[col];
                    if constexpr (UP)
                        v[u] = __ldcg(reinterpret_cast<const uint2 *>(p.x + a / p.k * p.d + el));
                    else
                        v[u] = __ldcg(reinterpret_cast<const float4 *>(p.h + a * p.m + el));
                }
            }
        }
        __device__ __forceinline__ void put(int batch) const
        {
            const int K = UP ? p.d : p.m, stride = col_stride(K, K / T::kGroup);
            bool range = false;
#pragma unroll
            for (int u = 0; u < kBatch; u++) {
                const int c = warp + (batch * kBatch + u) * NW, col = c / blocks;
                const int el = (c - col * blocks) * 128 + lane * 4;
                const bool in = c < items && el < K;
                uint8_t *xc = xbuf + col * stride;
                const int gi = el / T::kGroup, i8 = (el % T::kGroup) / 8;   // word in the group
                uint16_t *dst = reinterpret_cast<uint16_t *>(
                    xc + gi * T::kGroup * 2 + (i8 % T::kWords) * 64 + (i8 / T::kWords) * 16);
                float f[4];
                if constexpr (UP) {
                    f[0] = __uint_as_float(v[u].x << 16);
                    f[1] = __uint_as_float(v[u].x & 0xFFFF0000u);
                    f[2] = __uint_as_float(v[u].y << 16);
                    f[3] = __uint_as_float(v[u].y & 0xFFFF0000u);
                } else {
                    f[0] = v[u].x;
                    f[1] = v[u].y;
                    f[2] = v[u].z;
                    f[3] = v[u].w;
                }
                if constexpr (UP) {
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        range |= !(fabsf(f[i]) <= 65504.0f);
                        f[i] = saturated(f[i]);
                    }
                }
                uint32_t h01 = half_pair(f[0], f[1]), h23 = half_pair(f[2], f[3]);
                int up = 0;
                // an exponent field from 8 on: 2^-7 at least
                const unsigned large =
                    __ballot_sync(0xffffffffu, ((h01 | h23) & 0x60006000u) != 0 || !in);
                if (UP ? large == 0 : (large & 0xFFFFu) == 0 || large >> 16 == 0) {
                    up = shift_of(f[0], f[1], f[2], f[3], T::kGroup / 4);
                    h01 = half_pair(f[0] * power(up), f[1] * power(up));
                    h23 = half_pair(f[2] * power(up), f[3] * power(up));
                    s.scaled = 1;
                }
                float sum = 0.0f;
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const uint32_t bits = i < 2 ? h01 : h23;
                    const uint16_t hb = static_cast<uint16_t>(i & 1 ? bits >> 16 : bits);
                    sum += __half2float(__ushort_as_half(hb));
                    if (in)
                        dst[perm8((lane & 1) * 4 + i)] = hb;
                }
#pragma unroll
                for (int o = T::kGroup / 8; o > 0; o >>= 1)
                    sum += __shfl_xor_sync(0xffffffffu, sum, o);
                if (in && (lane & (T::kGroup / 4 - 1)) == 0) {
                    float *t = reinterpret_cast<float *>(xc + 2 * K) + gi;
                    t[0] = -sum / kSub;
                    t[K / T::kGroup] = power(-up);
                }
            }
            if (range && p.dev_status)
                atomicOr(p.dev_status, kDevFp16Range);
        }
    };

    // Adds group j of a unit to a lane's sums: codes at st + code0, activations at xc,
    // sums (and, G further, factors) of its two columns, scales and zeros at sc.
    template <bool UP, bool SCALED>
    static __device__ __forceinline__ void add_group(const uint8_t *st, int code0,
                                                     const uint8_t *xc, const float *sum0,
                                                     const float *sum1, const uint16_t *sc, int G,
                                                     int j, float (&acc)[4])
    {
        using T = Step<UP>;
        uint32_t q0[T::kWords], q1[T::kWords];
        if constexpr (UP) {
            const uint8_t *c = st + (code0 ^ (64 * j));
            *reinterpret_cast<uint4 *>(q0) = *reinterpret_cast<const uint4 *>(c);
            *reinterpret_cast<uint4 *>(q1) = *reinterpret_cast<const uint4 *>(c + 1024);
        } else {
            const uint8_t *c = st + (code0 ^ (32 * j));
            *reinterpret_cast<uint2 *>(q0) = *reinterpret_cast<const uint2 *>(c);
            *reinterpret_cast<uint2 *>(q1) = *reinterpret_cast<const uint2 *>(c + 1024);
        }
        const uint4 *b = reinterpret_cast<const uint4 *>(xc + j * T::kGroup * 2);
        float lo[4] = {}, hi[4] = {};
#pragma unroll
        for (int w = 0; w < T::kWords; w++)
            mma_word(lo, hi, q0[w], q1[w], b[4 * w]);
        // 2^-24 of the sum: acc += s (lo + hi / 16 - z 2^-24 sum)
        const float s0 = half_bits(sc + j), s1 = half_bits(sc + 8 * G + j);
        const float z0 = half_bits(sc + 16 * G + j), z1 = half_bits(sc + 24 * G + j);
        const float a0 = sum0[j], a1 = sum1[j];
        // s times a factor, a power of two, is exact
        const float f0 = SCALED ? sum0[G + j] : 1.0f, f1 = SCALED ? sum1[G + j] : 1.0f;
        acc[0] = fmaf(s0 * f0, fmaf(z0, a0, fmaf(hi[0], 0.0625f, lo[0])), acc[0]);
        acc[1] = fmaf(s0 * f1, fmaf(z0, a1, fmaf(hi[1], 0.0625f, lo[1])), acc[1]);
        acc[2] = fmaf(s1 * f0, fmaf(z1, a0, fmaf(hi[2], 0.0625f, lo[2])), acc[2]);
        acc[3] = fmaf(s1 * f1, fmaf(z1, a1, fmaf(hi[3], 0.0625f, lo[3])), acc[3]);
    }

    // The CTA's share of a step.  `between` runs once, after the first
    // requests are on their way; down's activations are read after it, gate_up's
    // first ones before the requests.
    template <bool UP, class F>
    static __device__ __forceinline__ void run(const FewArgs &p, Shared &s, Mem &mem, Ring &ring,
                                               uint8_t *scales, uint8_t *xbuf, F between)
    {
        using T = Step<UP>;
        const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
        const int K = UP ? p.d : p.m, G = K / T::kGroup, stride = col_stride(K, G);
        const int per_task = units_of(K), nbuf = scale_bufs(DEPTH, K);
        const int per_job = UP ? p.m / 8 : p.d / 16;
        // at most 256 jobs of 512 tasks of 32 units: 32 bits hold their products
        // with the grid and with the warps
        const uint32_t total = static_cast<uint32_t>(s.n) * per_job;
        const int t0 = static_cast<int>(total * blockIdx.x / gridDim.x);
        const int t1 = static_cast<int>(total * (blockIdx.x + 1) / gridDim.x);
        const int t4 = lane & 3, g = lane >> 2;
        // The weight row of this lane's MMA row g: g with its bits reversed,
        // so that the lanes of one shared-memory phase read distinct banks of
        // the 128-byte-swizzled box (rows 0 4 | 2 6 | 1 5 | 3 7).
        const int row = ((g & 1) << 2) | (g & 2) | (g >> 2);
        const int code0 = UP ? row * 128 + ((t4 ^ row) * 16)
                             : row * 128 + (((t4 >> 1) ^ row) * 16) + (t4 & 1) * 8;
        // A warp that is gone goes on without copies or waits and meets the others at
        // their barriers; what it stores is in its place, and worth nothing.
        volatile int *gone = &mem.gone[warp];
        bool first_pass = true;

        for (int p0 = t0; p0 < t1 || first_pass;) {
            // the jobs whose columns fit together (one pass, unless many
            // tokens share few experts)
            if (threadIdx.x == 0)
                s.scaled = 0;
            const int job0 = p0 / per_job;
            int job1 = job0, cols = 0;
            while (p0 < t1 && job1 * per_job < t1 && cols + s.count[job1] <= p.cols) {
                const int n = s.count[job1];
                if (threadIdx.x == 0)
                    s.col0[job1] = static_cast<int16_t>(cols);
                if (threadIdx.x < n)
                    s.col_a[cols + threadIdx.x] = s.a[job1][threadIdx.x];
                cols += n;
                job1++;
            }
            const int p1 = min(t1, max(p0, job1 * per_job));
            const uint32_t units = static_cast<uint32_t>(p1 - p0) * per_task;
            const int u0 = static_cast<int>(units * warp / NW);
            const int u1 = static_cast<int>(units * (warp + 1) / NW);

            int task = p0 + u0 / per_task, unit = u0 % per_task;
            // the next request: job, tile of its rows, unit, scale buffer
            int rj = min(task / per_job, max(s.n - 1, 0)), rt = task - rj * per_job;
            int rb = unit, rn = 0, left = u1 - u0;
            int re = s.expert[rj];
            auto ask = [&]() {                 // one lane asks; all keep count
                if (left > 0) {
                    if (lane == 0 && !*gone)
                        request<UP>(p, re, rt, rb, left == u1 - u0 || rb == 0,
                                    ring.buf + ring.ask_stage * kUnitBytes,
                                    ring.full + ring.ask_stage, scales + rn * 64 * G);
                    left--;
                    ring.ask_stage = ring.ask_stage + 1 == DEPTH ? 0 : ring.ask_stage + 1;
                    if (++rb == per_task) {
                        rb = 0;
                        rn = rn + 1 == nbuf ? 0 : rn + 1;
                        if (++rt == per_job) {
                            rt = 0;
                            rj = min(rj + 1, s.n - 1);
                            re = s.expert[rj];
                        }
                    }
                }
            };
            Columns<UP> columns(p, s, xbuf, cols, warp, lane);
            if constexpr (UP) {
                __syncthreads();               // col0 and col_a
                columns.load(0);
            }
#pragma unroll 1
            for (int i = 0; i < DEPTH; i++)
                ask();
            if (first_pass)
                between();
            if constexpr (!UP) {
                if (!first_pass)
                    __syncthreads();           // `between` has synchronised the CTA
                columns.load(0);
            }
            first_pass = false;
            columns.put(0);
#pragma unroll 1
            for (int b = 1; columns.more(b); b++) {
                columns.load(b);
                columns.put(b);
            }
            if (lane == 0)
                mem.head_task[warp] = -1;
            __syncthreads();

            int sn = 0;
            bool begun = unit == 0;            // this warp holds the task's first unit
            float acc[4] = {};
            auto consume = [&](auto scaled) {
                for (int u = u0; u < u1;) {
                    const int job = task / per_job, n = s.count[job];
                    const uint8_t *xj = xbuf + s.col0[job] * stride;
                    const uint8_t *xc = xj + (g < n ? g : 0) * stride + t4 * 16 + unit * 512;
                    const int first_group = unit * T::kUnitGroups;
                    const float *sum0 = reinterpret_cast<const float *>(
                        xj + (2 * t4 < n ? 2 * t4 : 0) * stride + 2 * K) + first_group;
                    const float *sum1 = reinterpret_cast<const float *>(
                        xj + (2 * t4 + 1 < n ? 2 * t4 + 1 : 0) * stride + 2 * K) + first_group;
                    const uint16_t *sc = reinterpret_cast<const uint16_t *>(scales + sn * 64 * G) +
                                         row * G + first_group;
                    const int end = min(per_task, unit + u1 - u);
                    u += end - unit;
                    int groups = G - first_group;              // left in the task
                    for (; unit < end; unit++) {
                        const uint32_t bar = smem_u32(ring.full + ring.stage);
                        if (!__all_sync(0xffffffffu, mbar_try_wait_a(bar, ring.phase)))
                            wait_long(ring.full, ring.stage, ring.ask_stage, ring.phase, DEPTH,
                                      gone, &mem.abort_flag, p.dev_status, p.wait_ns);
                        const uint8_t *st = ring.buf + ring.stage * kUnitBytes;
                        auto group = [&](int j) {
                            add_group<UP, scaled>(st, code0, xc, sum0, sum1, sc, G, j, acc);
                        };
                        // whole units without a branch between their groups, so that
                        // the groups' loads and MMAs overlap
                        if (groups >= T::kUnitGroups) {
#pragma unroll
                            for (int j = 0; j < T::kUnitGroups; j++)
                                group(j);
                        } else {
#pragma unroll 1
                            for (int j = 0; j < groups; j++)
                                group(j);
                        }
                        groups -= T::kUnitGroups;
                        xc += 512;
                        sum0 += T::kUnitGroups;
                        sum1 += T::kUnitGroups;
                        sc += T::kUnitGroups;
                        if (++ring.stage == DEPTH) {
                            ring.stage = 0;
                            ring.phase ^= 1;
                        }
                        __syncwarp();
                        ask();
                    }
                    if (unit == per_task) {
                        if (begun)
                            finish<UP>(p, s, task, acc, row, t4);
                        else {                     // begun by an earlier warp
                            *reinterpret_cast<float4 *>(mem.head[warp][lane]) =
                                make_float4(acc[0], acc[1], acc[2], acc[3]);
                            if (lane == 0)
                                mem.head_task[warp] = task;
                        }
                        unit = 0;
                        task++;
                        begun = true;
                        sn = sn + 1 == nbuf ? 0 : sn + 1;
                        acc[0] = acc[1] = acc[2] = acc[3] = 0.0f;
                    }
                }
            };
            if (s.scaled)
                consume(std::true_type{});
            else
                consume(std::false_type{});
            const bool open = u0 < u1 && unit != 0;    // the last task goes on in a later warp
            if (open && !begun) {                      // and began in an earlier one
                *reinterpret_cast<float4 *>(mem.head[warp][lane]) =
                    make_float4(acc[0], acc[1], acc[2], acc[3]);
                if (lane == 0)
                    mem.head_task[warp] = task;
            }
            __syncthreads();
            if (open && begun) {
                for (int w = warp + 1; w < NW; w++) {
                    if (mem.head_task[w] == task) {
                        const float4 v = *reinterpret_cast<const float4 *>(mem.head[w][lane]);
                        acc[0] += v.x;
                        acc[1] += v.y;
                        acc[2] += v.z;
                        acc[3] += v.w;
                    }
                }
                finish<UP>(p, s, task, acc, row, t4);
            }
            if (p1 >= t1)
                break;
            __syncthreads();
            p0 = p1;
        }
    }
};

template <int NW, int DEPTH>
__global__ void __launch_bounds__(32 * NW, 1) few_layer_kernel(const __grid_constant__ FewArgs p)
{
    using L = Layer<NW, DEPTH>;
    extern __shared__ __align__(1024) uint8_t raw[];
    __shared__ Shared s;
    __shared__ typename L::Mem mem;
    // the boxes' swizzle goes by address: 1024-byte aligned
    uint8_t *dyn = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    const int warp = threadIdx.x >> 5;
    typename L::Ring ring = {dyn + warp * L::kRingBytes, mem.full[warp], 0, 0, 0};
    if (threadIdx.x == 0) {
        for (int i = 0; i < NW * DEPTH; i++)
            mbar_init(&mem.full[0][0] + i, p.withhold && i % DEPTH == 0 ? 2 : 1);
        mem.abort_flag = 0;
        for (int i = 0; i < NW; i++)
            mem.gone[i] = 0;
        fence_mbar_init();
        prefetch_tmap(&p.gu_map);
        prefetch_tmap(&p.dn_map);
    }
    uint8_t *scales = dyn + NW * L::kRingBytes + warp * p.scale_bytes;
    uint8_t *xbuf = dyn + NW * (L::kRingBytes + p.scale_bytes);
    auto grid = cooperative_groups::this_grid();

    Seen &seen = *reinterpret_cast<Seen *>(xbuf);
    load_routing(p, s, seen);
    build_jobs(s, seen, p.M * p.k, p.E);
    L::template run<true>(p, s, mem, ring, scales, xbuf, [&] {
        // the weights, which only the combine needs, while the first bytes are on their way
        if (p.logits && blockIdx.x < p.M && warp == NW - 1)
            publish_routing(p, s, blockIdx.x, threadIdx.x & 31);
    });
    L::template run<false>(p, s, mem, ring, scales, xbuf, [&] { grid.sync(); });
    grid.sync();
    const int d4 = p.d / 4;
    for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < p.M * d4; i += gridDim.x * blockDim.x) {
        const int t = i / d4, c = (i - t * d4) * 4;
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int j = 0; j < p.k; j++) {
            const int a = t * p.k + j;
            if (s.ids[a] < 0)
                continue;
            const float4 y = __ldcg(reinterpret_cast<const float4 *>(
                p.y + static_cast<int64_t>(a) * p.d + c));
            const float w = __ldcg(p.w + a);
            v.x = fmaf(w, y.x, v.x);
            v.y = fmaf(w, y.y, v.y);
            v.z = fmaf(w, y.z, v.z);
            v.w = fmaf(w, y.w, v.w);
        }
        uint2 o;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o.x) : "f"(v.y), "f"(v.x));
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o.y) : "f"(v.w), "f"(v.z));
        *reinterpret_cast<uint2 *>(p.out + static_cast<int64_t>(t) * p.d + c) = o;
    }
}

// Shared memory of a variant for a shape: the scales' rings and the columns
// that fit beside them.  Needs room for one full job.
template <int NW, int DEPTH>
bool plan(int d, int m, int *scale_bytes, int *cols, size_t *smem)
{
    *scale_bytes = *cols = 0;
    *smem = 0;
    if (d > 65536 || m > 65536)        // no column of these fits, and 32 bits hold the rest
        return false;
    const int Gu = d / 128, Gd = m / 64;
    *scale_bytes = 64 * std::max(scale_bufs(DEPTH, d) * Gu, scale_bufs(DEPTH, m) * Gd);
    // the static arrays, up to the dynamic part's alignment
    const int stat =
        (sizeof(Shared) + sizeof(typename Layer<NW, DEPTH>::Mem) + 64 + 1023) / 1024 * 1024;
    const int rings = 1024 + NW * (DEPTH * kUnitBytes + *scale_bytes);
    const int room = 227 * 1024 - stat - rings;
    const int stride = std::max(col_stride(d, Gu), col_stride(m, Gd));
    *cols = room < 0 ? 0 : std::min(room / stride, kMaxA);
    *smem = static_cast<size_t>(rings) + static_cast<size_t>(*cols) * stride;
    return *cols >= kCols && *cols * stride >= static_cast<int>(sizeof(Seen));
}

template <int NW, int DEPTH>
cudaError_t launch_variant(FewArgs a, int dev, int sms, cudaStream_t stream)
{
    size_t smem;
    if (!plan<NW, DEPTH>(a.d, a.m, &a.scale_bytes, &a.cols, &smem))
        return cudaErrorInvalidValue;
    auto kern = few_layer_kernel<NW, DEPTH>;
    static std::atomic<uint64_t> raised{0};      // devices whose limit is raised already
    if (!(raised.load(std::memory_order_relaxed) >> (dev & 63) & 1u)) {
        cudaFuncAttributes at;
        cudaError_t err = cudaFuncGetAttributes(&at, kern);
        if (err == cudaSuccess)
            err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       227 * 1024 - static_cast<int>(at.sharedSizeBytes));
        if (err != cudaSuccess)
            return err;
        raised.fetch_or(1ull << (dev & 63), std::memory_order_relaxed);
    }
    void *args[] = {&a};
    return cudaLaunchCooperativeKernel(kern, dim3(sms), dim3(32 * NW), args, smem, stream);
}

// Sixteen warps with two units each in flight where the scales' rings and a
// job's columns leave room for it, else eight warps with three.  (At d = 2816, m = 704,
// sixteen and eight: 1 token 18.6 and 18.6 us, 7 tokens 45.4 and 54.8, 32 tokens 89 and
// 117.)
bool wide_fits(int d, int m)
{
    int sb, cols;
    size_t smem;
    return plan<16, 2>(d, m, &sb, &cols, &smem);
}

using EncodeFn = decltype(&cuTensorMapEncodeTiled);

EncodeFn encode_fn()
{
    static EncodeFn fn = [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000,
                                             cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            ptr = nullptr;
        return reinterpret_cast<EncodeFn>(ptr);
    }();
    return fn;
}

// Packed rows as [outer][rows][row_bytes], boxes of 128 bytes x 16 rows in
// all, 128-byte swizzle; what lies past a row's end reads as zero.
bool encode_rows(CUtensorMap *map, const uint8_t *base, int row_bytes, int rows, int outer,
                 int box_rows, int box_outer)
{
    const cuuint64_t dim[3] = {static_cast<cuuint64_t>(row_bytes), static_cast<cuuint64_t>(rows),
                               static_cast<cuuint64_t>(outer)};
    const cuuint64_t stride[2] = {dim[0], dim[0] * dim[1]};
    const cuuint32_t box[3] = {128, static_cast<cuuint32_t>(box_rows),
                               static_cast<cuuint32_t>(box_outer)};
    const cuuint32_t step[3] = {1, 1, 1};
    return encode_fn()(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t *>(base), dim,
                       stride, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                       CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

size_t h_bytes(int M, int m, int k)
{
    return (static_cast<size_t>(M) * k * m * 4 + 255) / 256 * 256;
}

}  // namespace

bool few_supported(int M, int d, int m, int k)
{
    int sb, cols;
    size_t smem;
    return M <= kMaxM && M * k <= kMaxA && (wide_fits(d, m) || plan<8, 3>(d, m, &sb, &cols, &smem));
}

size_t few_workspace_bytes(int M, int d, int m, int k)
{
    return h_bytes(M, m, k) + static_cast<size_t>(M) * k * d * 4;
}

cudaError_t launch_few(const FewProblem &q, cudaStream_t stream)
{
    int dev = 0, sms = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err == cudaSuccess)
        err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (err != cudaSuccess)
        return err;
    FewArgs a{};
    a.x = q.x;
    a.logits = q.logits;
    a.ids = q.ids;
    a.w = q.w;
    a.gu_s = q.gu_s;
    a.gu_z = q.gu_z;
    a.dn_s = q.dn_s;
    a.dn_z = q.dn_z;
    a.h = static_cast<float *>(q.workspace);
    a.y = reinterpret_cast<float *>(static_cast<uint8_t *>(q.workspace) + h_bytes(q.M, q.m, q.k));
    a.out = q.out;
    a.dev_status = q.dev_status;
    a.wait_ns = pipeline_test_hooks().wait_ns;
    a.withhold = pipeline_test_hooks().withhold_sz;
    a.M = q.M;
    a.d = q.d;
    a.m = q.m;
    a.E = q.E;
    a.k = q.k;
    if (!encode_fn())
        return cudaErrorNotSupported;
    if (!encode_rows(&a.gu_map, q.gu_q, q.d / 2, q.m, 2 * q.E, 8, 2) ||
        !encode_rows(&a.dn_map, q.dn_q, q.m / 2, q.d, q.E, 16, 1))
        return cudaErrorInvalidValue;
    return wide_fits(q.d, q.m) ? launch_variant<16, 2>(a, dev, sms, stream)
                               : launch_variant<8, 3>(a, dev, sms, stream);
}

}  // namespace w4
