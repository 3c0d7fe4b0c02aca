// linear_few_wide.cu -- the W4A16 linear for 9 to 32 tokens and many rows, on tcgen05:
//   y[t, n] = sum_g s[n, g] (sum_{k in g} q[n, k] x[t, k] - z[n, g] sum_{k in g} x[t, k])
// for groups of 128, or of 64 by twos.  linear_few.cu is the plain form of it; beyond 8 tokens its warps'
// MMAs and the unpacking of the codes for them take longer than the weights' way from HBM.
//
// A nibble is the e4m3 number q 2^-9, subnormals included, so a word of eight codes is two
// words of MMA operand for two ANDs and a shift: A, 128 weight rows in tensor memory.  B is
// the activations as e4m3 pairs x 2^e = P1 + P2 / 32, e for each token and group of 128 such
// that the largest lies in [2^7, 2^8): 4 bits each, which is all of a bf16 value down to 2^-13
// of the group's largest; what smaller ones lose is below 2^-22 of the largest.  P1 and P2
// are columns of one MMA (kind::f8f6f4, M 128, N twice the tokens), each group's sums
// have accumulators of their own, and a thread, which holds a weight row, adds
//   s (2^(9 - e) (D1 + D2 / 32) - z sum x)
// to its 32-bit sums, token by token.
//
// A CTA takes 128 rows at a time, its groups in turn by two sets of warps: four that unpack (a
// warp per 32 rows), one that issues the MMAs, four that add the sums up.  The sets' sums of a
// task meet in tensor memory, in a fixed order: bit-identical reruns.  Codes arrive by TMA, up
// to 16 groups ahead.
//
// Measured on GB300, 2816 -> 262144: 16 tokens 68 us, 32 tokens 94 (393 and 409 MB, 58 and
// 60 us at the copy bandwidth).  With 32 tokens the activations leave room for four groups
// only, whose round trip takes 86 us with all arithmetic taken out (with 16 tokens 63), and the
// roles' steps, each a chain of waits, take 0.34 us a group whatever the slots; asking for the
// codes in L2 ahead changes nothing.  Others, 32 tokens, step by step: one warp for unpacking and
// adding up 150, a division by the slots or groups in each role's step 142, a thread adds up one
// row of all tokens 107, the adding loop unrolled four times 99, activations laid out 8 values a
// lane instead of 16 97; a fifth slot 1 to 2 less, but for what it takes to tell the slot's turns
// 83 with 16 tokens instead of 73; two CTAs with half of the groups each, sums joined through the
// other's shared memory 162.
#include <algorithm>
#include <atomic>
#include <cuda_fp16.h>

#include "../../include/w4moe.h"
#include "checks.cuh"
#include "launch.h"
#include "ptx.cuh"

namespace w4 {

namespace {

constexpr int kRows = 128;                 // of a task
constexpr int kGroup = 128;                // codes of a step: one group, or two of 64
constexpr int kSlotBytes = kRows * kGroup / 2;
// first warps of the roles behind the eight that unpack
constexpr int kAdd = 8, kIssue = 16, kLoad = 18;
constexpr int kMaxSlots = 16;
constexpr int kMaxSmem = 227 * 1024;

struct WideArgs {
    CUtensorMap map;                       // codes [N][K / 2] bytes, box 64 x 128
    const uint16_t *x;                     // [M, K] bf16
    const uint16_t *s, *z;                 // [N, K / group] fp16
    uint16_t *y;                           // [M, N] bf16
    int32_t *dev_status;
    uint64_t wait_ns;
    int withhold;                          // test hook: the first slot never completes
    int M, K, N, groups, slots;
};

__device__ __forceinline__ uint64_t pair_of(float lo, float hi)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float low(uint64_t x) { return __uint_as_float(static_cast<uint32_t>(x)); }
__device__ __forceinline__ float high(uint64_t x)
{
    return __uint_as_float(static_cast<uint32_t>(x >> 32));
}

// Two values in e4m3 (the first in the lower byte), and back.
__device__ __forceinline__ uint32_t to_e4m3(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float2 from_e4m3(uint32_t v)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(v)));
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// A scale or zero.  Non-coherent, so that a row's neighbouring ones stay in L1 across the
// fences (coherent loads: 32 tokens, 2816 -> 262144, 217 us instead of 107); volatile, so
// that none moves before the wait for the kernel that may have written them.
__device__ __forceinline__ uint16_t load_weight(const uint16_t *at)
{
    uint16_t v;
    asm volatile("ld.global.nc.u16 %0, [%1];" : "=h"(v) : "l"(at));
    return v;
}

// One group: four steps of 32 codes, A in tensor memory (8 columns a step), by one elected
// lane; the sums begin anew.
__device__ __forceinline__ void mma_group(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc)
{
    asm volatile(
        "{\n\t.reg .pred p, f, e;\n\t.reg .b64 y;\n\t.reg .b32 x;\n\t"
        "setp.eq.b32 p, 0, 0;\n\tsetp.ne.b32 f, 0, 0;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, f;\n\t"
        "add.s32 x, %1, 8;\n\tadd.s64 y, %2, 2;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [x], y, %3, p;\n\t"
        "add.s32 x, %1, 16;\n\tadd.s64 y, %2, 4;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [x], y, %3, p;\n\t"
        "add.s32 x, %1, 24;\n\tadd.s64 y, %2, 6;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [x], y, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc)
        : "memory");
}

// Half of that, for a group of 64.
__device__ __forceinline__ void mma_half(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc)
{
    asm volatile(
        "{\n\t.reg .pred p, f, e;\n\t.reg .b64 y;\n\t.reg .b32 x;\n\t"
        "setp.eq.b32 p, 0, 0;\n\tsetp.ne.b32 f, 0, 0;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, f;\n\t"
        "add.s32 x, %1, 8;\n\tadd.s64 y, %2, 2;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [x], y, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc)
        : "memory");
}

// TOK: tokens, 16 or 32 (of groups of 64: 16, for two groups' sums a step take the columns of
// 32 tokens).
template <int TOK, int GROUP> struct Wide {
    static_assert(TOK == 16 || GROUP == 128);
    static constexpr int kSub = kGroup / GROUP;            // groups of a step
    static constexpr int kN = 2 * TOK;
    // With 32 tokens the warps that add up take more than an even share of the registers: 256
    // threads of 80, 256 of 128, 128 of 56 of the launch's 640 of 96 (107 us without; the last
    // warp only completes its group of four).  With 16 tokens they need no more.
    static constexpr bool kSplit = TOK == 32;
    static constexpr int kThreads = 32 * (kSplit ? 20 : 19);
    static constexpr int kUnpackRegs = 80, kAddRegs = 128, kOtherRegs = 56;
    static constexpr int kSplitSum = 256 * kUnpackRegs + 256 * kAddRegs + 128 * kOtherRegs;
    static constexpr int kXBytes = kN * kGroup;            // a step's B
    static constexpr uint32_t kD = 128, kX = kD + 4 * kN * kSub;  // TMEM columns; A from 0 on
    static constexpr uint32_t kIdesc = idesc_f16_f32(128, kN);   // (e4m3: the same bits)

    struct Shared {
        alignas(8) uint64_t full[kMaxSlots], empty[kMaxSlots];
        uint64_t a_full[2][2], d_full[2][2], d_empty[2][2], x_full[4], x_empty[4], drained[2];
        uint32_t tmem;
        int abort_flag;
    };

    static __host__ __device__ constexpr int fixed_bytes(int groups)
    {
        return 1024 + groups * (kXBytes + 8 * TOK * kSub);
    }

    static __device__ __forceinline__ bool wait(const WideArgs &p, Shared &s, uint64_t *bar,
                                                uint32_t parity)
    {
        return mbar_wait_warp(bar, parity, &s.abort_flag, p.dev_status, kDevPipelineTimeout,
                              p.wait_ns);
    }

    // The activations of tokens t0 .. t0 + TOK as B of every group, and for each two tokens
    // (2^(9 - e), 2^(9 - e), sum x, sum x).  8 lanes have a token's step, 16 values each, in
    // the order of the unpacked codes (0 2 4 6 1 3 5 7).
    static __device__ void stage(const WideArgs &p, int t0, uint8_t *xs, float *fs, int warp, int lane)
    {
        constexpr int kBatch = 2, kWarps = kLoad;
        const int items = p.groups * TOK, sub = lane >> 3, l = lane & 7;
        const uint64_t minus = pair_of(-1.0f, -1.0f), widen = pair_of(32.0f, 32.0f);
#pragma unroll 1
        for (int i0 = warp * 4 * kBatch; i0 < items; i0 += kWarps * 4 * kBatch) {
            uint4 v[kBatch][2];
#pragma unroll
            for (int u = 0; u < kBatch; u++) {
                const int i = i0 + 4 * u + sub, tok = i % TOK, t = t0 + tok;
                v[u][0] = v[u][1] = make_uint4(0, 0, 0, 0);
                if (i < items && t < p.M) {
                    const uint4 *x = reinterpret_cast<const uint4 *>(
                        p.x + static_cast<int64_t>(t) * p.K + i / TOK * kGroup + l * 16);
                    v[u][0] = x[0];
                    v[u][1] = x[1];
                }
            }
#pragma unroll
            for (int u = 0; u < kBatch; u++) {
                const int i = i0 + 4 * u + sub, tok = i % TOK, g = i / TOK;
                const uint32_t in[8] = {v[u][0].x, v[u][0].y, v[u][0].z, v[u][0].w,
                                        v[u][1].x, v[u][1].y, v[u][1].z, v[u][1].w};
                float f[16];
                uint64_t sums = 0;
                uint32_t tops = 0;             // magnitudes compare as integers
#pragma unroll
                for (int e = 0; e < 8; e++) {
                    f[2 * e] = __uint_as_float(in[e] << 16);
                    f[2 * e + 1] = __uint_as_float(in[e] & 0xFFFF0000u);
                    tops = __vmaxu2(tops, in[e] & 0x7FFF7FFFu);
                    sums = add2(sums, pair_of(f[2 * e], f[2 * e + 1]));
                }
                float sum = low(sums) + high(sums);
#pragma unroll
                for (int o = 4 / kSub; o > 0; o >>= 1) {
                    tops = __vmaxu2(tops, __shfl_xor_sync(0xffffffffu, tops, o));
                    sum += __shfl_xor_sync(0xffffffffu, sum, o);
                }
                const uint32_t top = max(tops & 0xFFFFu, tops >> 16);
                // the largest becomes 2^7 .. 2^8 (below 2^-120 less, for 2^e has to be a number; from
                // 2^126 on 2^(9 - e) is none: its token's results become NaN, for the parts would be
                // cut off at e4m3's largest value)
                const int e = min(max(134 - static_cast<int>(top >> 7), -118), 127);
                const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
                const uint64_t up2 = pair_of(up, up);
                uint32_t out[2][4];
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    // words of values 0 2 4 6, 1 3 5 7 and the same of the next eight
                    uint32_t part[2][2];
#pragma unroll
                    for (int h = 0; h < 2; h++) {
                        const int a = (j >> 1) * 8 + (j & 1) + 4 * h;
                        const uint64_t y = mul2(pair_of(f[a], f[a + 2]), up2);
                        part[0][h] = to_e4m3(low(y), high(y));
                        const float2 back = from_e4m3(part[0][h]);
                        const uint64_t rest = mul2(fma2(pair_of(back.x, back.y), minus, y), widen);
                        part[1][h] = to_e4m3(low(rest), high(rest));
                    }
                    out[0][j] = part[0][0] | part[0][1] << 16;
                    out[1][j] = part[1][0] | part[1][1] << 16;
                }
                if (i >= items)
                    continue;
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    const int n = h * TOK + tok;
                    if (W4_IN_BOUNDS(g < p.groups, p.dev_status))
                        *reinterpret_cast<uint4 *>(xs + g * kXBytes + n * 128 + ((l ^ (n & 7)) << 4)) =
                        make_uint4(out[h][0], out[h][1], out[h][2], out[h][3]);
                }
                if (l % (8 / kSub) == 0) {
                    const int group = g * kSub + l / (8 / kSub);
                    float *to = fs + (group * (TOK / 2) + (tok >> 1)) * 4 + (tok & 1);
                    to[0] = __uint_as_float(top >> 7 > 252 ? 0x7FC00000u
                                                           : static_cast<uint32_t>(127 + 9 - e) << 23);
                    to[2] = sum;
                }
            }
        }
    }

    // A role's place: its next group, its slot and how often the slots have been gone through
    // (counters: with divisions each role's step took some hundred cycles longer).
    struct Place {
        int task, g, slot, phase;
        __device__ __forceinline__ void next(const WideArgs &p, int by)
        {
            g += by;
            if (g >= p.groups) {
                g -= p.groups;
                task++;
            }
            slot += by;
            if (slot >= p.slots) {
                slot -= p.slots;
                phase ^= 1;
            }
        }
    };

    // The groups' codes in turn; returns how many were requested.
    static __device__ int load(const WideArgs &p, Shared &s, uint8_t *ring, int row0, int lane, Place &at,
                               int from, int to)
    {
        const uint64_t policy = l2_policy_evict_first();
        for (int i = from; i < to; i++, at.next(p, 1)) {
            if (i >= p.slots && !wait(p, s, &s.empty[at.slot], at.phase ^ 1))
                return i;
            if (lane == 0) {
                mbar_arrive_expect_tx(&s.full[at.slot], kSlotBytes);
                tma_load_2d(ring + at.slot * kSlotBytes, &p.map, at.g * (kGroup / 2),
                            row0 + at.task * kRows, &s.full[at.slot], policy);
            }
            __syncwarp();
        }
        return to;
    }

    // Set w's MMAs.
    static __device__ void issuer(const WideArgs &p, Shared &s, const uint8_t *xs, int w, int total)
    {
        const uint32_t tmem = s.tmem;
        const uint64_t bd = sdesc_sw128(smem_u32(xs));
        Place at{0, w, w, 0};
        for (int idx = w, i = 0; idx < total; idx += 2, i++, at.next(p, 2)) {
            const int b = i & 1, g = at.g;
            if (!wait(p, s, &s.a_full[w][b], i >> 1 & 1) ||
                (i > 1 && !wait(p, s, &s.d_empty[w][b], (i - 2) >> 1 & 1)))
                break;
            tc_fence_after();
            __syncwarp();
            const uint32_t d = tmem + kD + kN * kSub * (2 * w + b), a = tmem + 32 * (2 * w + b);
            const uint64_t x = bd + static_cast<uint64_t>(g) * (kXBytes >> 4);
            if constexpr (kSub == 1) {
                mma_group(d, a, x, kIdesc);
            } else {
                mma_half(d, a, x, kIdesc);
                mma_half(d + kN, a + 16, x + 4, kIdesc);
            }
            tc_commit_elect(&s.d_full[w][b]);
        }
        // nothing of this warp's is under way when the CTA ends
        __syncwarp();
        tc_commit_elect(&s.drained[w]);
        mbar_drain(&s.drained[w], 0);
        __syncwarp();
    }

    // 16 columns from t0 and 16 from t1, of 16 of the warp's lanes: a thread gets rows l / 4
    // and l / 4 + 8 of them, columns 2 (l % 4) and the next of each 8: of a row in v[4 i + 2 r].
    static __device__ __forceinline__ void load_sums(uint32_t t0, uint32_t t1, uint32_t (&a)[8],
                                                     uint32_t (&b)[8])
    {
        asm volatile(
            "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%16];\n\t"
            "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%8, %9, %10, %11, %12, %13, %14, %15}, [%17];"
            : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3]), "=r"(a[4]), "=r"(a[5]), "=r"(a[6]),
              "=r"(a[7]), "=r"(b[0]), "=r"(b[1]), "=r"(b[2]), "=r"(b[3]), "=r"(b[4]), "=r"(b[5]),
              "=r"(b[6]), "=r"(b[7])
            : "r"(t0), "r"(t1)
            : "memory");
    }
    static __device__ __forceinline__ void wait_loads(uint32_t (&a)[8], uint32_t (&b)[8])
    {
        // (what was loaded is not there before it)
        asm volatile("tcgen05.wait::ld.sync.aligned;"
                     : "+r"(a[0]), "+r"(a[1]), "+r"(a[2]), "+r"(a[3]), "+r"(a[4]), "+r"(a[5]),
                       "+r"(a[6]), "+r"(a[7]), "+r"(b[0]), "+r"(b[1]), "+r"(b[2]), "+r"(b[3]),
                       "+r"(b[4]), "+r"(b[5]), "+r"(b[6]), "+r"(b[7])
                     :
                     : "memory");
    }
    // 16 columns of 16 lanes in that layout.
    static __device__ __forceinline__ void store_sums(uint32_t to, const float (&v)[8])
    {
        asm volatile(
            "tcgen05.st.sync.aligned.16x256b.x2.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(to),
            "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
            : "memory");
    }

    // A warp that unpacks 32 rows of set w's groups.
    static __device__ void unpack(const WideArgs &p, Shared &s, const uint8_t *ring, int w, int quarter,
                                  int lane, int total)
    {
        const uint32_t tmem = s.tmem + (static_cast<uint32_t>(quarter * 32) << 16);
        const int mine = quarter * 32 + lane;
        Place at{0, w, w, 0};
        for (int idx = w, i = 0; idx < total; idx += 2, i++, at.next(p, 2)) {
            const int slot = at.slot, b = i & 1;
            if (!wait(p, s, &s.full[slot], at.phase))
                return;
            uint32_t q[16], a[32];
            const uint8_t *row = ring + slot * kSlotBytes + mine * 64;
#pragma unroll
            for (int j = 0; j < 4; j++)
                *reinterpret_cast<uint4 *>(q + 4 * j) =
                    *reinterpret_cast<const uint4 *>(row + ((j ^ (mine >> 1 & 3)) << 4));
#pragma unroll
            for (int j = 0; j < 16; j++) {
                a[2 * j] = q[j] & 0x0F0F0F0Fu;
                a[2 * j + 1] = q[j] >> 4 & 0x0F0F0F0Fu;
            }
            // these reads come before the copy that overwrites the slot, which is another proxy's:
            // without the fence some rows were the next codes in a call of fifty
            fence_proxy_async_smem();
            __syncwarp();
            mbar_arrive_elect(&s.empty[slot]);
            // the MMAs that read this A last are done when their sums are there
            if (i > 1 && !wait(p, s, &s.d_full[w][b], (i - 2) >> 1 & 1))
                return;
            tc_fence_after();
            __syncwarp();
            tmem_st_32x32b_x32(tmem + 32 * (2 * w + b), a);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            mbar_arrive_elect(&s.a_full[w][b]);
        }
    }

    // A warp that adds up 32 rows of set w's groups.  A thread has 4 of the rows and a quarter of
    // the tokens, so that it reads a quarter of the tokens' factors (a row of all tokens a thread:
    // 16 reads of 16 bytes a group, the same for all lanes and four wavefronts each).  Its
    // accumulators are in the order of load_sums, by 16 tokens and 16 rows.
    static __device__ void add(const WideArgs &p, Shared &s, const float *fs, int t0, int row0, int w,
                               int quarter, int lane, int total)
    {
        const uint32_t tmem = s.tmem + (static_cast<uint32_t>(quarter * 32) << 16);
        const int mine = quarter * 32 + lane;
        uint64_t acc[TOK / 16][2][4];
        auto clear = [&]() {
#pragma unroll
            for (int i = 0; i < TOK / 2; i++)
                acc[i / 8][i / 4 % 2][i % 4] = 0;
        };
        clear();
        // scale and zero of the group to come.  (Further ahead, the loop unrolled for it, costs
        // more than it hides: the roles' code together is more than the instruction cache
        // holds.  4 ahead 98 us, 6 ahead 106.)
        Place to{0, w, w, 0}, at = to;
        uint16_t sc[kSub], ze[kSub];
        auto scales = [&](int idx) {
            const int64_t row = min(row0 + to.task * kRows + mine, p.N - 1);
            const int64_t at = (row * p.groups + to.g) * kSub;
            const bool there =
                idx < total && W4_IN_BOUNDS(at >= 0 && at + kSub <= static_cast<int64_t>(p.N) *
                                                                        p.groups * kSub, p.dev_status);
#pragma unroll
            for (int k = 0; k < kSub; k++) {
                sc[k] = there ? load_weight(p.s + at + k) : static_cast<uint16_t>(0);
                ze[k] = there ? load_weight(p.z + at + k) : static_cast<uint16_t>(0);
            }
            to.next(p, 2);
        };
        scales(w);
#pragma unroll 1
        for (int idx = w, i = 0; idx < total; idx += 2, i++) {
            const int b = i & 1, g = at.g, task = at.task;
            uint32_t scale[kSub];
#pragma unroll
            for (int k = 0; k < kSub; k++)
                scale[k] = sc[k] | static_cast<uint32_t>(ze[k]) << 16;
            scales(idx + 2);
            const uint64_t small = pair_of(0.03125f, 0.03125f);
            const ulonglong2 *f =
                reinterpret_cast<const ulonglong2 *>(fs) + g * kSub * (TOK / 2) + (lane & 3);
            uint64_t s2[4], z2[4];
            // the four rows' scales and zeros of the step's group k
            auto share = [&](int k) {
#pragma unroll
                for (int r = 0; r < 4; r++) {
                    const uint32_t v = __shfl_sync(0xffffffffu, scale[k], 8 * r + (lane >> 2));
                    const float sv = __half2float(__ushort_as_half(static_cast<uint16_t>(v)));
                    const float zv = -__half2float(__ushort_as_half(static_cast<uint16_t>(v >> 16)));
                    s2[r] = pair_of(sv, sv);
                    z2[r] = pair_of(zv, zv);
                }
            };
            share(0);
            if (!wait(p, s, &s.d_full[w][b], i >> 1 & 1))
                return;
            tc_fence_after();
            __syncwarp();
            uint32_t d1[2][8], d2[2][8];
            const uint32_t d = tmem + kD + kN * kSub * (2 * w + b);
            load_sums(d, d + TOK, d1[0], d2[0]);
            constexpr int kParts = TOK / 8;                    // of 16 tokens and 16 rows, of a group
#pragma unroll
            for (int j0 = 0; j0 < kParts * kSub; j0++) {
                const int k = j0 / kParts, i = j0 % kParts, c = i / 2, h = i % 2;
                if (k > 0 && i == 0)
                    share(k);
                wait_loads(d1[h], d2[h]);
                if (j0 + 1 < kParts * kSub) {
                    const int n = (j0 + 1) % kParts;
                    const uint32_t next =
                        d + (j0 + 1) / kParts * kN + n / 2 * 16 + ((n % 2 * 16) << 16);
                    load_sums(next, next + TOK, d1[h ^ 1], d2[h ^ 1]);
                } else {
                    tc_fence_before();
                    __syncwarp();
                    mbar_arrive_elect(&s.d_empty[w][b]);
                }
#pragma unroll
                for (int j = 0; j < 2; j++) {
                    // two tokens' factors, their sums
                    const ulonglong2 fv = f[k * (TOK / 2) + c * 8 + j * 4];
#pragma unroll
                    for (int r = 0; r < 2; r++) {
                        const int at = 4 * j + 2 * r;
                        const uint64_t e1 = static_cast<uint64_t>(d1[h][at + 1]) << 32 | d1[h][at];
                        const uint64_t e2 = static_cast<uint64_t>(d2[h][at + 1]) << 32 | d2[h][at];
                        uint64_t &to = acc[c][h][2 * j + r];
                        to = fma2(s2[2 * h + r],
                                  fma2(fv.x, fma2(e2, small, e1), mul2(z2[2 * h + r], fv.y)), to);
                    }
                }
            }
            at.next(p, 2);
            if (at.task != task) {                         // that was the set's last of the task
                if (!finish(p, s, t0, row0 + task * kRows + mine, w, quarter, task, tmem, acc))
                    return;
                clear();
            }
        }
    }

    // Whether y has a value at `at`.
    static __device__ __forceinline__ bool in_y(const WideArgs &p, const uint16_t *at)
    {
        return at >= p.y && at < p.y + static_cast<int64_t>(p.M) * p.N;
    }

    // A task's sums: the second set's through tensor memory to the first, which stores them.
    static __device__ __forceinline__ bool finish(const WideArgs &p, Shared &s, int t0, int row, int w,
                                                  int quarter, int done, uint32_t tmem,
                                                  const uint64_t (&acc)[TOK / 16][2][4])
    {
        uint32_t v[TOK];
        if (w == 1) {
            if (done > 0 && !wait(p, s, &s.x_empty[quarter], (done - 1) & 1))
                return false;
            tc_fence_after();
            __syncwarp();
#pragma unroll
            for (int j = 0; j < TOK / 2; j++) {
                v[2 * j] = static_cast<uint32_t>(acc[j / 8][j / 4 % 2][j % 4]);
                v[2 * j + 1] = static_cast<uint32_t>(acc[j / 8][j / 4 % 2][j % 4] >> 32);
            }
            if constexpr (TOK == 16)
                tmem_st_32x32b_x16(tmem + kX, v);
            else
                tmem_st_32x32b_x32(tmem + kX, v);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            mbar_arrive_elect(&s.x_full[quarter]);
            return true;
        }
        if (!wait(p, s, &s.x_full[quarter], done & 1))
            return false;
        tc_fence_after();
        __syncwarp();
        if constexpr (TOK == 16)
            tmem_ld_32x32b_x16(tmem + kX, v);
        else
            tmem_ld_32x32b_x32(tmem + kX, v);
        // from a thread's own values to its row's, for wider stores
#pragma unroll
        for (int i = 0; i < TOK / 8; i++) {
            float sum[8];
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const uint64_t mine = acc[i / 2][i % 2][j];
                sum[2 * j] = low(mine) + __uint_as_float(v[8 * i + 2 * j]);
                sum[2 * j + 1] = high(mine) + __uint_as_float(v[8 * i + 2 * j + 1]);
            }
            store_sums(tmem + kX + i / 2 * 16 + ((i % 2 * 16) << 16), sum);
        }
        tmem_wait_st();
        if constexpr (TOK == 16)
            tmem_ld_32x32b_x16(tmem + kX, v);
        else
            tmem_ld_32x32b_x32(tmem + kX, v);
        tc_fence_before();
        __syncwarp();
        mbar_arrive_elect(&s.x_empty[quarter]);
#pragma unroll
        for (int j = 0; j < TOK / 2; j++) {
            const uint32_t r = bf16_pair(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
            const int t = t0 + 2 * j;
            uint16_t *y = p.y + static_cast<int64_t>(t) * p.N + row;
            if (row < p.N && t < p.M && W4_IN_BOUNDS(in_y(p, y), p.dev_status))
                y[0] = static_cast<uint16_t>(r);
            if (row < p.N && t + 1 < p.M && W4_IN_BOUNDS(in_y(p, y + p.N), p.dev_status))
                y[p.N] = static_cast<uint16_t>(r >> 16);
        }
        __syncwarp();
        return true;
    }
};

// CTA (share, part): its share of the tasks, for the part's TOK tokens.
template <int TOK, int GROUP>
__global__ void __launch_bounds__(Wide<TOK, GROUP>::kThreads, 1)
    few_linear_wide_kernel(const __grid_constant__ WideArgs p, int parts)
{
    using W = Wide<TOK, GROUP>;
    extern __shared__ __align__(1024) uint8_t raw[];
    __shared__ __align__(16) typename W::Shared s;
    uint8_t *ring = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    uint8_t *xs = ring + p.slots * kSlotBytes;
    float *fs = reinterpret_cast<float *>(xs + p.groups * W::kXBytes);
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int share = blockIdx.x / parts, shares = gridDim.x / parts;
    const int t0 = (blockIdx.x - share * parts) * TOK;
    const int tasks = (p.N + kRows - 1) / kRows;
    const int first = static_cast<int>(static_cast<int64_t>(tasks) * share / shares);
    const int end = static_cast<int>(static_cast<int64_t>(tasks) * (share + 1) / shares);
    const int row0 = first * kRows, total = (end - first) * p.groups;
    if (tid == 0) {
        for (int i = 0; i < p.slots; i++) {
            mbar_init(&s.full[i], p.withhold && i == 0 ? 2 : 1);
            mbar_init(&s.empty[i], 4);
        }
        for (int i = 0; i < 2; i++) {
            for (int j = 0; j < 2; j++) {
                mbar_init(&s.a_full[i][j], 4);
                mbar_init(&s.d_full[i][j], 1);
                mbar_init(&s.d_empty[i][j], 4);
            }
            mbar_init(&s.drained[i], 1);
        }
        for (int i = 0; i < 4; i++) {
            mbar_init(&s.x_full[i], 1);
            mbar_init(&s.x_empty[i], 1);
        }
        s.abort_flag = 0;
        fence_mbar_init();
        prefetch_tmap(&p.map);
    }
    if (warp == kLoad) {
        tmem_alloc(&s.tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_wait();
    pdl_trigger();
    const int ahead = min(p.slots, total);
    typename W::Place place{0, 0, 0, 0};
    if (warp == kLoad) {
        W::load(p, s, ring, row0, lane, place, 0, ahead);
    } else if (warp < kLoad) {
        W::stage(p, t0, xs, fs, warp, lane);
        fence_proxy_async_smem();
    }
    __syncthreads();
    if constexpr (W::kSplit) {
        if (warp < kAdd)
            asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(W::kUnpackRegs));
        else if (warp < kIssue)
            asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(W::kAddRegs));
        else
            asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(W::kOtherRegs));
    }
    if (warp < kAdd) {
        W::unpack(p, s, ring, warp >> 2, warp & 3, lane, total);
    } else if (warp < kIssue) {
        W::add(p, s, fs, t0, row0, (warp - kAdd) >> 2, warp & 3, lane, total);
    } else if (warp < kLoad) {
        W::issuer(p, s, xs, warp - kIssue, total);
    } else if (warp == kLoad) {
        const int i = W::load(p, s, ring, row0, lane, place, ahead, total);
        // every copy requested has landed, or had its time to: of a slot only the last can be
        // under way
        for (int slot = 0; slot < min(i, p.slots); slot++)
            mbar_drain(&s.full[slot], (i - 1 - slot) / p.slots & 1);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == kLoad) {
        tc_fence_after();
        __syncwarp();
        tmem_dealloc(s.tmem, 512);
    }
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

// Slots that fit beside the activations: even, so that a slot is always the same set's.
template <int TOK, int GROUP> int slots_of(int groups)
{
    return std::min((kMaxSmem - 2048 - Wide<TOK, GROUP>::fixed_bytes(groups)) / kSlotBytes / 2 * 2,
                    kMaxSlots);
}

template <int TOK, int GROUP>
cudaError_t launch_as(WideArgs &a, int sms, int dev, cudaStream_t stream)
{
    using W = Wide<TOK, GROUP>;
    auto kern = few_linear_wide_kernel<TOK, GROUP>;
    static std::atomic<uint64_t> raised{0};      // devices whose limit is raised already
    if (!(raised.load(std::memory_order_relaxed) >> (dev & 63) & 1u)) {
        cudaError_t err =
            cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem - 2048);
        if (err != cudaSuccess)
            return err;
        if (W::kSplit) {                       // what setmaxnreg shares out is there
            cudaFuncAttributes attr;
            if ((err = cudaFuncGetAttributes(&attr, kern)) != cudaSuccess)
                return err;
            if (attr.numRegs * W::kThreads < W::kSplitSum)
                return cudaErrorLaunchOutOfResources;
        }
        raised.fetch_or(1ull << (dev & 63), std::memory_order_relaxed);
    }
    a.slots = slots_of<TOK, GROUP>(a.groups);
    const int parts = (a.M + TOK - 1) / TOK, tasks = (a.N + kRows - 1) / kRows;
    const int shares = std::min(tasks, std::max(sms / parts, 1));
    const int smem = W::fixed_bytes(a.groups) + a.slots * kSlotBytes;
    return launch_pdl(kern, dim3(shares * parts), dim3(W::kThreads), smem, stream, a, parts);
}

}  // namespace

// The tokens of a CTA, 32 or 16; 0: the shape is not for this kernel.
int few_linear_wide_tokens(int M, int K, int group)
{
    constexpr int kLeast = 4;                  // slots, and steps
    if (K % kGroup || K < kLeast * kGroup || M <= 8)
        return 0;
    const int steps = K / kGroup;
    if (group == 64)
        return slots_of<16, 64>(steps) >= kLeast ? 16 : 0;
    if (M > 16 && slots_of<32, 128>(steps) >= kLeast)
        return 32;
    return slots_of<16, 128>(steps) >= kLeast ? 16 : 0;
}

cudaError_t launch_few_linear_wide(const FewLinearProblem &q, cudaStream_t stream)
{
    int dev = 0, sms = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err == cudaSuccess)
        err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (err != cudaSuccess)
        return err;
    if (!encode_fn())
        return cudaErrorNotSupported;
    WideArgs a{};
    const cuuint64_t dim[2] = {static_cast<cuuint64_t>(q.K / 2), static_cast<cuuint64_t>(q.N)};
    const cuuint64_t stride[1] = {static_cast<cuuint64_t>(q.K / 2)};
    const cuuint32_t box[2] = {kGroup / 2, kRows}, step[2] = {1, 1};
    if (encode_fn()(&a.map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t *>(q.q), dim, stride,
                    box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    a.x = q.x;
    a.s = q.s;
    a.z = q.z;
    a.y = q.y;
    a.dev_status = q.dev_status;
    a.wait_ns = pipeline_test_hooks().wait_ns;
    a.withhold = pipeline_test_hooks().withhold_sz;
    a.M = q.M;
    a.K = q.K;
    a.N = q.N;
    a.groups = q.K / kGroup;
    if (q.group == 64)
        return launch_as<16, 64>(a, sms, dev, stream);
    return few_linear_wide_tokens(q.M, q.K, q.group) == 32 ? launch_as<32, 128>(a, sms, dev, stream)
                                                           : launch_as<16, 128>(a, sms, dev, stream);
}

}  // namespace w4
