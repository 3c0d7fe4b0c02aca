// linear_few.cu -- the dense W4A16 linear for a few tokens, in one launch:
//   y[t, n] = sum_k x[t, k] s[n, g] (q[n, k] - z[n, g]),  g = k / group
//
// With up to 32 tokens the product is the stream of the packed weights.  A warp's
// MMA (16 weight rows x 8 tokens x 16, bf16) takes the codes as they lie in memory:
// a nibble masked in place is the bf16 number q 2^-133 (low nibble of a byte) or
// 16 q 2^-133 (high nibble), below and just above where bf16's subnormals end and
// linear throughout, so codes enter exactly for one AND each.  Activations are bf16
// already; they are scaled by 2^70 (the high nibbles' by 2^66), which is exact, so
// that products lie in fp32's normal range.  A group's scale and zero are applied to
// its fp32 sum,
//   sum_k s (q_k - z) x_k = s (sum_k q_k x_k - z sum_k x_k),
// so neither weights nor activations are rounded.  The contraction order inside a
// group is free as long as codes and activations agree on it: a lane takes the 8 codes
// of a word, and the activations are stored to match.
//
// A task is 16 RT weight rows, a unit 128 codes of each.  A CTA has up to 8 NT of the
// tokens and an equal contiguous share of the tasks, its warps equal shares of those
// tasks' units; a task that crosses warps is added up in warp order through shared
// memory.  A warp copies the codes that it will use itself into its own ring in shared
// memory, S units ahead, and waits for nobody else's.  Sums run in a fixed order:
// bit-identical reruns.
//
// Measured on GB300 from a graph: 1 token, 2816 -> 4096: 4.4 us (latency: launch, the
// activations' way to shared memory, one round of copies, the warps' sums; 0.9 for the
// bytes); 11 tokens, 704 -> 2815, groups of 64: 3.1; 8 tokens, 2816 -> 262144: 68 to 74 (60 at
// the copy bandwidth), 8192 -> 38912 43 (25), with groups of 64 64 (27): the scales' sectors, and
// where the activations take most of shared memory little is in flight.  With 16 tokens the
// MMAs (2 cycles each an SM) and the unpacking are at some 45 % of their rates each (2816 ->
// 262144 85); codes requested into registers instead of the ring: 87 and 101, and 7 for the
// small ones.
#include <algorithm>
#include <atomic>
#include <cuda_fp16.h>

#include "../../include/w4moe.h"
#include "checks.cuh"
#include "launch.h"
#include "ptx.cuh"

namespace w4 {

namespace {

constexpr float kUp = 0x1p70f, kUpHigh = 0x1p66f;  // of activations for low and high nibbles
constexpr float kSum = 0x1p-63f;                   // 2^70 2^-133: of sums
constexpr float kDown = 0x1p63f;                   // undone at the end

struct FewLinearArgs {
    const uint16_t *x;                     // [M, K] bf16
    const uint8_t *q;                      // [N, K / 2]
    const uint16_t *s, *z;                 // [N, K / group] fp16
    uint16_t *y;                           // [M, N] bf16
    int32_t *dev_status;
    int M, K, N;
    int blocks;                            // of 128 codes, the last may be half of one
};

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ void copy_async(void *to, const void *from)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to)), "l"(from)
                 : "memory");
}

__device__ __forceinline__ float half_of(uint16_t h) { return __half2float(__ushort_as_half(h)); }

// NT: tiles of 8 tokens; RT: tiles of 16 weight rows; NW: warps; S: units in flight a warp.
template <int GROUP, int NT, int RT, int NW, int S>
struct FewLinear {
    static constexpr int kGroups = 128 / GROUP;            // of a unit
    static constexpr int kWords = 4 / kGroups;             // of a lane's row and group
    static constexpr int kRows = 16 * RT;
    static constexpr int kRingBytes = NW * S * RT * 1024;

    // Bytes of a tile of 8 tokens: the activations [block][4][8 tokens][4] x 16 bytes, then
    // the groups' sums [block][groups][8 tokens].
    static __host__ __device__ constexpr int tile_bytes(int blocks)
    {
        return blocks * (4 * 512 + kGroups * 32);
    }

    // Of a unit in flight, by lane: a scale or zero of weight row 2 g or 2 g + 1 of each row
    // tile (s, z, s, z for the four lanes of g); its codes are in the ring.
    struct Unit {
        uint16_t sz[RT][kGroups];
    };

    // Where a unit's half (a group of 64) of the rows of lanes g lies in their 64 bytes: other
    // rows' other way round, so that eight bytes of four rows have banks of their own.
    static __device__ __forceinline__ int half_at(int g, int h) { return (h ^ (g >> 1 & 1)) * 32; }

    // Requests a unit: the codes of rows 2 g and 2 g + 1 into the slot, 16 bytes a lane and row.
    // With groups of 128 they are the lane's own; with groups of 64 two lanes have 8 of them
    // each, and the warp waits for one another.  (Copies of 8 bytes, each lane's own, go
    // through what is left of L1: 5632 -> 38912 73 us.)
    static __device__ __forceinline__ void load(const FewLinearArgs &p, int64_t row0, int block,
                                                int lane, uint8_t *slot, Unit &u)
    {
        const int g = lane >> 2, t4 = lane & 3, G = p.K / GROUP;
        const uint16_t *sz = t4 & 1 ? p.z : p.s;
#pragma unroll
        for (int r = 0; r < RT; r++) {
            // rows past the last one repeat it; what they give is not stored
            const int64_t last = static_cast<int64_t>(p.N) - 1, row = row0 + r * 16 + 2 * g;
#pragma unroll
            for (int i = 0; i < 2; i++) {
                const uint8_t *q = p.q + min(row + i, last) * (p.K / 2) + block * 64;
                uint8_t *to = slot + (r * 2 + i) * 512 + g * 64;
                if constexpr (GROUP == 128) {
                    copy_async(to + t4 * 16, q + t4 * 16);
                } else {
                    // of half a unit at the end the first half stands for the second,
                    // whose scales are zero
                    const int c = block * 2 + 1 < G ? t4 : t4 & 1;
                    copy_async(to + half_at(g, t4 >> 1) + (t4 & 1) * 16, q + c * 16);
                }
            }
#pragma unroll
            for (int h = 0; h < kGroups; h++)
                u.sz[r][h] = kGroups == 1 || block * kGroups + h < G
                                 ? sz[min(row + (t4 >> 1), last) * G + block * kGroups + h]
                                 : static_cast<uint16_t>(0);
        }
    }

    static __device__ __forceinline__ void add(const uint8_t *xs, int tile_stride, int blocks,
                                               int block, int lane, const uint8_t *slot,
                                               const Unit &u, float (&acc)[RT][NT][4])
    {
        const int g = lane >> 2, t4 = lane & 3;
        uint32_t q[RT][2][4];
#pragma unroll
        for (int r = 0; r < RT; r++)
#pragma unroll
            for (int i = 0; i < 2; i++) {
                const uint8_t *row = slot + (r * 2 + i) * 512 + g * 64;
                if constexpr (GROUP == 128) {
                    *reinterpret_cast<uint4 *>(q[r][i]) =
                        *reinterpret_cast<const uint4 *>(row + t4 * 16);
                } else {
#pragma unroll
                    for (int h = 0; h < 2; h++)
                        *reinterpret_cast<uint2 *>(q[r][i] + 2 * h) =
                            *reinterpret_cast<const uint2 *>(row + half_at(g, h) + t4 * 8);
                }
            }
#pragma unroll
        for (int h = 0; h < kGroups; h++) {
            float part[RT][NT][4] = {};
#pragma unroll
            for (int w = 0; w < kWords; w++) {
                const int j = h * kWords + w;
                uint4 b[NT];
#pragma unroll
                for (int n = 0; n < NT; n++)
                    b[n] = *reinterpret_cast<const uint4 *>(xs + n * tile_stride +
                                                            (block * 4 + j) * 512 + lane * 16);
#pragma unroll
                for (int r = 0; r < RT; r++) {
                    const uint32_t w0 = q[r][0][j], w1 = q[r][1][j];
                    const uint32_t v0 = w0 >> 8, v1 = w1 >> 8;
#pragma unroll
                    for (int n = 0; n < NT; n++) {
                        mma_bf16(part[r][n], w0 & 0x000F000Fu, w1 & 0x000F000Fu, v0 & 0x000F000Fu,
                                 v1 & 0x000F000Fu, b[n].x, b[n].y);
                        mma_bf16(part[r][n], w0 & 0x00F000F0u, w1 & 0x00F000F0u, v0 & 0x00F000F0u,
                                 v1 & 0x00F000F0u, b[n].z, b[n].w);
                    }
                }
            }
            float2 sum[NT];
#pragma unroll
            for (int n = 0; n < NT; n++)
                sum[n] = *reinterpret_cast<const float2 *>(
                    xs + n * tile_stride + blocks * 2048 + (block * kGroups + h) * 32 + t4 * 8);
#pragma unroll
            for (int r = 0; r < RT; r++) {
                const float mine = half_of(u.sz[r][h]);
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    const float s = __shfl_sync(0xffffffffu, mine, 2 * i, 4);
                    const float z = __shfl_sync(0xffffffffu, mine, 2 * i + 1, 4);
#pragma unroll
                    for (int n = 0; n < NT; n++) {
                        float *a = &acc[r][n][2 * i];
                        a[0] = fmaf(s, fmaf(-z, sum[n].x, part[r][n][2 * i]), a[0]);
                        a[1] = fmaf(s, fmaf(-z, sum[n].y, part[r][n][2 * i + 1]), a[1]);
                    }
                }
            }
        }
    }

    // Activations t0 .. t0 + 8 NT of x into shared memory, in the order of the codes, with
    // their groups' sums; tokens past the last and columns past K are zero.  A warp takes a
    // tile's block at a time, a lane what the MMA's lane of that place will read: 4 words of
    // one token.
    static __device__ __forceinline__ void stage(const FewLinearArgs &p, int t0, uint8_t *xs,
                                                 int tile_stride, int lane, int warp)
    {
        const int tok = lane >> 2, t4 = lane & 3;
        for (int i = warp; i < NT * p.blocks; i += NW) {
            const int n = i / p.blocks, block = i - n * p.blocks, t = t0 + n * 8 + tok;
            const uint16_t *x = p.x + static_cast<int64_t>(t) * p.K + block * 128;
            uint4 v[4];
#pragma unroll
            for (int j = 0; j < 4; j++) {
                // in a unit of two groups the lane has two words of each
                const int word = kGroups == 1 ? t4 * 4 + j : (j >> 1) * 8 + t4 * 2 + (j & 1);
                v[j] = make_uint4(0, 0, 0, 0);
                if (t < p.M && block * 128 + word * 8 < p.K)
                    v[j] = *reinterpret_cast<const uint4 *>(x + word * 8);
            }
            uint8_t *tile = xs + n * tile_stride;
            float sums[kGroups] = {};
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const uint32_t in[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
                float f[8];
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    f[2 * e] = __uint_as_float(in[e] << 16);
                    f[2 * e + 1] = __uint_as_float(in[e] & 0xFFFF0000u);
                }
#pragma unroll
                for (int e = 0; e < 8; e++)
                    sums[j / kWords] += f[e];
                uint4 out;
                out.x = bf16_pair(f[0] * kUp, f[4] * kUp);
                out.y = bf16_pair(f[2] * kUp, f[6] * kUp);
                out.z = bf16_pair(f[1] * kUpHigh, f[5] * kUpHigh);
                out.w = bf16_pair(f[3] * kUpHigh, f[7] * kUpHigh);
                if (W4_IN_BOUNDS(n < NT && block * 4 + j < p.blocks * 4, p.dev_status))
                    *reinterpret_cast<uint4 *>(tile + (block * 4 + j) * 512 + lane * 16) = out;
            }
#pragma unroll
            for (int h = 0; h < kGroups; h++) {
                float sum = sums[h];
                sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                if (t4 == 0)
                    *reinterpret_cast<float *>(tile + p.blocks * 2048 +
                                               (block * kGroups + h) * 32 + tok * 4) = sum * kSum;
            }
        }
    }

    static constexpr int kHeadBytes = NW * RT * NT * 512;
    static __device__ __forceinline__ void put_head(float4 *heads, int warp, int lane,
                                                    const float (&acc)[RT][NT][4])
    {
#pragma unroll
        for (int r = 0; r < RT; r++)
#pragma unroll
            for (int n = 0; n < NT; n++)
                heads[((warp * RT + r) * NT + n) * 32 + lane] =
                    make_float4(acc[r][n][0], acc[r][n][1], acc[r][n][2], acc[r][n][3]);
    }

    // Whether y has n values from `at` on.
    static __device__ __forceinline__ bool in_y(const FewLinearArgs &p, const uint16_t *at, int n)
    {
        return at >= p.y && at + n <= p.y + static_cast<int64_t>(p.M) * p.N;
    }

    // A finished task's sums to y, two neighbouring rows of a token at a time.
    static __device__ __forceinline__ void store(const FewLinearArgs &p, int t0, int64_t row0,
                                                 int lane, const float (&acc)[RT][NT][4])
    {
        const int g = lane >> 2, t4 = lane & 3;
#pragma unroll
        for (int n = 0; n < NT; n++)
#pragma unroll
            for (int c = 0; c < 2; c++) {
                const int t = t0 + n * 8 + 2 * t4 + c;
                if (t >= p.M)
                    continue;
#pragma unroll
                for (int r = 0; r < RT; r++) {
                    const int64_t row = row0 + r * 16 + 2 * g;
                    const uint32_t v = bf16_pair(acc[r][n][c] * kDown, acc[r][n][2 + c] * kDown);
                    uint16_t *y = p.y + static_cast<int64_t>(t) * p.N + row;
                    if (row + 1 < p.N && (p.N & 1) == 0) {
                        if (W4_IN_BOUNDS(in_y(p, y, 2), p.dev_status))
                            *reinterpret_cast<uint32_t *>(y) = v;
                    } else {
                        if (row < p.N && W4_IN_BOUNDS(in_y(p, y, 1), p.dev_status))
                            y[0] = static_cast<uint16_t>(v);
                        if (row + 1 < p.N && W4_IN_BOUNDS(in_y(p, y + 1, 1), p.dev_status))
                            y[1] = static_cast<uint16_t>(v >> 16);
                    }
                }
            }
    }
};

// CTA (share, part): its share of the tasks, for the part's 8 NT tokens.  The parts of a
// share run side by side, so the weights come from HBM once.
template <int GROUP, int NT, int RT, int NW, int S>
__global__ void __launch_bounds__(32 * NW, 1) few_linear_kernel(const FewLinearArgs p, int parts)
{
    using F = FewLinear<GROUP, NT, RT, NW, S>;
    extern __shared__ __align__(16) uint8_t xs[];
    const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
    const int tile_stride = F::tile_bytes(p.blocks);
    // each warp's sums of the task that another one began, then its ring
    float4 *heads = reinterpret_cast<float4 *>(xs + NT * tile_stride);
    uint8_t *ring = xs + NT * tile_stride + F::kHeadBytes + warp * (S * RT * 1024);
    const int share = blockIdx.x / parts, shares = gridDim.x / parts;
    const int t0 = (blockIdx.x - share * parts) * (8 * NT);
    const int tasks = (p.N + F::kRows - 1) / F::kRows;
    const int a = static_cast<int>(static_cast<int64_t>(tasks) * share / shares);
    const int e = static_cast<int>(static_cast<int64_t>(tasks) * (share + 1) / shares);
    const int units = (e - a) * p.blocks;
    const int u0 = static_cast<int>(static_cast<int64_t>(units) * warp / NW);
    const int u1 = static_cast<int>(static_cast<int64_t>(units) * (warp + 1) / NW);
    pdl_wait();
    pdl_trigger();
    typename F::Unit unit[S];
    // the next unit to request, the next to add
    int ask = u0, ask_task = u0 / p.blocks, ask_block = u0 - ask_task * p.blocks;
    int task = ask_task, block = ask_block;
    auto request = [&](int slot) {
        if (ask < u1)
            F::load(p, static_cast<int64_t>(a + ask_task) * F::kRows, ask_block, lane,
                    ring + slot * (RT * 1024), unit[slot]);
        asm volatile("cp.async.commit_group;" ::: "memory");
        ask++;
        if (++ask_block == p.blocks) {
            ask_block = 0;
            ask_task++;
        }
    };
#pragma unroll
    for (int i = 0; i < S; i++)
        request(i);
    F::stage(p, t0, xs, tile_stride, lane, warp);
    __syncthreads();
    float acc[RT][NT][4] = {};
    bool in_head = block > 0 && u0 < u1;       // another warp has the task's first part
    for (int u = u0; u < u1;) {
#pragma unroll
        for (int i = 0; i < S; i++) {
            if (u < u1) {
                asm volatile("cp.async.wait_group %0;" ::"n"(S - 1) : "memory");
                if constexpr (GROUP == 64)
                    __syncwarp();              // other lanes' copies
                F::add(xs, tile_stride, p.blocks, block, lane, ring + i * (RT * 1024), unit[i], acc);
                if constexpr (GROUP == 64)
                    __syncwarp();              // and reads
                request(i);
                u++;
                if (++block == p.blocks) {
                    if (in_head)
                        F::put_head(heads, warp, lane, acc);
                    else
                        F::store(p, t0, static_cast<int64_t>(a + task) * F::kRows, lane, acc);
                    in_head = false;
#pragma unroll
                    for (int r = 0; r < RT; r++)
#pragma unroll
                        for (int n = 0; n < NT; n++)
#pragma unroll
                            for (int c = 0; c < 4; c++)
                                acc[r][n][c] = 0.0f;
                    block = 0;
                    task++;
                }
            }
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    // a share that ends inside the task it began in is a head as a whole
    const bool open = block > 0 && !in_head && u0 < u1;
    if (in_head)
        F::put_head(heads, warp, lane, acc);
    __syncthreads();
    if (open) {
        // the rest of this task lies with the warps behind
        const int end = (task + 1) * p.blocks;
        for (int w = warp + 1; w < NW; w++) {
            const int w0 = static_cast<int>(static_cast<int64_t>(units) * w / NW);
            const int w1 = static_cast<int>(static_cast<int64_t>(units) * (w + 1) / NW);
            if (w0 >= end)
                break;
            if (w0 == w1)
                continue;
#pragma unroll
            for (int r = 0; r < RT; r++)
#pragma unroll
                for (int n = 0; n < NT; n++) {
                    const float4 v = heads[((w * RT + r) * NT + n) * 32 + lane];
                    acc[r][n][0] += v.x;
                    acc[r][n][1] += v.y;
                    acc[r][n][2] += v.z;
                    acc[r][n][3] += v.w;
                }
        }
        F::store(p, t0, static_cast<int64_t>(a + task) * F::kRows, lane, acc);
    }
}

constexpr int kMaxSmem = 227 * 1024;
// Up to here 60 KB are left of L1, in which scales and zeros stay, two bytes a row and group,
// until the rest of their sectors is used; above it 28.  (1 token, 38912 rows, us: groups of 128
// <1, 2, 16, 3> and <1, 2, 16, 2>, K 5632 28.3 and 24.5, K 7040 40.6 and 30.8; <1, 2, 16, 2> and
// <1, 1, 16, 3>, K 8192 45.4 and 42.1; groups of 64 <1, 2, 16, 3> and <1, 1, 16, 2>, K 4096 30.8 and
// 33.0, K 5632 44.8 and 29.8, K 7040 59.9 and 37.9, K 8192 73.4 and 63.0.)
constexpr int kRoomySmem = 195 * 1024;
// Rows from which on linear_few_wide.cu is taken for more than 8 tokens: a task of 128 for each
// SM, two where K is short and the tasks are over soon.  (Here and there, groups of 128, us, 16
// tokens: K 1024, 19456 rows 6.2 and 6.2, 29184 7.2 and 8.1, 77824 12.3 and 12.2; K 2816,
// 14592 10.1 and 10.6, 19456 11.7 and 10.9, 29184 15.8 and 16.1; K 5632, 19456 26.0 and 21.5.
// 32 tokens: K 1024, 19456 8.0 and 8.3; K 2816, 19456 16.7 and 15.3, 29184 23.2 and 21.6; K 5632,
// 14592 34.4 and 30.0.  8 tokens: K 2816, 19456 9.0 and 10.9, 262144 68.3 and 66.6.)
// With groups of 64 a step there has twice the sums to add up: the same rows only where K is
// too long for two tiles of tokens here.  (16 tokens: K 1024, 38912 rows 8.9 and 9.8, 131072 22.1
// and 21.4; K 2816, 29184 16.2 and 18.6, 38912 19.6 and 18.9, 131072 54.5 and 48.2; K 5632, 19456
// 29.3 and 25.1, 38912 52.2 and 39.9; 32 tokens 98.0 and 71.1.)
constexpr int wide_rows(int K, int group)
{
    return group == 128 ? (K >= 2048 ? 128 : 256) : K >= 4096 ? 128 : K >= 2048 ? 256 : 512;
}

template <class F> constexpr int smem_of(int blocks, int nt)
{
    return nt * F::tile_bytes(blocks) + F::kHeadBytes + F::kRingBytes;
}

template <int GROUP, int NT, int RT, int NW, int S>
cudaError_t launch_few_linear_as(const FewLinearArgs &a, int sms, int dev, cudaStream_t stream)
{
    using F = FewLinear<GROUP, NT, RT, NW, S>;
    auto kern = few_linear_kernel<GROUP, NT, RT, NW, S>;
    static std::atomic<uint64_t> raised{0};      // devices whose limit is raised already
    if (!(raised.load(std::memory_order_relaxed) >> (dev & 63) & 1u)) {
        cudaError_t err =
            cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
        if (err != cudaSuccess)
            return err;
        raised.fetch_or(1ull << (dev & 63), std::memory_order_relaxed);
    }
    const int tasks = (a.N + F::kRows - 1) / F::kRows, parts = (a.M + 8 * NT - 1) / (8 * NT);
    const int shares = std::min(tasks, std::max(sms / parts, 1));
    return launch_pdl(kern, dim3(shares * parts), dim3(32 * NW), smem_of<F>(a.blocks, NT), stream, a,
                      parts);
}

constexpr int kMaxBlocks = 11264 / 128;
using Narrowest = FewLinear<64, 1, 1, 16, 2>;
static_assert(smem_of<Narrowest>(kMaxBlocks, 1) <= kMaxSmem);

template <int GROUP>
cudaError_t launch_few_linear_group(const FewLinearArgs &a, int sms, int dev, cudaStream_t stream)
{
    // Tiles of 8 tokens at once: two share the unpacking of the codes.  Two tiles of weight
    // rows share the reading of the activations, where there are enough of them for every SM.
    const int tiles = (a.M + 7) / 8;
    const bool many = a.N >= 64 * sms;
    if (tiles > 1 && many && smem_of<FewLinear<GROUP, 2, 2, 16, 2>>(a.blocks, 2) <= kMaxSmem)
        return launch_few_linear_as<GROUP, 2, 2, 16, 2>(a, sms, dev, stream);
    if (many && smem_of<FewLinear<GROUP, 1, 2, 16, 3>>(a.blocks, 1) <= kRoomySmem)
        return launch_few_linear_as<GROUP, 1, 2, 16, 3>(a, sms, dev, stream);
    if constexpr (GROUP == 128)
        if (many && smem_of<FewLinear<GROUP, 1, 2, 16, 2>>(a.blocks, 1) <= kRoomySmem)
            return launch_few_linear_as<GROUP, 1, 2, 16, 2>(a, sms, dev, stream);
    if (!many && smem_of<FewLinear<GROUP, 1, 1, 16, 4>>(a.blocks, 1) <= kRoomySmem)
        return launch_few_linear_as<GROUP, 1, 1, 16, 4>(a, sms, dev, stream);
    if constexpr (GROUP == 128)
        if (smem_of<FewLinear<GROUP, 1, 1, 16, 3>>(a.blocks, 1) <= kRoomySmem)
            return launch_few_linear_as<GROUP, 1, 1, 16, 3>(a, sms, dev, stream);
    return launch_few_linear_as<GROUP, 1, 1, 16, 2>(a, sms, dev, stream);
}

}  // namespace

cudaError_t launch_few_linear(const FewLinearProblem &q, cudaStream_t stream)
{
    int dev = 0, sms = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err == cudaSuccess)
        err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (err != cudaSuccess)
        return err;
    if (q.N >= wide_rows(q.K, q.group) * sms && few_linear_wide_tokens(q.M, q.K, q.group) > 0)
        return launch_few_linear_wide(q, stream);
    FewLinearArgs a{};
    a.x = q.x;
    a.q = q.q;
    a.s = q.s;
    a.z = q.z;
    a.y = q.y;
    a.dev_status = q.dev_status;
    a.M = q.M;
    a.K = q.K;
    a.N = q.N;
    a.blocks = (q.K + 127) / 128;
    return q.group == 128 ? launch_few_linear_group<128>(a, sms, dev, stream)
                          : launch_few_linear_group<64>(a, sms, dev, stream);
}

}  // namespace w4
