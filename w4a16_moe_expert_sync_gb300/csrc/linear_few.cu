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
// A task is 16 RT weight rows, a unit 128 codes of each.  A CTA takes an equal
// contiguous share of the tasks, its warps equal shares of those tasks' units; a task
// that crosses warps is added up in warp order through shared memory.  Sums run in a
// fixed order: bit-identical reruns.
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

__device__ __forceinline__ uint4 load_codes16(const uint8_t *p)
{
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}
__device__ __forceinline__ uint2 load_codes8(const uint8_t *p)
{
    uint2 v;
    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];"
                 : "=r"(v.x), "=r"(v.y)
                 : "l"(p));
    return v;
}

__device__ __forceinline__ float half_of(uint16_t h) { return __half2float(__ushort_as_half(h)); }

// NT: tiles of 8 tokens; RT: tiles of 16 weight rows; NW: warps; PF: units in flight a warp.
template <int GROUP, int NT, int RT, int NW, int PF>
struct FewLinear {
    static constexpr int kGroups = 128 / GROUP;            // of a unit
    static constexpr int kWords = 4 / kGroups;             // of a lane's row and group
    static constexpr int kRows = 16 * RT;

    // Bytes of a tile of 8 tokens: the activations [block][4][8 tokens][4] x 16 bytes, then
    // the groups' sums [block][groups][8 tokens].
    static __host__ __device__ constexpr int tile_bytes(int blocks)
    {
        return blocks * (4 * 512 + kGroups * 32);
    }

    // A lane's codes, scales and zeros of one unit: of weight rows 2 g and 2 g + 1 of each
    // row tile.
    struct Unit {
        uint32_t q[RT][2][4];
        uint16_t s[RT][2][kGroups], z[RT][2][kGroups];
    };

    static __device__ __forceinline__ void load(const FewLinearArgs &p, int64_t row0, int block,
                                                int lane, Unit &u)
    {
        const int g = lane >> 2, t4 = lane & 3, G = p.K / GROUP;
#pragma unroll
        for (int r = 0; r < RT; r++)
#pragma unroll
            for (int i = 0; i < 2; i++) {
                // rows past the last one repeat it; what they give is not stored
                const int64_t row = min(row0 + r * 16 + 2 * g + i, static_cast<int64_t>(p.N) - 1);
                const uint8_t *q = p.q + row * (p.K / 2) + block * 64;
                if constexpr (GROUP == 128) {
                    const uint4 v = load_codes16(q + t4 * 16);
                    u.q[r][i][0] = v.x;
                    u.q[r][i][1] = v.y;
                    u.q[r][i][2] = v.z;
                    u.q[r][i][3] = v.w;
                } else {
#pragma unroll
                    for (int h = 0; h < 2; h++) {
                        uint2 v = make_uint2(0, 0);
                        if (block * 2 + h < G)
                            v = load_codes8(q + h * 32 + t4 * 8);
                        u.q[r][i][2 * h] = v.x;
                        u.q[r][i][2 * h + 1] = v.y;
                    }
                }
#pragma unroll
                for (int h = 0; h < kGroups; h++) {
                    const int64_t at = row * G + block * kGroups + h;
                    const bool in = kGroups == 1 || block * kGroups + h < G;
                    u.s[r][i][h] = in ? __ldg(p.s + at) : static_cast<uint16_t>(0);
                    u.z[r][i][h] = in ? __ldg(p.z + at) : static_cast<uint16_t>(0);
                }
            }
    }

    static __device__ __forceinline__ void add(const uint8_t *xs, int tile_stride, int blocks,
                                               int block, int lane, const Unit &u,
                                               float (&acc)[RT][NT][4])
    {
        const int t4 = lane & 3;
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
                    const uint32_t w0 = u.q[r][0][j], w1 = u.q[r][1][j];
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
#pragma unroll
            for (int n = 0; n < NT; n++) {
                const float2 sum = *reinterpret_cast<const float2 *>(
                    xs + n * tile_stride + blocks * 2048 + (block * kGroups + h) * 32 + t4 * 8);
#pragma unroll
                for (int r = 0; r < RT; r++)
#pragma unroll
                    for (int i = 0; i < 2; i++) {
                        const float s = half_of(u.s[r][i][h]), z = half_of(u.z[r][i][h]);
                        float *a = &acc[r][n][2 * i];
                        a[0] = fmaf(s, fmaf(-z, sum.x, part[r][n][2 * i]), a[0]);
                        a[1] = fmaf(s, fmaf(-z, sum.y, part[r][n][2 * i + 1]), a[1]);
                    }
            }
        }
    }

    // Activations t0 .. t0 + 8 NT of x into shared memory, in the order of the codes, with
    // their groups' sums; tokens past the last and columns past K are zero.
    static __device__ void stage(const FewLinearArgs &p, int t0, uint8_t *xs, int tile_stride)
    {
        const int words = p.blocks * 16, lane = threadIdx.x & 31;
        const int items = 8 * NT * words;
        for (int i0 = threadIdx.x - lane; i0 < items; i0 += 32 * NW) {
            const int i = i0 + lane, tok = i / words, word = i - tok * words;
            const int t = t0 + tok;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (t < p.M && word * 8 < p.K)
                v = __ldg(reinterpret_cast<const uint4 *>(p.x + static_cast<int64_t>(t) * p.K +
                                                          word * 8));
            const uint32_t in[4] = {v.x, v.y, v.z, v.w};
            float f[8], sum = 0.0f;
#pragma unroll
            for (int e = 0; e < 4; e++) {
                f[2 * e] = __uint_as_float(in[e] << 16);
                f[2 * e + 1] = __uint_as_float(in[e] & 0xFFFF0000u);
            }
#pragma unroll
            for (int e = 0; e < 8; e++)
                sum += f[e];
            uint4 out;
            out.x = bf16_pair(f[0] * kUp, f[4] * kUp);
            out.y = bf16_pair(f[2] * kUp, f[6] * kUp);
            out.z = bf16_pair(f[1] * kUpHigh, f[5] * kUpHigh);
            out.w = bf16_pair(f[3] * kUpHigh, f[7] * kUpHigh);
            // words of a group in the order of the lanes that hold their codes
            constexpr int kLaneWords = kWords;
            const int block = word / 16, h = word % 16 / (16 / kGroups);
            const int in_group = word % (16 / kGroups), t4 = in_group / kLaneWords;
            const int j = h * kLaneWords + in_group % kLaneWords;
            uint8_t *tile = xs + (tok >> 3) * tile_stride;
            *reinterpret_cast<uint4 *>(tile + (block * 4 + j) * 512 + (tok & 7) * 64 + t4 * 16) = out;
#pragma unroll
            for (int o = 8 / kGroups; o > 0; o >>= 1)
                sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (in_group == 0)
                *reinterpret_cast<float *>(tile + p.blocks * 2048 + (block * kGroups + h) * 32 +
                                           (tok & 7) * 4) = sum * kSum;
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
                        *reinterpret_cast<uint32_t *>(y) = v;
                    } else {
                        if (row < p.N)
                            y[0] = static_cast<uint16_t>(v);
                        if (row + 1 < p.N)
                            y[1] = static_cast<uint16_t>(v >> 16);
                    }
                }
            }
    }
};

template <int GROUP, int NT, int RT, int NW, int PF>
__global__ void __launch_bounds__(32 * NW, 1) few_linear_kernel(const FewLinearArgs p)
{
    using F = FewLinear<GROUP, NT, RT, NW, PF>;
    extern __shared__ __align__(16) uint8_t xs[];
    const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
    const int tile_stride = F::tile_bytes(p.blocks);
    // each warp's sums of the task that another one began
    float4 *heads = reinterpret_cast<float4 *>(xs + NT * tile_stride);
    const int tasks = (p.N + F::kRows - 1) / F::kRows;
    const int a = static_cast<int>(static_cast<int64_t>(tasks) * blockIdx.x / gridDim.x);
    const int e = static_cast<int>(static_cast<int64_t>(tasks) * (blockIdx.x + 1) / gridDim.x);
    const int units = (e - a) * p.blocks;                  // below 2^31: blocks <= 104
    const int u0 = static_cast<int>(static_cast<int64_t>(units) * warp / NW);
    const int u1 = static_cast<int>(static_cast<int64_t>(units) * (warp + 1) / NW);
    pdl_wait();
    pdl_trigger();
    for (int t0 = 0; t0 < p.M; t0 += 8 * NT) {
        typename F::Unit ring[PF];
        // the next unit to request, the next to add
        int ask = u0, ask_task = u0 / p.blocks, ask_block = u0 - ask_task * p.blocks;
        int task = ask_task, block = ask_block;
        auto request = [&](typename F::Unit &u) {
            if (ask < u1)
                F::load(p, static_cast<int64_t>(a + ask_task) * F::kRows, ask_block, lane, u);
            ask++;
            if (++ask_block == p.blocks) {
                ask_block = 0;
                ask_task++;
            }
        };
#pragma unroll
        for (int i = 0; i < PF; i++)
            request(ring[i]);
        F::stage(p, t0, xs, tile_stride);
        __syncthreads();
        float acc[RT][NT][4] = {};
        bool in_head = block > 0 && u0 < u1;       // another warp has the task's first part
        for (int u = u0; u < u1;) {
#pragma unroll
            for (int i = 0; i < PF; i++) {
                if (u < u1) {
                    F::add(xs, tile_stride, p.blocks, block, lane, ring[i], acc);
                    request(ring[i]);
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
        __syncthreads();                   // the sums have been read: the next tokens may come
    }
}

constexpr int kMaxSmem = 227 * 1024;
constexpr int kMaxBlocks = 13568 / 128;
using Narrowest = FewLinear<64, 1, 1, 16, 3>;
static_assert(Narrowest::tile_bytes(kMaxBlocks) + Narrowest::kHeadBytes <= kMaxSmem);

template <int GROUP, int NT, int RT, int NW, int PF>
cudaError_t launch_few_linear_as(const FewLinearArgs &a, int sms, int dev, cudaStream_t stream)
{
    using F = FewLinear<GROUP, NT, RT, NW, PF>;
    auto kern = few_linear_kernel<GROUP, NT, RT, NW, PF>;
    static std::atomic<uint64_t> raised{0};      // devices whose limit is raised already
    if (!(raised.load(std::memory_order_relaxed) >> (dev & 63) & 1u)) {
        cudaError_t err =
            cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
        if (err != cudaSuccess)
            return err;
        raised.fetch_or(1ull << (dev & 63), std::memory_order_relaxed);
    }
    const int tasks = (a.N + F::kRows - 1) / F::kRows;
    const int smem = NT * F::tile_bytes(a.blocks) + F::kHeadBytes;
    return launch_pdl(kern, dim3(std::min(tasks, sms)), dim3(32 * NW), smem, stream, a);
}

// Whether the instance's tokens fit shared memory at once.
template <class F> bool fits(int blocks, int nt)
{
    return nt * F::tile_bytes(blocks) + F::kHeadBytes <= kMaxSmem;
}

template <int GROUP>
cudaError_t launch_few_linear_group(const FewLinearArgs &a, int sms, int dev, cudaStream_t stream)
{
    // as many tiles of 8 tokens at once as there are and as fit; with more the weights
    // are read again
    const int tiles = (a.M + 7) / 8;
    if (tiles > 2 && fits<FewLinear<GROUP, 4, 2, 8, 3>>(a.blocks, 4))
        return launch_few_linear_as<GROUP, 4, 2, 8, 3>(a, sms, dev, stream);
    if (tiles > 1 && fits<FewLinear<GROUP, 2, 2, 16, 2>>(a.blocks, 2))
        return launch_few_linear_as<GROUP, 2, 2, 16, 2>(a, sms, dev, stream);
    return launch_few_linear_as<GROUP, 1, 1, 16, 3>(a, sms, dev, stream);
}

}  // namespace

cudaError_t launch_few_linear(const uint16_t *x, int M, int K, int N, const uint8_t *q,
                              const uint16_t *s, const uint16_t *z, int group, uint16_t *y,
                              cudaStream_t stream)
{
    int dev = 0, sms = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err == cudaSuccess)
        err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (err != cudaSuccess)
        return err;
    FewLinearArgs a{};
    a.x = x;
    a.q = q;
    a.s = s;
    a.z = z;
    a.y = y;
    a.M = M;
    a.K = K;
    a.N = N;
    a.blocks = (K + 127) / 128;
    return group == 128 ? launch_few_linear_group<128>(a, sms, dev, stream)
                        : launch_few_linear_group<64>(a, sms, dev, stream);
}

}  // namespace w4
