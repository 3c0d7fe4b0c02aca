// attention.cu -- attention over a paged cache for a batch whose sequences
// share a prefix, the prefix computed once for all of them:
//   o = sum_l p_l v_l / sum_l p_l,  p_l = exp(scale q.k_l - m)
// over the keys l that a query sees.
//
// Per kv head, the queries of a whole group of sequences (and of the query
// heads that share the kv head) are the rows of one matrix against the
// prefix's keys; each sequence's own rows meet only its own keys.  Both kinds
// of work are the same tile step, S = Q K^T and O += P V on tcgen05 with 128
// rows x 128 keys, so a K or V tile is read from HBM once whatever the number
// of rows, and a step with few valid rows costs no more than the memory time
// of its 64 KB tile.
//
// An entry is a group's prefix or a sequence's own keys; an item is an entry's
// row tile for one kv head.  Entries of more than 128 rows are taken as pairs:
// two 128-row tiles of one CTA against the same K and V tile.  The tiles of
// all pair items laid end to end are split evenly over some of the CTAs, those of
// all single items over the others' two streams, wherever item borders fall; each
// piece leaves unnormalised sums with their maximum and denominator, which a
// second kernel joins per row.  So one long prefix fills the GPU as evenly as
// a thousand short ones.  The split follows from the lengths, which live on
// the device: every CTA works it out for itself (a scan over the entries).
//
// Roles of a CTA's twelve warps: warps 0-3 and 4-7 are the softmax of streams
// 0 and 1 (a thread per row), warp 8 loads K and V by TMA into a ring of
// slots, warps 9 and 10 issue the MMAs (of both streams of a pair; of streams 0
// and 1), warp 11 only completes its group of four.  While one stream's softmax
// runs the tensor cores work for the other.
//
// Bounds and measured times (GB300, both kernels, back to back in a graph):
//   32 questions about 120,000 shared tokens, 32/4 heads of 128: 69 us; 257 MB
//     (38 us at the copy bandwidth), 63 GFLOP (32 us).  The pairs' loop takes
//     some 3000 cycles a tile; its MMAs take 2048, and so do the 256 KB that it
//     moves through shared memory (their operands, and K and V as they land).
//     Without the exponentials it is 1 to 3 % faster: the softmax does not pace it
//   64 sequences of 33 to 1500 tokens behind 8192: 59 us; 242 MB (36 us).  Plan 4 us,
//     first tile 6, change of piece 1.5 each, join and its launch 6
//   four times 256 queries over 4096 + 256: 46 us; 37 GFLOP (19 us), the pairs' loop
//   two sequences of 240 tokens: 14 us, all of it plan, one tile and join
#include <algorithm>
#include <atomic>
#include <climits>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/w4moe.h"
#include "attention_plan.cuh"
#include "checks.cuh"
#include "launch.h"
#include "ptx.cuh"

namespace w4 {

namespace {

using plan::kItemCost;
using plan::kKeys;
using plan::kRows;
using plan::pair_ctas;
using plan::worker_begin;
using plan::worker_of;

constexpr int kThreads = 32 * 12;
// Registers a thread: 168 at launch; the loading warps give some of theirs to
// the softmax warps, which hold a row of 128 scores (2 x 216 + 72 = 3 x 168).
constexpr int kSoftmaxRegs = 216, kOtherRegs = 72;

// A group's prefix (first G) or a sequence's own keys.
struct Entry {
    int place, item0;                      // length and items before it, in its region
    int span;                              // of one item: kItemCost + tiles; 0: nothing
    int row_tiles;                         // items per kv head
    int pair;
    int row;                               // a sequence's first row among its group's
};

// What the joining kernel needs to know of a sequence.
struct alignas(16) Joint {
    int tok0, tokens;                      // tokens < 0: nothing to write
    int all[2];                            // length of the single [0] and pair [1] region
    int workers[2];                        // and among how many it is split
    Entry e[2];                            // of its group's prefix and of its own keys
};

// A worker's piece of one item.
struct Seg {
    int row_of_table, kbase;               // where its keys are: absolute position of tile 0
    int k0, k1;                            // the entry's keys
    int tile0, tiles;                      // this piece's tiles
    int row0, rows;                        // its rows (of the entry), both streams' in a pair
    int tok0;                              // the entry's first token
    int seq;                               // the sequence, or -1 for a group's prefix
    int head;                              // kv head
    int piece;                             // where its sums go; -1: nowhere
};

// How TMA sees the pages.  kRows: values, tokens, heads, pages; a box is 64 values of
// each of a page's tokens, and the 64-value blocks of a K or V tile lie one after the
// other.  Pages of kShortPage tokens with more than one such block have a box with all
// of them, which lie in turn there, 8 tokens each: half as many boxes.  (128 sequences
// of 6000 tokens in pages of 16, one kv and two query heads of 128, 396 MB: 104 us by
// kRows, 87 like this; larger pages gain nothing.)  The axes are then 64 values, 8 tokens,
// blocks, the page's groups of 8 tokens and one more: with the heads side by side their blocks are one axis, with
// the heads of all pages evenly spaced they are one axis with the pages; else
// (kGroups) a box is 8 tokens.
enum class PageView { kRows, kHeadsAsBlocks, kHeadsAsPages, kGroups };
constexpr int kShortPage = 16;

struct AttnArgs {
    CUtensorMap k_map, v_map;              // see PageView
    const uint16_t *q;
    uint16_t *out;
    const int32_t *table, *lens, *q_offsets, *group_offsets, *shared;
    int32_t *status;
    Seg *segs;                      // workspace: the pieces of all workers
    Joint *joints;                         // workspace: [B], for the joining kernel
    // workspace: the sums of pieces of pairs, of single items of groups and of
    // sequences, and their rows' maximum and denominator
    float *part[3];
    float2 *ml[3];
    int64_t q_tok, q_head;
    float scale_log2;
    uint64_t wait_ns;
    int withhold;                          // test hook: slot 0's barrier never completes
    int T, B, G, W, P, page, page_shift, Hq, Hkv, rep, max_q, causal;
    PageView view;
    int rows_b;                            // a sequence's single item's rows at most
    int cap_a, cap_g, cap_b;               // pieces that the workspace holds; cap_b: all single
};

// ------------------------------------------------------------- tensor memory
// All 128 columns of this thread's lane, and the wait for them.
__device__ __forceinline__ void tmem_ld_32x32b_x128(uint32_t taddr, uint32_t (&r)[128])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x128.b32 {"
        "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, "
        "%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
        "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63, "
        "%64, %65, %66, %67, %68, %69, %70, %71, %72, %73, %74, %75, %76, %77, %78, %79, "
        "%80, %81, %82, %83, %84, %85, %86, %87, %88, %89, %90, %91, %92, %93, %94, %95, "
        "%96, %97, %98, %99, %100, %101, %102, %103, %104, %105, %106, %107, %108, %109, %110, %111, "
        "%112, %113, %114, %115, %116, %117, %118, %119, %120, %121, %122, %123, %124, %125, %126, %127}, [%128];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
          "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]),
          "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
          "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
          "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63]),
          "=r"(r[64]), "=r"(r[65]), "=r"(r[66]), "=r"(r[67]), "=r"(r[68]), "=r"(r[69]), "=r"(r[70]), "=r"(r[71]),
          "=r"(r[72]), "=r"(r[73]), "=r"(r[74]), "=r"(r[75]), "=r"(r[76]), "=r"(r[77]), "=r"(r[78]), "=r"(r[79]),
          "=r"(r[80]), "=r"(r[81]), "=r"(r[82]), "=r"(r[83]), "=r"(r[84]), "=r"(r[85]), "=r"(r[86]), "=r"(r[87]),
          "=r"(r[88]), "=r"(r[89]), "=r"(r[90]), "=r"(r[91]), "=r"(r[92]), "=r"(r[93]), "=r"(r[94]), "=r"(r[95]),
          "=r"(r[96]), "=r"(r[97]), "=r"(r[98]), "=r"(r[99]), "=r"(r[100]), "=r"(r[101]), "=r"(r[102]), "=r"(r[103]),
          "=r"(r[104]), "=r"(r[105]), "=r"(r[106]), "=r"(r[107]), "=r"(r[108]), "=r"(r[109]), "=r"(r[110]), "=r"(r[111]),
          "=r"(r[112]), "=r"(r[113]), "=r"(r[114]), "=r"(r[115]), "=r"(r[116]), "=r"(r[117]), "=r"(r[118]), "=r"(r[119]),
          "=r"(r[120]), "=r"(r[121]), "=r"(r[122]), "=r"(r[123]), "=r"(r[124]), "=r"(r[125]), "=r"(r[126]), "=r"(r[127])
        : "r"(taddr)
        : "memory");
}

// D (+)= A B^T with both operands in shared memory, by one elected lane.
__device__ __forceinline__ void mma_ss_elect(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                             uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

// A 128-byte-swizzled operand whose contiguous axis is N (V: a token's
// values): 64 values x 8 tokens to an atom of 1024 bytes, 8-token groups
// `group` bytes apart, 64-value blocks `block` bytes apart.  It does for K as well,
// whose contiguous axis is the contraction: there blocks are operands of their own.
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t addr, uint32_t group, uint32_t block)
{
    uint64_t d = 0;
    d |= static_cast<uint64_t>((addr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(block >> 4) << 16;
    d |= static_cast<uint64_t>(group >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(2) << 61;
    return d;
}

__device__ __forceinline__ void tma_load_5d(void *dst, const CUtensorMap *map, int x, int y, int z,
                                            int u, int v, uint64_t *bar)
{
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(u), "r"(v),
        "r"(smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ void tma_load_4d(void *dst, const CUtensorMap *map, int x, int y, int z,
                                            int w, uint64_t *bar)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ void cp_async_wait_all()
{
    asm volatile("cp.async.wait_all;" ::: "memory");
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two fp32 values in a register pair, and the paired operations.
__device__ __forceinline__ uint64_t pair_of(uint32_t lo, uint32_t hi)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
    return r;
}
__device__ __forceinline__ uint64_t both(float x)
{
    return pair_of(__float_as_uint(x), __float_as_uint(x));
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

__device__ __forceinline__ float low(uint64_t x) { return __uint_as_float(static_cast<uint32_t>(x)); }
__device__ __forceinline__ float high(uint64_t x)
{
    return __uint_as_float(static_cast<uint32_t>(x >> 32));
}

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

template <bool BF16> __device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    uint32_t r;
    if constexpr (BF16)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// -------------------------------------------------------------------- plan
// The index arrays as the plan reads them: staged in shared memory, for its
// searches are chains of dependent reads.
struct Index {
    const int *lens, *q_offsets, *group_offsets, *shared;
};

// The shared length of group g, never beyond its first sequence.
__device__ __forceinline__ int shared_of(const AttnArgs &p, const Index &x, int g)
{
    const int first = x.group_offsets[g];
    if (first < 0 || first >= p.B)
        return 0;
    return max(0, min(min(x.shared[g], x.lens[first]), p.W * p.page));
}

// The group of sequence b, or -1: the last whose first sequence is <= b, if
// b lies before its end.
__device__ __forceinline__ int group_of(const AttnArgs &p, const Index &x, int b)
{
    int lo = 0, hi = p.G - 1;
    if (p.G == 0 || x.group_offsets[0] > b)
        return -1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (x.group_offsets[mid] <= b)
            lo = mid;
        else
            hi = mid - 1;
    }
    return b < x.group_offsets[lo + 1] ? lo : -1;
}

// Rows of a piece's place: of a pair, a group's single item, a sequence's.
__device__ __forceinline__ int rows_of(const AttnArgs &p, int kind)
{
    return kind == 0 ? 2 * kRows : kind == 1 ? kRows : p.rows_b;
}

// An entry's queries and keys, and its items: span is an item's length in the
// split (kItemCost + tiles; 0: nothing to do), items of one kv head.
struct Work {
    int tok0, tokens, k0, k1;
    int span, row_tiles_pair;              // 2 row_tiles + pair
    __device__ __forceinline__ int row_tiles() const { return row_tiles_pair >> 1; }
    __device__ __forceinline__ bool pair() const { return row_tiles_pair & 1; }
};

// What entry e asks for.  More than max_q tokens a sequence: nothing.  Offsets
// that do not ascend within their bounds set bad.
__device__ __forceinline__ Work work_of(const AttnArgs &p, const Index &x, int e, bool flag,
                                        bool &bad)
{
    Work w{};
    int members = 1;
    if (e < p.G) {
        const int b0 = x.group_offsets[e], b1 = x.group_offsets[e + 1];
        if (b0 < 0 || b1 < b0 || b1 > p.B) {
            bad = true;
            return w;
        }
        w.tok0 = x.q_offsets[b0];
        w.tokens = x.q_offsets[b1] - w.tok0;
        w.k1 = b1 > b0 ? shared_of(p, x, e) : 0;
        members = b1 - b0;
    } else {
        const int b = e - p.G, g = group_of(p, x, b), len = x.lens[b];
        const int t0 = x.q_offsets[b], t1 = x.q_offsets[b + 1];
        if (t0 < 0 || t1 < t0 || t1 > p.T) {
            bad = true;
            return w;
        }
        w.tok0 = t0;
        w.tokens = t1 - t0;
        w.k1 = min(max(len, 0), p.W << p.page_shift);
        w.k0 = g >= 0 ? min(shared_of(p, x, g), w.k1) : 0;
        if (w.k1 != len && flag && p.status)
            atomicOr(p.status, W4_DEV_BAD_SLOT);
    }
    if (w.tokens > static_cast<int64_t>(members) * p.max_q) {
        w.tokens = 0;
        if (flag && p.status)
            atomicOr(p.status, W4_DEV_BAD_SLOT);
    }
    const int rows = w.tokens * p.rep;
    if (rows > 0 && w.k1 > w.k0) {
        w.span = plan::key_tiles(w.k0, w.k1, p.page_shift) + kItemCost;
        w.row_tiles_pair = 2 * plan::row_tiles(rows) + plan::is_pair(rows);
    }
    return w;
}

// Exclusive sums of four counts over the CTA's threads; whether any thread is
// bad comes with the same barrier.
__device__ __forceinline__ int4 scan4(int4 v, int4 *sums, int4 *total, bool *bad)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int4 s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, s.x, o), y = __shfl_up_sync(0xffffffffu, s.y, o);
        const int z = __shfl_up_sync(0xffffffffu, s.z, o), w = __shfl_up_sync(0xffffffffu, s.w, o);
        if (lane >= o) {
            s.x += x;
            s.y += y;
            s.z += z;
            s.w += w;
        }
    }
    if (lane == 31)
        sums[warp] = s;
    *bad = __syncthreads_or(*bad);
    int4 before = make_int4(0, 0, 0, 0), all = before;
    for (int i = 0; i < kThreads / 32; i++) {
        const int4 u = sums[i];
        if (i < warp) {
            before.x += u.x;
            before.y += u.y;
            before.z += u.z;
            before.w += u.w;
        }
        all.x += u.x;
        all.y += u.y;
        all.z += u.z;
        all.w += u.w;
    }
    *total = all;
    return make_int4(before.x + s.x - v.x, before.y + s.y - v.y, before.z + s.z - v.z,
                     before.w + s.w - v.w);
}

// The entry that tile (or item) x of a region belongs to: the last with a
// running count <= x, for entries with nothing in the region carry the count
// on and the owner's successor has more than x.
__device__ __forceinline__ int find_entry(const int *start, int n, int x)
{
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (start[mid] <= x)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// IN_TURN: a K or V tile's blocks of 64 values lie in turn (see PageView).
template <int D, bool BF16, bool IN_TURN>
struct Kernel {
    static constexpr int kBlocks = D / 64;                     // 128-byte column blocks
    static constexpr int kTileBytes = kKeys * D * 2;           // a K, V or Q tile
    // bytes from 8 of a K or V tile's tokens to the next, from a block to the next
    static constexpr int kGroup = IN_TURN ? 1024 * kBlocks : 1024;
    static constexpr int kBlock = IN_TURN ? 1024 : kKeys * 128;
    static constexpr int kSlots = 160 * 1024 / kTileBytes;
    static constexpr int kQBytes = 2 * kTileBytes;
    static constexpr int kRingBytes = kSlots * kTileBytes;
    static constexpr size_t kSmem = 1024 + kQBytes + kRingBytes;
    static constexpr uint32_t kS = 0, kO = 256;                // TMEM columns of stream 0
    static constexpr uint32_t kQk = idesc_16bit_f32(128, kKeys, BF16);
    static constexpr uint32_t kPv = idesc_16bit_f32(128, D, BF16) | (1u << 16);   // V is N-major

    struct Shared {
        alignas(8) uint64_t full[kSlots], empty[kSlots];
        uint64_t q_ready[2], s_full[2], p_ready[2], o_full[2], cleared, drained[2];
        uint32_t tmem;
        int abort_flag;
        int requested;                         // fills requested of the ring so far
        int seg0[3], segs[3], tiles[3];        // single items of streams 0 and 1; pairs
        Seg first[3];                          // the first piece of each
        int4 sums[kThreads / 32];
    };

    // The plan: this CTA's pieces into the workspace, the first ones also into
    // shared memory.  Scratch is the queries' room and the ring (192 KB at least,
    // 48 bytes an entry), before anything is loaded into them.
    static __device__ void make_plan(const AttnArgs &p, Shared &s, uint8_t *scratch)
    {
        const int n = p.G + p.B, tid = threadIdx.x;
        Work *work = reinterpret_cast<Work *>(scratch);                // [n]
        // running counts before each entry: length and items, singles and pairs
        int *start = reinterpret_cast<int *>(work + n);                // [4][n]
        int *lens = start + 4 * n, *qo = lens + p.B, *go = qo + p.B + 1, *sh = go + p.G + 1;
        for (int i = tid; i <= p.B; i += kThreads) {
            qo[i] = p.q_offsets[i];
            if (i < p.B)
                lens[i] = p.lens[i];
        }
        for (int i = tid; i <= p.G && p.G > 0; i += kThreads) {
            go[i] = p.group_offsets[i];
            if (i < p.G)
                sh[i] = p.shared[i];
        }
        __syncthreads();
        const Index x{lens, qo, go, sh};
        const int run = (n + kThreads - 1) / kThreads, e0 = min(n, tid * run);
        const int e1 = min(n, e0 + run);
        int4 sum = make_int4(0, 0, 0, 0);
        bool bad = false;
        for (int e = e0; e < e1; e++) {
            const Work w = work_of(p, x, e, blockIdx.x == 0, bad);
            const int items = w.row_tiles() * p.Hkv;
            work[e] = w;
            (w.pair() ? sum.z : sum.x) += items * w.span;
            (w.pair() ? sum.w : sum.y) += items;
        }
        int4 total;
        int4 at = scan4(sum, s.sums, &total, &bad);
        if (bad) {                             // nothing is done
            total = make_int4(0, 0, 0, 0);
            if (tid == 0 && blockIdx.x == 0 && p.status)
                atomicOr(p.status, W4_DEV_BAD_SLOT);
        }
        for (int e = e0; e < e1; e++) {
            const Work w = work[e];
            const int items = w.row_tiles() * p.Hkv;
            start[e] = at.x;
            start[n + e] = at.y;
            start[2 * n + e] = at.z;
            start[3 * n + e] = at.w;
            (w.pair() ? at.z : at.x) += items * w.span;
            (w.pair() ? at.w : at.y) += items;
        }
        __syncthreads();
        auto placed = [&](int e) {
            const Work w = work[e];
            Entry en{};
            en.span = w.span;
            en.row_tiles = w.row_tiles();
            en.pair = w.pair();
            en.place = start[(en.pair ? 2 * n : 0) + e];
            en.item0 = start[(en.pair ? 3 * n : n) + e];
            return en;
        };
        const int for_pairs = pair_ctas(total.x, total.z, gridDim.x);
        const int for_singles = gridDim.x - for_pairs;
        // warps 0, 1 and 2 work out the pieces of streams 0 and 1 and of the pairs
        const int which = tid >> 5, lane = tid & 31;
        if (which < 3) {
            const bool pair = which == 2;
            const int all = pair ? total.z : total.x, cta = blockIdx.x;
            const int workers = pair ? for_pairs : min(all, 2 * for_singles);
            // one stream of every CTA before the other
            const int w = pair ? cta : cta < for_pairs ? workers
                                                       : which * for_singles + cta - for_pairs;
            const int *ts = start + (pair ? 2 * n : 0), *is = start + (pair ? 3 * n : n);
            int first = 0, count = 0, lo = 0, hi = 0;
            if (w < workers) {
                lo = worker_begin(all, workers, w);
                hi = worker_begin(all, workers, w + 1);
                // lane 0 finds the first tile's item, lane 1 the last's
                const int at = lane == 0 ? lo : hi - 1, e = find_entry(ts, n, at);
                const int item = is[e] + (at - ts[e]) / work[e].span;
                first = __shfl_sync(0xffffffffu, item, 0);
                count = __shfl_sync(0xffffffffu, item, 1) - first + 1;
            }
            // pieces are numbered by item + worker, which no two share
            Seg *segs = p.segs + (pair ? p.cap_b : 0);
            if (first + w + count > (pair ? p.cap_a : p.cap_b)) {
                count = 0;
                if (lane == 0 && p.status)
                    atomicOr(p.status, W4_DEV_BAD_SLOT);
            }
            int mine = 0;
            for (int i = lane; i < count; i += 32) {
                const int item = first + i, e = find_entry(is, n, item);
                const Work wa = work[e];
                const int local = item - is[e];
                const int t0 = ts[e] + local * wa.span + kItemCost;   // its first tile's place
                Seg g;
                g.seq = e < p.G ? -1 : e - p.G;
                g.row_of_table = e < p.G ? x.group_offsets[e] : e - p.G;
                g.k0 = wa.k0;
                g.k1 = wa.k1;
                g.kbase = wa.k0 >> p.page_shift << p.page_shift;
                g.tok0 = wa.tok0;
                g.head = pair ? local / wa.row_tiles() : local;
                const int step = (pair ? 2 : 1) * kRows;
                g.row0 = (local - g.head * wa.row_tiles()) * step;
                g.rows = min(step, wa.tokens * p.rep - g.row0);
                g.tile0 = max(lo - t0, 0);
                int end = min(hi - t0, wa.span - kItemCost);
                if (p.causal && g.seq >= 0)
                    end = min(end, plan::causal_tiles(wa.k1, wa.tokens, g.kbase,
                                                      g.row0 + g.rows - 1, p.rep));
                g.tiles = max(end - g.tile0, 0);
                g.piece = item + w;
                if (W4_IN_BOUNDS(g.piece >= 0 && g.piece < (pair ? p.cap_a : p.cap_b), p.status))
                    segs[g.piece] = g;
                if (i == 0)
                    s.first[which] = g;
                mine += g.tiles;
            }
            mine = __reduce_add_sync(0xffffffffu, mine);
            if (lane == 0) {
                s.seg0[which] = first + w;
                s.segs[which] = count;
                s.tiles[which] = mine;
            }
        } else {
            // the others tell the joining kernel of the sequences, a share per CTA
            for (int b = blockIdx.x + (tid - 96) * gridDim.x; b < p.B;
                 b += (kThreads - 96) * gridDim.x) {
                Joint j{};
                j.tok0 = qo[b];
                j.tokens = !bad && qo[b + 1] - qo[b] <= p.max_q ? qo[b + 1] - qo[b] : -1;
                j.all[0] = total.x;
                j.all[1] = total.z;
                j.workers[0] = min(total.x, 2 * for_singles);
                j.workers[1] = for_pairs;
                const int g = bad ? -1 : group_of(p, x, b);
                if (g >= 0) {
                    j.e[0] = placed(g);
                    j.e[0].row = (qo[b] - qo[go[g]]) * p.rep;
                }
                if (!bad)
                    j.e[1] = placed(p.G + b);
                p.joints[b] = j;
            }
        }
        __syncthreads();
    }

    static __device__ __forceinline__ int fill_of(const Shared &s, int which, int r)
    {
        return plan::fill_of(s.tiles[0], s.tiles[1], which, r);
    }

    // Every wait has a limit.  A role whose wait gives up, by the limit or because
    // another's has, returns without a further copy, MMA or store; what is under
    // way by then is awaited before tensor memory is freed and the CTA ends (issuer,
    // softmax, land).
    static __device__ __forceinline__ bool wait(const AttnArgs &p, Shared &s, uint64_t *bar,
                                                uint32_t parity)
    {
        return mbar_wait_warp(bar, parity, &s.abort_flag, p.status, kDevPipelineTimeout,
                              p.wait_ns);
    }

    // Fill `fill` has landed.  A slot's fills may alternate between the streams,
    // so this one may be awaited while the slot's last, the other stream's, has
    // yet to land; by its parity alone that would pass for landed.  Hence first
    // the count of fills requested: when this one has been, the slot's last has
    // been used, and the parity says what it means.
    static __device__ __forceinline__ bool wait_full(const AttnArgs &p, Shared &s, int fill)
    {
        volatile int *requested = &s.requested, *abort_flag = &s.abort_flag;
        if (!__all_sync(0xffffffffu, *requested > fill)) {
            const uint64_t t0 = global_timer_ns();
            for (uint32_t it = 1; !__all_sync(0xffffffffu, *requested > fill); it++) {
                __nanosleep(20);
                if ((it & 63u) == 0) {
                    if (__any_sync(0xffffffffu, *abort_flag != 0))
                        return false;
                    const bool late = global_timer_ns() - t0 > p.wait_ns;
                    if (__any_sync(0xffffffffu, late)) {
                        if ((threadIdx.x & 31) == 0) {
                            *abort_flag = 1;
                            if (p.status)
                                atomicOr(p.status, kDevPipelineTimeout);
                        }
                        return false;
                    }
                }
            }
        }
        return wait(p, s, &s.full[fill % kSlots], (fill / kSlots) & 1);
    }

    // One look at whether fill `fill` has landed.
    static __device__ __forceinline__ bool landed(Shared &s, int fill)
    {
        volatile int *requested = &s.requested;
        return __all_sync(0xffffffffu, *requested > fill) &&
               __all_sync(0xffffffffu, mbar_try_wait(&s.full[fill % kSlots], (fill / kSlots) & 1));
    }

    // ------------------------------------------------------------- loading
    static __device__ bool load_slot(const AttnArgs &p, Shared &s, uint8_t *ring, int fill,
                                     const CUtensorMap *map, int head, int page_id,
                                     int lane)
    {
        const int slot = fill % kSlots, use = fill / kSlots;
        if (use > 0 && !wait(p, s, &s.empty[slot], (use - 1) & 1))
            return false;
        uint8_t *dst = ring + slot * kTileBytes;
        if (lane == 0) {
            mbar_arrive_expect_tx(&s.full[slot], kTileBytes);
            __threadfence_block();
            *static_cast<volatile int *>(&s.requested) = fill + 1;
        }
        __syncwarp();
        if constexpr (IN_TURN) {
            const int tok = p.view == PageView::kGroups ? lane * 8 : lane << p.page_shift;
            const int pg = __shfl_sync(0xffffffffu, page_id, (tok & (kKeys - 1)) >> p.page_shift);
            uint8_t *to = dst + tok / 8 * kGroup;
            if (tok >= kKeys)
                ;
            else if (p.view == PageView::kHeadsAsBlocks)
                tma_load_5d(to, map, 0, 0, head * kBlocks, 0, pg, &s.full[slot]);
            else if (p.view == PageView::kHeadsAsPages)
                tma_load_5d(to, map, 0, 0, 0, 0, pg * p.Hkv + head, &s.full[slot]);
            else
                tma_load_5d(to, map, 0, tok & (p.page - 1), 0, head, pg, &s.full[slot]);
        } else {
            const int boxes = kKeys / p.page * kBlocks;
            const int pg = __shfl_sync(0xffffffffu, page_id, lane / kBlocks);
            if (lane < boxes)
                tma_load_4d(dst + (lane % kBlocks) * kBlock + (lane / kBlocks) * p.page * 128, map,
                            (lane % kBlocks) * 64, 0, head, pg, &s.full[slot]);
        }
        return true;
    }

    // Every fill requested has landed, or had its time to: a slot is requested anew
    // only after its last fill was used, so only the last of each can be under way.
    // One warp, once no role requests any more.
    static __device__ void land(Shared &s)
    {
        const int n = s.requested;
        for (int slot = 0; slot < min(n, kSlots); slot++) {
            const int fill = (n - 1 - slot) / kSlots * kSlots + slot;
            mbar_drain(&s.full[slot], (fill / kSlots) & 1);
        }
    }

    // The id of this lane's page of tile t: P, which reads as zeros, past the
    // entry's keys and for an id that is none.
    static __device__ __forceinline__ int page_of(const AttnArgs &p, const Seg &g, int t, int lane)
    {
        const int key = g.kbase + t * kKeys + lane * p.page;
        if (lane >= kKeys / p.page || key >= g.k1)
            return p.P;
        const int id = __ldg(p.table + static_cast<int64_t>(g.row_of_table) * p.W + key / p.page);
        if (id >= 0 && id < p.P)
            return id;
        if (p.status)
            atomicOr(p.status, W4_DEV_BAD_PAGE);
        return p.P;
    }

    // The pieces of a worker in turn, tile by tile.
    struct Walk {
        const Seg *next, *first;
        int left, t, end;                      // pieces behind this one; tile, its end
        Seg g;
        __device__ __forceinline__ bool more()
        {
            while (t >= end) {
                if (left == 0)
                    return false;
                g = first ? *first : *next;
                first = nullptr;
                next++;
                left--;
                t = g.tile0;
                end = g.tile0 + g.tiles;
            }
            return true;
        }
    };

    static __device__ __forceinline__ Walk walk(const AttnArgs &p, const Shared &s, int which)
    {
        Walk w;
        w.next = p.segs + (which == 2 ? p.cap_b : 0) + s.seg0[which];
        w.left = s.segs[which];
        w.first = &s.first[which];
        w.t = w.end = 0;
        return w;
    }

    // The tiles in the order of fill_of; a tile's page ids are read while the
    // tile before it waits for its slots.
    static __device__ void loader(const AttnArgs &p, Shared &s, uint8_t *ring, int lane)
    {
        Walk pairs = walk(p, s, 2), one = walk(p, s, 0), two = walk(p, s, 1);
        bool first = false;                    // whose turn it was last
        bool held = false;
        int held_head = 0, held_id = 0, fill = 0;
        for (bool more = true; more || held;) {
            bool got = true;
            int head = 0, id = 0;
            if (pairs.more()) {
                head = pairs.g.head;
                id = page_of(p, pairs.g, pairs.t++, lane);
            } else {
                const bool a = one.more(), b = two.more();
                first = a && !(first && b);    // streams in turn; one that is out drops out
                if (first) {
                    head = one.g.head;
                    id = page_of(p, one.g, one.t++, lane);
                } else if (b) {
                    head = two.g.head;
                    id = page_of(p, two.g, two.t++, lane);
                } else {
                    got = false;
                }
            }
            if (held) {
                if (!load_slot(p, s, ring, 2 * fill, &p.k_map, held_head, held_id, lane) ||
                    !load_slot(p, s, ring, 2 * fill + 1, &p.v_map, held_head, held_id, lane))
                    return;
                fill++;
            }
            more = held = got;
            held_head = head;
            held_id = id;
        }
    }

    // ------------------------------------------------------------- issuing
    // S = Q K^T of a stream's tile, whose K has landed; it is let go with the last use.
    static __device__ __forceinline__ void issue_qk(const AttnArgs &p, Shared &s, uint8_t *qbuf,
                                                    uint8_t *ring, int stream, int fill, bool last_use)
    {
        const int slot = fill % kSlots;
        tc_fence_after();
        __syncwarp();
        const uint64_t qd = sdesc_sw128(smem_u32(qbuf + stream * kTileBytes));
        const uint64_t kd = sdesc_mn_sw128(smem_u32(ring + slot * kTileBytes), kGroup, kBlock);
#pragma unroll
        for (int k = 0; k < D / 16; k++)
            mma_ss_elect(s.tmem + kS + 128 * stream, qd + (k / 4) * (kRows * 128 >> 4) + k % 4 * 2,
                         kd + (k / 4) * (kBlock >> 4) + k % 4 * 2, kQk, k > 0);
        tc_commit_elect(&s.s_full[stream]);
        if (last_use)
            tc_commit_elect(&s.empty[slot]);
    }

    // O (+)= P V of a stream's tile, whose V has landed, 16 keys at a time; steps that lie wholly
    // before the entry's first key or past its last stay out.
    static __device__ __forceinline__ void issue_pv(const AttnArgs &p, Shared &s, uint8_t *ring,
                                                    int stream, int fill, int before, int keys,
                                                    bool first, bool last, bool last_use)
    {
        const int slot = fill % kSlots;
        tc_fence_after();
        __syncwarp();
        const uint32_t va = smem_u32(ring + slot * kTileBytes);
        const uint32_t ts = s.tmem + kS + 128 * stream, to = s.tmem + kO + D * stream;
        const uint64_t vd = sdesc_mn_sw128(va, kGroup, kBlock);
        if (before <= 0 && keys > kKeys - 16) {
#pragma unroll
            for (int k = 0; k < kKeys / 16; k++)
                tc_mma_ts_elect(to, ts + 8 * k, vd + k * (2 * kGroup >> 4), kPv, !first || k > 0);
        } else {
            const int begin = max(before, 0) / 16, end = (min(keys, kKeys) + 15) / 16;
            for (int k = begin; k < end; k++)
                tc_mma_ts_elect(to, ts + 8 * k, vd + k * (2 * kGroup >> 4), kPv, !first || k > begin);
        }
        if (last_use)
            tc_commit_elect(&s.empty[slot]);
        if (last)
            tc_commit_elect(&s.o_full[stream]);
    }

    // A stream's MMAs in turn: S of a tile, then, when its P is there, O.  The
    // next tile's S overwrites this one's P: MMAs of one thread complete in
    // order.
    //
    // Pairs have one issuer for both streams, which alternates strictly: PV
    // and the next QK of stream 0, then of stream 1.  That keeps the streams half
    // a period apart, one's softmax under the other's MMAs; two issuers drift
    // into step and leave the tensor cores idle during both softmaxes
    // (4400 cycles a pair tile instead of 3000; its MMAs take 2048).  Single items'
    // streams are independent and bound by their loads; each has its own issuer.
    static __device__ __forceinline__ void issue_all(const AttnArgs &p, Shared &s, uint8_t *qbuf,
                                                     uint8_t *ring, int stream)
    {
        uint32_t seg_phase = 0, tile_phase = 0;
        if (stream == 0) {
            const Seg *segs = p.segs + p.cap_b + s.seg0[2];
            for (int i = 0, r = 0; i < s.segs[2]; i++) {
                const Seg &g = i == 0 ? s.first[2] : segs[i];
                const int tiles = g.tiles, base = g.kbase + g.tile0 * kKeys;
                if (tiles == 0)
                    continue;
                if (!wait_full(p, s, 2 * r))
                    return;
                for (int st = 0; st < 2; st++) {
                    if (!wait(p, s, &s.q_ready[st], seg_phase))
                        return;
                    issue_qk(p, s, qbuf, ring, st, 2 * r, st == 1);
                }
                seg_phase ^= 1;
                for (int t = 0; t < tiles; t++, r++) {
                    if (!wait_full(p, s, 2 * r + 1))
                        return;
                    bool here = t + 1 < tiles && landed(s, 2 * r + 2);
                    for (int st = 0; st < 2; st++) {
                        if (!wait(p, s, &s.p_ready[st], tile_phase))
                            return;
                        const int at = base + t * kKeys;
                        issue_pv(p, s, ring, st, 2 * r + 1, g.k0 - at, g.k1 - at, t == 0,
                                 t == tiles - 1, st == 1);
                        if (t + 1 < tiles && !here) {
                            if (!wait_full(p, s, 2 * r + 2))
                                return;
                            here = true;
                        }
                        if (t + 1 < tiles)
                            issue_qk(p, s, qbuf, ring, st, 2 * r + 2, st == 1);
                    }
                    tile_phase ^= 1;
                }
            }
        }
        const Seg *segs = p.segs + s.seg0[stream];
        for (int i = 0, r = 0; i < s.segs[stream]; i++) {
            const Seg &g = i == 0 ? s.first[stream] : segs[i];
            const int tiles = g.tiles, base = g.kbase + g.tile0 * kKeys;
            if (tiles == 0)
                continue;
            if (!wait(p, s, &s.q_ready[stream], seg_phase))
                return;
            seg_phase ^= 1;
            for (int t = 0; t < tiles; t++, r++) {
                const int fill = 2 * fill_of(s, stream, r);
                if (!wait_full(p, s, fill))
                    return;
                issue_qk(p, s, qbuf, ring, stream, fill, true);
                if (!wait_full(p, s, fill + 1) || !wait(p, s, &s.p_ready[stream], tile_phase))
                    return;
                tile_phase ^= 1;
                const int at = base + t * kKeys;
                issue_pv(p, s, ring, stream, fill + 1, g.k0 - at, g.k1 - at, t == 0,
                         t == tiles - 1, true);
            }
        }
    }

    static __device__ void issuer(const AttnArgs &p, Shared &s, uint8_t *qbuf, uint8_t *ring,
                                  int stream)
    {
        issue_all(p, s, qbuf, ring, stream);
        // nothing of this warp's is under way when the CTA ends
        __syncwarp();
        tc_commit_elect(&s.drained[stream]);
        mbar_drain(&s.drained[stream], 0);
        __syncwarp();
    }

    // ------------------------------------------------------------- softmax
    // A stream's rows: Q into shared memory, P from S tile by tile, and the
    // sums out at the end of a piece.  Thread i holds row i.
    static __device__ void softmax(const AttnArgs &p, Shared &s, uint8_t *qbuf, uint8_t *ring,
                                   int stream)
    {
        if (!all_pieces(p, s, qbuf, ring, stream))
            cp_async_wait_all();               // queries on their way
    }

    // False once a wait has given up.
    static __device__ __forceinline__ bool all_pieces(const AttnArgs &p, Shared &s, uint8_t *qbuf,
                                                      uint8_t *ring, int stream)
    {
        const int tid = threadIdx.x & 127, warp = tid >> 5;
        const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
        const uint32_t ts = s.tmem + lanes + kS + 128 * stream;
        const uint32_t to = s.tmem + lanes + kO + D * stream;
        uint8_t *q = qbuf + stream * kTileBytes;
        uint32_t s_phase = 0, o_phase = 0, clear_phase = 0;
        // a CTA has pairs, or each stream its own single items
        const bool pair = s.segs[2] > 0;
        const int which = pair ? 2 : stream, count = s.segs[which];
        const Seg *segs = p.segs + (pair ? p.cap_b : 0) + s.seg0[which];
        auto piece = [&](int i) -> const Seg & { return i == 0 ? s.first[which] : segs[i]; };
        // A piece's queries on their way to shared memory.  Called when no MMA
        // reads the queries any more.
        auto fetch = [&](int i) {
            const Seg &g = piece(i);
            if (g.tiles > 0)
                load_q(p, q, g, g.row0 + (pair ? stream * kRows : 0), rows_here(g, pair, stream),
                       tid);
        };
        // How many keys this thread's row of a piece sees.  The lanes part ways in
        // it, and the tensor-memory instructions that follow need them together
        // again.
        auto sees = [&](int i) {
            const Seg &g = piece(i);
            int n = INT_MAX;                   // no row: nothing to mask, nothing kept
            if (tid < rows_here(g, pair, stream)) {
                const int row = g.row0 + (pair ? stream * kRows : 0) + tid;
                n = min(limit_of(p, g, g.tok0 + row / p.rep), g.k1);
            }
            __syncwarp();
            return n;
        };
        auto hand_over = [&](int i) {          // the queries to the issuer
            if (piece(i).tiles == 0)
                return;
            cp_async_wait_all();
            fence_proxy_async_smem();
            __syncwarp();
            mbar_arrive_elect(&s.q_ready[stream]);
        };
        int limit = 0, next = 0;
        if (count > 0) {
            fetch(0);
            hand_over(0);
            limit = sees(0);
        }
        for (int i = 0, r = 0; i < count; i++, limit = next) {
            const bool another = i + 1 < count;
            const Seg g = piece(i);
            const int rows = rows_here(g, pair, stream);
            const bool busy = rows > (tid & ~31);
            float m = -INFINITY, l = 0.0f;     // m in units of log2
            int base = g.kbase + g.tile0 * kKeys;
            for (int t = 0; t < g.tiles; t++, r++, base += kKeys) {
                if (!wait(p, s, &s.s_full[stream], s_phase))
                    return false;
                s_phase ^= 1;
                tc_fence_after();
                if (t == g.tiles - 1 && another) {
                    fetch(i + 1);
                    next = sees(i + 1);
                }
                // a warp without rows leaves P as it is: a row's P only meets its own O
                __syncwarp();
                if (busy)
                    tile(p, ts, to, limit == INT_MAX ? 0 : g.k0 - base,
                         limit == INT_MAX ? kKeys : limit - base, t > 0, m, l);
                if (((g.k1 - base < kKeys && (g.k1 & 15)) || (g.k0 > base && (g.k0 & 15))) &&
                    !clear_ends(p, s, ring, 2 * fill_of(s, which, r) + 1, g.k0 - base,
                                g.k1 - base, pair, stream, tid, clear_phase))
                    return false;
                // one arrival a warp: a thread's each would take a few cycles of the barrier
                tc_fence_before();
                __syncwarp();
                mbar_arrive_elect(&s.p_ready[stream]);
            }
            if (another) {
                if (g.tiles == 0) {
                    fetch(i + 1);
                    next = sees(i + 1);
                }
                // the next piece's first S may be made while this one's sums are stored
                hand_over(i + 1);
            }
            if (g.tiles > 0) {
                if (!wait(p, s, &s.o_full[stream], o_phase))
                    return false;
                o_phase ^= 1;
                tc_fence_after();
            }
            store(p, g, pair, pair ? stream * kRows : 0, rows, to, m, l, tid);
        }
        return true;
    }

    // A stream's rows of a piece.
    static __device__ __forceinline__ int rows_here(const Seg &g, bool pair, int stream)
    {
        return min(max(g.rows - (pair ? stream * kRows : 0), 0), kRows);
    }

    // Rows [row0, row0 + rows) of a piece's queries, 16 bytes a thread and
    // step; rows past the end are zero.
    static __device__ __forceinline__ void load_q(const AttnArgs &p, uint8_t *q, const Seg &g,
                                                  int row0, int rows, int tid)
    {
        constexpr int kChunks = D / 8, kStep = 128 / kChunks;
        const int c = tid % kChunks;
        const uint16_t *src = p.q + g.tok0 * p.q_tok +
                              static_cast<int64_t>(g.head) * p.rep * p.q_head + c * 8;
        int row = tid / kChunks;
        int64_t tok = (row0 + row) / p.rep;
        int h = row0 + row - static_cast<int>(tok) * p.rep;
        const int tok_step = kStep / p.rep, h_step = kStep - tok_step * p.rep;
#pragma unroll 4
        for (; row < kRows; row += kStep) {
            uint8_t *dst = q + (c / 8) * (kRows * 128) + row * 128 + ((c % 8) ^ (row & 7)) * 16;
            if (row < rows)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)),
                             "l"(src + tok * p.q_tok + h * p.q_head)
                             : "memory");
            else
                *reinterpret_cast<uint4 *>(dst) = make_uint4(0, 0, 0, 0);
            tok += tok_step;
            h += h_step;
            if (h >= p.rep) {
                h -= p.rep;
                tok++;
            }
        }
    }

    // How many keys, from position 0, the query token sees.
    static __device__ int limit_of(const AttnArgs &p, const Seg &g, int tok)
    {
        int b = g.seq;
        if (b < 0) {                           // the sequence of a group that has the token
            // where every sequence has max_q tokens it can be told at once
            b = min(g.row_of_table + (tok - g.tok0) / p.max_q, p.B - 1);
            if (p.q_offsets[b] > tok || p.q_offsets[b + 1] <= tok) {
                int lo = g.row_of_table, hi = p.B - 1;
                while (lo < hi) {
                    const int mid = (lo + hi + 1) >> 1;
                    if (p.q_offsets[mid] <= tok)
                        lo = mid;
                    else
                        hi = mid - 1;
                }
                b = lo;
            }
        }
        const int len = min(max(p.lens[b], 0), p.W * p.page);
        return p.causal ? len - (p.q_offsets[b + 1] - tok) + 1 : len;
    }

    // P of one tile from its S; columns outside [lo, hi) are masked.  m is the
    // reference of the exponents, not always the maximum: it moves only when
    // the maximum has grown by more than 2^8 since it last moved, so O is seldom
    // rescaled.  For bf16 it moves to the maximum, for fp16 to 2^7 below, so that P lies
    // in 0 .. 2^15 and a weight vanishes only 2^32 below the largest (2^25 otherwise: a
    // hundred thousand keys beside one that outweighs them can be 0.4 % of the result).
    // P is rounded to the values' type for the MMA (its
    // denominator sums the unrounded).  When S is here, every MMA before it has
    // completed, so O may be changed.
    static __device__ __forceinline__ void tile(const AttnArgs &p, uint32_t ts, uint32_t to, int lo,
                                                int hi, bool has_o, float &m, float &l)
    {
        uint32_t v[128];
        tmem_ld_32x32b_x128(ts, v);
        if (__any_sync(0xffffffffu, lo > 0 || hi < kKeys)) {
#pragma unroll
            for (int c = 0; c < 128; c++)
                if (c < lo || c >= hi)
                    v[c] = 0xff800000u;        // -inf
        }
        float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < 128; c += 2)
            top[c / 2 & 3] = max3(top[c / 2 & 3], __uint_as_float(v[c]), __uint_as_float(v[c + 1]));
        const float tm = max3(fmaxf(top[0], top[1]), top[2], top[3]) * p.scale_log2;
        constexpr float kLift = BF16 ? 0.0f : 7.0f;
        const bool move = tm > m + (8.0f + kLift);         // also from -inf
        if (__any_sync(0xffffffffu, move)) {
            const float alpha = move ? ex2(m - (tm - kLift)) : 1.0f;
            m = move ? tm - kLift : m;
            l *= alpha;
            if (has_o)
                rescale(to, alpha);
        }
        const float ref = m == -INFINITY ? 0.0f : m;
        const uint64_t scale2 = both(p.scale_log2), ref2 = both(-ref);
        uint64_t sum[2] = {both(0.0f), both(0.0f)};
#pragma unroll
        for (int c = 0; c < 128; c += 32) {
            uint32_t pk[16];
#pragma unroll
            for (int j = 0; j < 16; j++) {
                const uint64_t x = fma2(pair_of(v[c + 2 * j], v[c + 2 * j + 1]), scale2, ref2);
                const float a = ex2(low(x)), b = ex2(high(x));
                sum[j & 1] = add2(sum[j & 1], pair_of(__float_as_uint(a), __float_as_uint(b)));
                pk[j] = pack2<BF16>(a, b);
            }
            tmem_st_32x32b_x16(ts + c / 2, pk);
        }
        const uint64_t all = add2(sum[0], sum[1]);
        l += low(all) + high(all);
        tmem_wait_st();
    }

    static __device__ __forceinline__ void rescale(uint32_t to, float alpha)
    {
        __syncwarp();
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
            uint32_t o[32];
            tmem_ld_32x32b_x32(to + c, o);
#pragma unroll
            for (int j = 0; j < 32; j++)
                o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
            tmem_st_32x32b_x32(to + c, o);
        }
        tmem_wait_st();
    }

    // Values before the first key and past the last, in the 16-key steps that
    // these lie in: P is zero there, but memory nobody has written may hold NaN.
    // In a pair both streams clear, and wait for each other, before either uses
    // the tile.
    static __device__ bool clear_ends(const AttnArgs &p, Shared &s, uint8_t *ring, int fill,
                                      int before, int valid, bool pair, int stream, int tid,
                                      uint32_t &phase)
    {
        const int slot = fill % kSlots;
        if (!wait_full(p, s, fill))
            return false;
        uint8_t *v = ring + slot * kTileBytes;
        const int at = pair ? stream * 128 + tid : tid, step = pair ? 256 : 128;
        auto clear = [&](int from, int to) {
            for (int i = at; i < (to - from) * 8 * kBlocks; i += step) {
                const int row = from + i / (8 * kBlocks), c = i % (8 * kBlocks);
                *reinterpret_cast<uint4 *>(v + (c / 8) * kBlock + (row / 8) * kGroup +
                                           (row % 8) * 128 + (c % 8) * 16) =
                    make_uint4(0, 0, 0, 0);
            }
        };
        if (before > 0)
            clear(before & ~15, before);
        if (valid < kKeys)
            clear(valid, (valid + 15) & ~15);
        fence_proxy_async_smem();
        __syncwarp();
        if (pair) {
            mbar_arrive_elect(&s.cleared);
            if (!wait(p, s, &s.cleared, phase))
                return false;
            phase ^= 1;
        }
        return true;
    }

    // A piece's sums: [D / 4][rows][4] floats, so that a warp's rows are
    // written side by side.
    static __device__ void store(const AttnArgs &p, const Seg &g, bool pair, int row, int rows,
                                 uint32_t to, float m, float l, int tid)
    {
        const int kind = pair ? 0 : g.seq < 0 ? 1 : 2;
        const int all = rows_of(p, kind);
        const int64_t base = static_cast<int64_t>(g.piece) * all;
        if (!W4_IN_BOUNDS(g.piece >= 0 && row + rows <= all &&
                              g.piece < (kind == 0 ? p.cap_a : kind == 1 ? p.cap_g : p.cap_b),
                          p.status))
            return;
        if (tid < rows)
            (pair ? p.ml[0] : kind == 1 ? p.ml[1] : p.ml[2])[base + row + tid] = make_float2(m, l);
        __syncwarp();
        if (g.tiles == 0 || rows <= (tid & ~31))
            return;
        float4 *out = reinterpret_cast<float4 *>(pair ? p.part[0] : kind == 1 ? p.part[1]
                                                                              : p.part[2]) +
                      base * (D / 4) + row + tid;
#pragma unroll 1
        for (int c = 0; c < D; c += 16) {
            uint32_t o[16];
            __syncwarp();
            tmem_ld_32x32b_x16(to + c, o);
            if (tid < rows) {
#pragma unroll
                for (int j = 0; j < 4; j++)
                    out[static_cast<int64_t>(c / 4 + j) * all] =
                        make_float4(__uint_as_float(o[4 * j]), __uint_as_float(o[4 * j + 1]),
                                    __uint_as_float(o[4 * j + 2]), __uint_as_float(o[4 * j + 3]));
            }
        }
        tc_fence_before();
    }
};

template <int D, bool BF16, bool IN_TURN>
__global__ void __launch_bounds__(kThreads, 1) attn_kernel(const __grid_constant__ AttnArgs p)
{
    using K = Kernel<D, BF16, IN_TURN>;
    extern __shared__ __align__(1024) uint8_t raw[];
    __shared__ __align__(16) typename K::Shared s;
    uint8_t *qbuf = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    uint8_t *ring = qbuf + K::kQBytes;
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    if (tid == 0) {
        for (int i = 0; i < K::kSlots; i++) {
            mbar_init(&s.full[i], p.withhold && i == 0 ? 2 : 1);
            mbar_init(&s.empty[i], 1);
        }
        for (int i = 0; i < 2; i++) {
            mbar_init(&s.q_ready[i], kRows / 32);
            mbar_init(&s.s_full[i], 1);
            mbar_init(&s.p_ready[i], kRows / 32);
            mbar_init(&s.o_full[i], 1);
            mbar_init(&s.drained[i], 1);
        }
        mbar_init(&s.cleared, 2 * kRows / 32);
        s.abort_flag = 0;
        s.requested = 0;
        fence_mbar_init();
        prefetch_tmap(&p.k_map);
        prefetch_tmap(&p.v_map);
    }
    if (warp == 8) {
        tmem_alloc(&s.tmem, 512);
        tmem_relinquish();
    }
    pdl_wait();
    pdl_trigger();
    K::make_plan(p, s, qbuf);
    fence_proxy_async_smem();              // the plan's scratch becomes queries and ring
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    __syncwarp();
    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        K::softmax(p, s, qbuf, ring, warp >> 2);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp == 8)
            K::loader(p, s, ring, lane);
        else if (warp < 11)
            K::issuer(p, s, qbuf, ring, warp - 9);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        if (*static_cast<volatile int *>(&s.abort_flag)) {
            K::land(s);
            __syncwarp();
        }
        tc_fence_after();
        __syncwarp();
        tmem_dealloc(s.tmem, 512);
    }
}

// -------------------------------------------------------------------- join
// A row's pieces joined: CTA (b, y, z) takes 32 of sequence b's rows (a lane
// each: neighbouring rows are side by side in a piece) and some of the D
// values.  A warp has 16 of those and every SPLIT-th piece, kBatch pieces'
// loads in flight; the SPLIT parts are added up at the end, in a fixed order.
// Few rows can have many pieces (one long prefix cut for every CTA), many rows
// have few: SPLIT is 4 up to kJoinFewRows rows in all and 1 above.  (Both kernels with
// SPLIT 4 and 1: 1024 rows of 120,000 shared tokens 72 and 93 us, 1024 of 64 ragged sequences 59
// and 65, some 5000 of nine small groups 28.0 and 26.2, 16384 of four canvases 60 and 47.)
constexpr int kJoinFewRows = 4096;
template <int D, int SPLIT> constexpr int kJoinSides = 8 / SPLIT < D / 16 ? 8 / SPLIT : D / 16;

template <int D, bool BF16, int SPLIT>
__global__ void __launch_bounds__(32 * SPLIT *kJoinSides<D, SPLIT>, SPLIT == 1 ? 3 : 2)
    attn_join_kernel(const __grid_constant__ AttnArgs p)
{
    constexpr int kBatch = SPLIT == 1 ? 2 : 3, kSides = kJoinSides<D, SPLIT>;
    __shared__ float4 so[SPLIT][4][kSides][32];
    __shared__ float2 sm[SPLIT][kSides][32];
    pdl_wait();
    pdl_trigger();
    const Joint j = p.joints[blockIdx.x];
    const int rows = j.tokens * p.rep;         // of one kv head
    const int n = rows * p.Hkv;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int side = warp % kSides, cg = kSides * blockIdx.z + side, split = warp / kSides;
    for (int i0 = blockIdx.y * 32; i0 < n; i0 += gridDim.y * 32) {
        const int i = min(i0 + lane, n - 1), head = i / rows, row = i - head * rows;
        float m = -INFINITY, l = 0.0f;
        float4 o[4] = {};
        // (the loop and the batches stay small: the kernel is short enough for the
        // fetching of its instructions to show)
#pragma unroll 1
        for (int k = 0; k < 2; k++) {          // the prefix's pieces, the sequence's own
            const Entry en = k ? j.e[1] : j.e[0];
            if (en.span == 0)
                continue;
            const int er = row + en.row, step = en.pair ? 2 * kRows : kRows;
            const int kind = en.pair ? 0 : k + 1, stride = rows_of(p, kind), at = er % step;
            const int local = head * en.row_tiles + er / step;
            const int all = en.pair ? j.all[1] : j.all[0];
            const int workers = en.pair ? j.workers[1] : j.workers[0];
            const int x0 = en.place + local * en.span;
            const int w0 = worker_of(all, workers, x0);
            const int w1 = worker_of(all, workers, x0 + en.span - 1);
            if (en.item0 + local + w1 >= (kind == 0 ? p.cap_a : kind == 1 ? p.cap_g : p.cap_b))
                continue;
            const int64_t first = static_cast<int64_t>(en.item0 + local) * stride;
            const float2 *ml = (en.pair ? p.ml[0] : p.ml[k + 1]) + first + at;
            const float4 *part = reinterpret_cast<const float4 *>(en.pair ? p.part[0]
                                                                          : p.part[k + 1]) +
                                 first * (D / 4) + cg * 4 * stride + at;
            for (int w = w0 + split; w <= w1; w += SPLIT * kBatch) {
                float4 v[kBatch][4];
                float2 s[kBatch];
#pragma unroll
                for (int u = 0; u < kBatch; u++) {
                    const int64_t x = w + SPLIT * u;
                    s[u] = make_float2(-INFINITY, 0.0f);
                    if (x <= w1) {
                        s[u] = ml[x * stride];
#pragma unroll
                        for (int c = 0; c < 4; c++)
                            v[u][c] = part[x * stride * (D / 4) + c * stride];
                    }
                }
                float top = m;
#pragma unroll
                for (int u = 0; u < kBatch; u++)
                    top = fmaxf(top, s[u].x);
                // with nothing visible yet every factor is zero
                const float ref = top == -INFINITY ? 0.0f : top;
                const float f0 = ex2(m - ref);
                m = top;
                l *= f0;
#pragma unroll
                for (int c = 0; c < 4; c++)
                    o[c] = make_float4(o[c].x * f0, o[c].y * f0, o[c].z * f0, o[c].w * f0);
#pragma unroll
                for (int u = 0; u < kBatch; u++) {
                    if (!(s[u].y > 0.0f) && s[u].y == s[u].y)
                        continue;              // nothing visible in this piece
                    const float f = ex2(s[u].x - ref);
                    l = fmaf(s[u].y, f, l);
#pragma unroll
                    for (int c = 0; c < 4; c++) {
                        o[c].x = fmaf(v[u][c].x, f, o[c].x);
                        o[c].y = fmaf(v[u][c].y, f, o[c].y);
                        o[c].z = fmaf(v[u][c].z, f, o[c].z);
                        o[c].w = fmaf(v[u][c].w, f, o[c].w);
                    }
                }
            }
        }
        if (split > 0) {
            sm[split - 1][side][lane] = make_float2(m, l);
#pragma unroll
            for (int c = 0; c < 4; c++)
                so[split - 1][c][side][lane] = o[c];
        }
        __syncthreads();
        if (split == 0 && i0 + lane < n) {
#pragma unroll
            for (int k = 0; k < SPLIT - 1; k++) {
                const float2 s = sm[k][side][lane];
                const float top = fmaxf(m, s.x), ref = top == -INFINITY ? 0.0f : top;
                const float f0 = ex2(m - ref), f1 = ex2(s.x - ref);
                m = top;
                l = l * f0 + s.y * f1;
#pragma unroll
                for (int c = 0; c < 4; c++) {
                    const float4 v = so[k][c][side][lane];
                    o[c] = make_float4(o[c].x * f0 + v.x * f1, o[c].y * f0 + v.y * f1,
                                       o[c].z * f0 + v.z * f1, o[c].w * f0 + v.w * f1);
                }
            }
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;     // a row that sees nothing is zero
            const int tok = j.tok0 + row / p.rep, h = head * p.rep + row % p.rep;
            uint32_t r[8];
#pragma unroll
            for (int c = 0; c < 4; c++) {
                r[2 * c] = pack2<BF16>(o[c].x * inv, o[c].y * inv);
                r[2 * c + 1] = pack2<BF16>(o[c].z * inv, o[c].w * inv);
            }
            uint4 *out = reinterpret_cast<uint4 *>(
                p.out + (static_cast<int64_t>(tok) * p.Hq + h) * D + cg * 16);
            if (W4_IN_BOUNDS(tok >= 0 && tok < p.T && h < p.Hq, p.status)) {
                out[0] = make_uint4(r[0], r[1], r[2], r[3]);
                out[1] = make_uint4(r[4], r[5], r[6], r[7]);
            }
        }
        __syncthreads();
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

PageView view_of(const AttnProblem &q)
{
    if (q.page > kShortPage || q.D == 64)
        return PageView::kRows;
    if (q.head_stride == q.D)
        return PageView::kHeadsAsBlocks;
    if (q.page_stride == q.Hkv * q.head_stride &&
        (static_cast<int64_t>(q.P) + 1) * q.Hkv < (1ll << 31))
        return PageView::kHeadsAsPages;
    return PageView::kGroups;
}

// What lies past the last page reads as zeros.
bool encode_pages(CUtensorMap *map, const AttnProblem &q, PageView view, const uint16_t *base)
{
    const bool rows = view == PageView::kRows, heads = view == PageView::kHeadsAsBlocks;
    const bool groups = view == PageView::kGroups, together = view == PageView::kHeadsAsPages;
    const cuuint64_t tok = static_cast<cuuint64_t>(q.tok_stride) * 2;
    const cuuint64_t head = static_cast<cuuint64_t>(q.head_stride) * 2;
    const cuuint64_t page = static_cast<cuuint64_t>(q.page_stride) * 2;
    const cuuint64_t P = q.P, Hkv = q.Hkv, size = q.page, D = q.D, blocks = D / 64;
    const cuuint64_t dim4[4] = {D, size, Hkv, P}, stride4[3] = {tok, head, page};
    const cuuint32_t box4[4] = {64, static_cast<cuuint32_t>(size), 1, 1};
    const cuuint64_t dim5[5] = {64, groups ? size : 8, heads ? Hkv * blocks : blocks,
                                groups ? Hkv : size / 8, together ? P * Hkv : P};
    const cuuint64_t stride5[4] = {tok, 128, groups ? head : 8 * tok, together ? head : page};
    const cuuint32_t box5[5] = {64, 8, static_cast<cuuint32_t>(blocks),
                                groups ? 1u : static_cast<cuuint32_t>(size / 8), 1};
    const cuuint32_t step[5] = {1, 1, 1, 1, 1};
    return encode_fn()(map, q.bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                       rows ? 4 : 5, const_cast<uint16_t *>(base), rows ? dim4 : dim5,
                       rows ? stride4 : stride5, rows ? box4 : box5, step,
                       CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                       CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Where a call's pieces lie in its workspace.
struct Space {
    int cap_a, cap_g, cap_b, rows_b;
    size_t joints, segs, ml[3], part[3], total;
};

constexpr int kMaxGrid = 256;              // CTAs that a workspace allows for

Space space_of(int T, int B, int G, int max_q, int Hq, int Hkv, int D)
{
    Space s{};
    const int64_t rep = Hq / Hkv;
    const plan::Caps caps = plan::caps_of(T, rep, B, G, Hkv, kMaxGrid);
    s.cap_a = caps.pairs;
    s.cap_g = caps.groups;
    s.cap_b = caps.singles;
    s.rows_b = static_cast<int>(std::min<int64_t>(rep * max_q, kRows));
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += (bytes + 255) / 256 * 256;
        return here;
    };
    s.joints = take(sizeof(Joint) * static_cast<size_t>(B));
    s.segs = take(sizeof(Seg) * (static_cast<size_t>(s.cap_a) + s.cap_b));
    const size_t rows[3] = {static_cast<size_t>(s.cap_a) * 2 * kRows,
                            G > 0 ? static_cast<size_t>(s.cap_g) * kRows : 0,
                            static_cast<size_t>(s.cap_b) * s.rows_b};
    for (int i = 0; i < 3; i++) {
        s.ml[i] = take(sizeof(float2) * rows[i]);
        s.part[i] = take(sizeof(float) * rows[i] * D);
    }
    s.total = at;
    return s;
}

template <int D, bool BF16, bool IN_TURN>
cudaError_t launch_variant(const AttnArgs &a, int dev, int sms, cudaStream_t stream)
{
    using K = Kernel<D, BF16, IN_TURN>;
    auto kern = attn_kernel<D, BF16, IN_TURN>;
    static std::atomic<uint64_t> raised{0};      // devices whose limit is raised already
    cudaError_t err;
    if (!(raised.load(std::memory_order_relaxed) >> (dev & 63) & 1u)) {
        err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   static_cast<int>(K::kSmem));
        if (err != cudaSuccess)
            return err;
        raised.fetch_or(1ull << (dev & 63), std::memory_order_relaxed);
    }
    const int grid = std::min(sms, kMaxGrid);
    err = launch_pdl(kern, dim3(grid), dim3(kThreads), K::kSmem, stream, a);
    if (err != cudaSuccess)
        return err;
    const int y = std::min((a.max_q * a.Hq + 31) / 32, std::max(65535 / a.B, 1));
    if (static_cast<int64_t>(a.T) * a.Hq <= kJoinFewRows)
        return launch_pdl(attn_join_kernel<D, BF16, 4>, dim3(a.B, y, D / 16 / kJoinSides<D, 4>),
                          dim3(128 * kJoinSides<D, 4>), 0, stream, a);
    return launch_pdl(attn_join_kernel<D, BF16, 1>, dim3(a.B, y, D / 16 / kJoinSides<D, 1>),
                      dim3(32 * kJoinSides<D, 1>), 0, stream, a);
}

}  // namespace

size_t attn_workspace_bytes(int T, int B, int G, int max_q, int Hq, int Hkv, int D)
{
    return space_of(T, B, G, max_q, Hq, Hkv, D).total;
}

cudaError_t launch_attn(const AttnProblem &q, cudaStream_t stream)
{
    int dev = 0, sms = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err == cudaSuccess)
        err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (err != cudaSuccess)
        return err;
    AttnArgs a{};
    if (!encode_fn())
        return cudaErrorNotSupported;
    a.view = view_of(q);
    if (!encode_pages(&a.k_map, q, a.view, q.k_pages) ||
        !encode_pages(&a.v_map, q, a.view, q.v_pages))
        return cudaErrorInvalidValue;
    const Space s = space_of(q.T, q.B, q.G, q.max_q, q.Hq, q.Hkv, q.D);
    uint8_t *ws = static_cast<uint8_t *>(q.workspace);
    a.joints = reinterpret_cast<Joint *>(ws + s.joints);
    a.segs = reinterpret_cast<Seg *>(ws + s.segs);
    for (int i = 0; i < 3; i++) {
        a.ml[i] = reinterpret_cast<float2 *>(ws + s.ml[i]);
        a.part[i] = reinterpret_cast<float *>(ws + s.part[i]);
    }
    a.cap_a = s.cap_a;
    a.cap_g = s.cap_g;
    a.cap_b = s.cap_b;
    a.rows_b = s.rows_b;
    a.q = q.q;
    a.out = q.out;
    a.table = q.table;
    a.lens = q.lens;
    a.q_offsets = q.q_offsets;
    a.group_offsets = q.group_offsets;
    a.shared = q.shared;
    a.status = q.dev_status;
    a.q_tok = q.q_tok;
    a.q_head = q.q_head;
    a.scale_log2 = q.scale * 1.4426950408889634f;
    a.wait_ns = pipeline_test_hooks().wait_ns;
    a.withhold = pipeline_test_hooks().withhold_sz;
    a.T = q.T;
    a.B = q.B;
    a.G = q.G;
    a.W = q.W;
    a.P = q.P;
    a.page = q.page;
    a.page_shift = q.page == 16 ? 4 : q.page == 32 ? 5 : q.page == 64 ? 6 : 7;
    a.Hq = q.Hq;
    a.Hkv = q.Hkv;
    a.rep = q.Hq / q.Hkv;
    a.max_q = q.max_q;
    a.causal = q.causal;
    if (a.view != PageView::kRows)             // D is 128
        return q.bf16 ? launch_variant<128, true, true>(a, dev, sms, stream)
                      : launch_variant<128, false, true>(a, dev, sms, stream);
    if (q.D == 128)
        return q.bf16 ? launch_variant<128, true, false>(a, dev, sms, stream)
                      : launch_variant<128, false, false>(a, dev, sms, stream);
    return q.bf16 ? launch_variant<64, true, false>(a, dev, sms, stream)
                  : launch_variant<64, false, false>(a, dev, sms, stream);
}

}  // namespace w4
