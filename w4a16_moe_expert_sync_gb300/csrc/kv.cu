// kv.cu -- the pages of a key/value cache: reserving, forking, freeing,
// compacting, copying and filling them, all on the device and in stream
// order, so that a serving step can be captured whole.
//
// State: table [B, W] holds each sequence's pages in order (-1: none), lens
// [B] its tokens, refs [P] how many sequences hold a page.  A page is free
// when refs is 0, and the lowest free pages are handed out first, in the order
// of the requests: no free list to keep, the same result on every run, and
// the pool's front stays dense.  Finding them is a scan of refs by one CTA
// (4096 pages a round, 7 to 10 us for a few thousand pages); the rest are plain
// grid-wide copies, bound by HBM.  Measured on GB300, against the bytes at the copy
// bandwidth: whole pages 1.47 GB in 232 us (217) and, with the plan and the table, 2.50 to
// 2.63 GB in 372 to 404 us (369 to 388: how many pages move, and from where, differs);
// releasing, reserving and filling 48 prompts, 574 MB, 98 us (85); releasing and forking
// 96 drafts, 271 MB, 41 us (40).
#include <algorithm>
#include <atomic>

#include "../../include/w4moe.h"
#include "checks.cuh"
#include "launch.h"
#include "ptx.cuh"

namespace w4 {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kMaxSlots = kPlanThreads;      // requests of one call: a thread each

__device__ __forceinline__ void raise_status(int32_t *status, int32_t bit)
{
    if (status)
        atomicOr(status, bit);
}

// Exclusive sum over the CTA (1024 threads); every thread gets the total.
// `sums` is 33 ints; the caller may reuse it after its next barrier.
__device__ __forceinline__ int block_exclusive_sum(int v, int *sums, int *total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, incl, o);
        incl += lane >= o ? u : 0;
    }
    if (lane == 31)
        sums[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        const int mine = sums[lane];
        int s = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, s, o);
            s += lane >= o ? u : 0;
        }
        sums[lane] = s - mine;
        if (lane == 31)
            sums[32] = s;
    }
    __syncthreads();
    *total = sums[32];
    return sums[warp] + incl - v;
}

struct PlanShared {
    int sums[2][33];
    alignas(16) int slot[kMaxSlots];
    int start[kMaxSlots + 1];      // pages asked for before request i
    int at[kMaxSlots];             // request i's first table entry
};

// Whether an earlier request names the same slot.
__device__ __forceinline__ bool repeated(const int *slot, int i)
{
    const int mine = slot[i];
    bool again = false;
    for (int j = 0; j < i; j += 4) {       // what lies past i holds other requests: not counted
        const int4 s = *reinterpret_cast<const int4 *>(slot + j);
        again |= s.x == mine || (j + 1 < i && s.y == mine) || (j + 2 < i && s.z == mine) ||
                 (j + 3 < i && s.w == mine);
    }
    return again;
}

// The request that the rank-th page goes to.
__device__ __forceinline__ int owner_of(const int *start, int n, int rank)
{
    int lo = 0, hi = n - 1;              // the last i with start[i] <= rank
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (start[mid] <= rank)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// Hands the `total` lowest free pages out: page of rank r goes to table entry
// at[i] + r - start[i] of slot[i].  Returns how many requests, in order, got
// all of theirs; the pages of the first that did not are given back.  (A request
// that needs none is served wherever it stands.)
__device__ int hand_out(PlanShared &s, int n, int total, int32_t *table, int B, int W,
                        int32_t *refs, int P, int32_t *status)
{
    const int tid = threadIdx.x;
    int found = 0;
    for (int p0 = 0, round = 0; p0 < P && found < total; p0 += 4 * kPlanThreads, round ^= 1) {
        const int p = p0 + 4 * tid;
        bool open[4];
        int mine = 0;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            open[i] = p + i < P && refs[p + i] == 0;
            mine += open[i];
        }
        int here;
        int rank = found + block_exclusive_sum(mine, s.sums[round], &here);
#pragma unroll
        for (int i = 0; i < 4; i++) {
            if (open[i] && rank < total) {
                const int r = owner_of(s.start, n, rank), col = s.at[r] + rank - s.start[r];
                if (W4_IN_BOUNDS(s.slot[r] >= 0 && s.slot[r] < B && col >= 0 && col < W, status)) {
                    table[static_cast<int64_t>(s.slot[r]) * W + col] = p + i;
                    refs[p + i] = 1;
                }
            }
            rank += open[i];
        }
        found += here;
    }
    if (found >= total)
        return n;
    __syncthreads();
    int served = n;                      // the first request that lacks a page
    for (int lo = 0, hi = n; lo < hi;) {
        const int mid = (lo + hi) >> 1;
        if (s.start[mid + 1] > found)
            served = hi = mid;
        else
            lo = mid + 1;
    }
    for (int r = s.start[served] + tid; r < found; r += kPlanThreads) {
        int32_t *e = &table[static_cast<int64_t>(s.slot[served]) * W + s.at[served] + r -
                            s.start[served]];
        if (W4_IN_BOUNDS(*e >= 0 && *e < P, status))
            refs[*e] = 0;
        *e = -1;
    }
    return served;
}

// --------------------------------------------------------------- reserve
__global__ void __launch_bounds__(kPlanThreads) kv_reserve_kernel(
    int32_t *table, int B, int W, int32_t *lens, int32_t *refs, int P, const int32_t *slots,
    const int32_t *new_lens, int n, int page, int32_t *status)
{
    __shared__ PlanShared s;
    const int i = threadIdx.x;
    pdl_wait();
    pdl_trigger();
    const int slot = i < n ? slots[i] : -1, want = i < n ? new_lens[i] : 0;
    s.slot[i] = slot;
    __syncthreads();
    bool ok = false;
    int first = 0, need = 0;
    if (i < n) {
        ok = slot >= 0 && slot < B && !repeated(s.slot, i);
        if (ok) {
            const int len = lens[slot];
            first = (len + page - 1) / page;
            const int last = want / page + (want % page != 0);
            ok = len >= 0 && want >= len && last <= W;
            // From the page of the next token on, what the slot holds already (its
            // length has been lowered) it keeps; a page that others hold too is not
            // to be written.
            if (ok && want > len) {
                const int32_t *row = table + static_cast<int64_t>(slot) * W;
                int c = len / page;
                for (; ok && c < last && row[c] >= 0 && row[c] < P; c++)
                    ok = refs[row[c]] <= 1;
                first = max(first, c);
            }
            need = ok ? last - first : 0;
        }
        if (!ok)
            raise_status(status, W4_DEV_BAD_SLOT);
    }
    int total;
    s.start[i] = block_exclusive_sum(need, s.sums[0], &total);
    s.at[i] = first;
    if (i == 0)
        s.start[n] = total;
    __syncthreads();
    // threads past n hold start = total as well, which the search never reaches
    const int served = hand_out(s, n, total, table, B, W, refs, P, status);
    if (ok) {
        if (i < served || need == 0)
            lens[slot] = want;
        else
            raise_status(status, W4_DEV_NO_PAGES);
    }
}

// ------------------------------------------------------------------- free
__global__ void __launch_bounds__(256) kv_free_kernel(int32_t *table, int B, int W, int32_t *lens,
                                                      int32_t *refs, int P, const int32_t *slots,
                                                      int32_t *status)
{
    pdl_wait();
    pdl_trigger();
    const int slot = slots[blockIdx.x];
    const int c0 = blockIdx.y * blockDim.x + threadIdx.x;
    if (slot < 0 || slot >= B) {
        if (c0 == 0)
            raise_status(status, W4_DEV_BAD_SLOT);
        return;
    }
    if (c0 == 0)
        lens[slot] = 0;
    int32_t *row = table + static_cast<int64_t>(slot) * W;
    for (int c = c0; c < W; c += gridDim.y * blockDim.x) {
        if (row[c] == -1)
            continue;
        const int p = atomicExch(&row[c], -1);     // a slot named twice is freed once
        if (p == -1)
            continue;
        if (p < 0 || p >= P || atomicSub(&refs[p], 1) <= 0) {
            if (p >= 0 && p < P)
                atomicAdd(&refs[p], 1);
            raise_status(status, W4_DEV_BAD_PAGE);
        }
    }
}

// ------------------------------------------------------------------- fork
// plan: [n] {parent slot or -1, page of the copied tail or -1}
__global__ void __launch_bounds__(kPlanThreads) kv_fork_plan_kernel(
    int32_t *table, int B, int W, int32_t *lens, int32_t *refs, int P, const int32_t *parents,
    const int32_t *children, int n, int page, int2 *plan, int32_t *status)
{
    __shared__ PlanShared s;
    const int i = threadIdx.x;
    pdl_wait();
    pdl_trigger();
    const int a = i < n ? parents[i] : -1, b = i < n ? children[i] : -1;
    s.slot[i] = b;
    __syncthreads();
    bool ok = false;
    int len = 0, full = 0, need = 0;
    if (i < n) {
        ok = a >= 0 && a < B && b >= 0 && b < B && a != b && lens[b] == 0 &&
             table[static_cast<int64_t>(b) * W] == -1 && !repeated(s.slot, i);
        if (ok) {
            len = lens[a];
            full = len / page;
            need = len % page != 0;
            ok = len >= 0 && full + need <= W;
            need = ok ? need : 0;
        }
        if (!ok)
            raise_status(status, W4_DEV_BAD_SLOT);
    }
    int total;
    s.start[i] = block_exclusive_sum(need, s.sums[0], &total);
    s.at[i] = full;
    if (i == 0)
        s.start[n] = total;
    __syncthreads();               // every length is read before one is written
    const int served = hand_out(s, n, total, table, B, W, refs, P, status);
    __syncthreads();
    if (i < n) {
        const bool done = ok && (i < served || need == 0);
        if (ok && !done)
            raise_status(status, W4_DEV_NO_PAGES);
        if (done)
            lens[b] = len;
        plan[i] = make_int2(done ? a : -1, done && need ? table[static_cast<int64_t>(b) * W + full]
                                                        : -1);
    }
}

// `bytes` (a multiple of 16) copied by the CTA, four vectors a thread in flight.
__device__ __forceinline__ void copy_bytes(uint8_t *dst, const uint8_t *src, int64_t bytes)
{
    constexpr int kUnroll = 4;
    const int64_t vecs = bytes / 16, step = blockDim.x;
    int64_t v = threadIdx.x;
    const int4 *in = reinterpret_cast<const int4 *>(src);
    int4 *out = reinterpret_cast<int4 *>(dst);
    for (; v + (kUnroll - 1) * step < vecs; v += kUnroll * step) {
        int4 r[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; u++)
            r[u] = __ldcs(in + v + u * step);
#pragma unroll
        for (int u = 0; u < kUnroll; u++)
            __stcs(out + v + u * step, r[u]);
    }
    for (; v < vecs; v += step)
        __stcs(out + v, __ldcs(in + v));
}

// CTA (i, plane) copies pair i's tail rows of one plane; plane 0's also shares
// the full pages.
__global__ void __launch_bounds__(256) kv_fork_kernel(uint8_t *cache, int64_t page_bytes,
                                                      int32_t *table, int W, const int32_t *lens,
                                                      int32_t *refs, int P,
                                                      const int32_t *children, int page,
                                                      const int2 *plan, int32_t *status)
{
    pdl_wait();
    pdl_trigger();
    const int2 pl = plan[blockIdx.x];
    if (pl.x < 0)
        return;
    const int b = children[blockIdx.x], len = lens[b], full = len / page;
    const int32_t *from = table + static_cast<int64_t>(pl.x) * W;
    if (blockIdx.y == 0) {
        int32_t *to = table + static_cast<int64_t>(b) * W;
        for (int c = threadIdx.x; c < full; c += blockDim.x) {
            if (!W4_IN_BOUNDS(c < W, status))
                break;
            const int p = from[c];
            const bool ok = p >= 0 && p < P;
            to[c] = ok ? p : -1;
            if (ok)
                atomicAdd(&refs[p], 1);
            else
                raise_status(status, W4_DEV_BAD_PAGE);
        }
    }
    if (pl.y < 0)
        return;
    const int old = from[full];
    if (old < 0 || old >= P) {
        if (blockIdx.y == 0 && threadIdx.x == 0)
            raise_status(status, W4_DEV_BAD_PAGE);
        return;
    }
    uint8_t *plane = cache + static_cast<int64_t>(blockIdx.y) * P * page_bytes;
    if (W4_IN_BOUNDS(full < W && pl.y < P, status))
        copy_bytes(plane + pl.y * page_bytes, plane + old * page_bytes,
                   page_bytes / page * (len % page));
}

// ------------------------------------------------------------- copy pages
// Whole pages by bulk copies through shared memory: one warp a CTA walks its
// chunks of at most 32 KB, lane 0 issuing; the loads run kAhead chunks before
// the stores, and a slot is loaded again once its store has read it.  No value
// passes through registers, so two warps an SM keep 2 x 96 KB under way.  (1.47 GB
// and 2.61 GB: six slots of 16 KB, three ahead, 245 and 418 us; six, one ahead 264 and
// 451; three of 32 KB, two ahead 241 and 400, one ahead 232 and 382; two of 48 KB 239
// and 401; one warp an SM, three of 64 KB 244 and 406.)
constexpr int kSlots = 3, kAhead = 1, kChunk = 32 * 1024;

__device__ __forceinline__ void bulk_store(void *dst, const void *src, uint32_t bytes)
{
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;\n\t"
                 "cp.async.bulk.commit_group;" ::"l"(dst), "r"(smem_u32(src)), "r"(bytes)
                 : "memory");
}

__global__ void __launch_bounds__(32) kv_copy_kernel(uint8_t *cache, int planes,
                                                     int64_t page_bytes, int P, const int32_t *src,
                                                     const int32_t *dst, const int32_t *count,
                                                     int n, int32_t *status,
                                                     const int32_t *table_in, int32_t *table_out,
                                                     int64_t entries, const int32_t *remap,
                                                     uint64_t wait_ns, int withhold)
{
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ __align__(8) uint64_t full[kSlots];
    __shared__ int abort_flag;
    const int lane = threadIdx.x;
    if (lane == 0) {
        for (int i = 0; i < kSlots; i++)
            mbar_init(&full[i], withhold && i == 0 ? 2 : 1);   // test hook: slot 0 never completes
        abort_flag = 0;
        fence_mbar_init();
    }
    __syncwarp();
    pdl_wait();
    pdl_trigger();
    // a share of the table's entries first (compaction only)
    for (int64_t e = static_cast<int64_t>(blockIdx.x) * 32 + lane; e < entries;
         e += static_cast<int64_t>(gridDim.x) * 32) {
        const int p = table_in[e];
        const bool ok = p >= 0 && p < P;
        if (!ok && p != -1)
            raise_status(status, W4_DEV_BAD_PAGE);
        table_out[e] = ok ? remap[p] : p;
    }
    const int64_t pairs = count ? *count : n, parts = (page_bytes + kChunk - 1) / kChunk;
    const int64_t chunks = pairs * planes * parts;
    uint8_t *to[kAhead];                   // of the chunks loaded and not yet stored (lane 0)
    uint32_t size[kAhead];
    int issued = 0, stored = 0;
    bool ok = true;                        // false once a wait has given up: no more loads, stores
    auto store_next = [&](uint8_t *out, uint32_t bytes) {
        const int slot = stored % kSlots;
        ok = ok && mbar_wait(&full[slot], (stored / kSlots) & 1, &abort_flag, status,
                             kDevPipelineTimeout, wait_ns);
        if (ok) {
            bulk_store(out, ring + slot * kChunk, bytes);
            stored++;
        }
    };
    for (int64_t c0 = blockIdx.x; c0 < chunks; c0 += 32ll * gridDim.x) {
        // the next 32 chunks' places, a lane each: one memory latency for all
        const int64_t c = c0 + static_cast<int64_t>(lane) * gridDim.x;
        int64_t from = -1, into = 0;
        uint32_t bytes = 0;
        if (c < chunks) {
            const int64_t part = c % parts, item = c / parts, plane = item % planes;
            const int64_t i = item / planes;
            const int a = src[i], b = dst[i];
            if (a >= 0 && a < P && b >= 0 && b < P) {
                from = (plane * P + a) * page_bytes + part * kChunk;
                into = (plane * P + b) * page_bytes + part * kChunk;
                bytes = static_cast<uint32_t>(min(static_cast<int64_t>(kChunk),
                                                  page_bytes - part * kChunk));
                if (!W4_IN_BOUNDS(into + bytes <= planes * P * page_bytes, status))
                    from = -1;
            } else if (plane == 0 && part == 0) {
                raise_status(status, W4_DEV_BAD_PAGE);
            }
        }
        for (int l = 0; l < 32; l++) {
            const int64_t f = __shfl_sync(0xffffffffu, from, l), t = __shfl_sync(0xffffffffu, into, l);
            const uint32_t size_l = __shfl_sync(0xffffffffu, bytes, l);
            if (f < 0 || lane != 0 || !ok)
                continue;
            if (issued - stored == kAhead) {
                store_next(to[0], size[0]);
                if (!ok)
                    continue;
#pragma unroll
                for (int u = 0; u + 1 < kAhead; u++) {
                    to[u] = to[u + 1];
                    size[u] = size[u + 1];
                }
            }
            // the store of kSlots chunks ago has read its slot when all but the last
            // kSlots - kAhead have
            if (issued >= kSlots)
                asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kSlots - kAhead) : "memory");
            const int slot = issued % kSlots;
            mbar_arrive_expect_tx(&full[slot], size_l);
            bulk_load_nohint(ring + slot * kChunk, cache + f, size_l, &full[slot]);
#pragma unroll
            for (int u = 0; u < kAhead; u++)
                if (u == issued - stored) {
                    to[u] = cache + t;
                    size[u] = size_l;
                }
            issued++;
        }
    }
    if (lane == 0) {
#pragma unroll
        for (int u = 0; u < kAhead; u++)
            if (stored < issued)
                store_next(to[u], size[u]);
        // after a wait that gave up, the loads still under way land
        for (; stored < issued; stored++)
            mbar_drain(&full[stored % kSlots], (stored / kSlots) & 1);
        asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }
}

// ---------------------------------------------------------------- compact
// Pages in use behind the first `live` pages (movers) go to the free ones
// among those (holes), k-th to k-th: sources and destinations never overlap.
__global__ void __launch_bounds__(kPlanThreads) kv_compact_plan_kernel(
    const int32_t *refs, int32_t *refs_out, int P, int32_t *count, int32_t *src, int32_t *dst,
    int32_t *remap, int32_t *status)
{
    __shared__ int sums[2][33];
    const int tid = threadIdx.x;
    pdl_wait();
    pdl_trigger();
    int mine = 0;
    for (int p = tid; p < P; p += kPlanThreads)
        mine += refs[p] > 0;
    int live;
    block_exclusive_sum(mine, sums[0], &live);
    int holes = 0, movers = 0;
    for (int p0 = 0, round = 1; p0 < P; p0 += kPlanThreads, round ^= 1) {
        const int p = p0 + tid;
        const bool in = p < P, used = in && refs[p] > 0;
        const bool hole = in && !used && p < live, mover = used && p >= live;
        // holes lie before `live` and movers behind it: one sum serves both,
        // in the round that contains `live` as two halves of a word
        int total;
        const int before = block_exclusive_sum(hole + (mover << 16), sums[round], &total);
        // as many movers as holes: half of the pages at most
        if (hole && W4_IN_BOUNDS(holes + (before & 0xFFFF) < P / 2, status))
            dst[holes + (before & 0xFFFF)] = p;
        if (mover && W4_IN_BOUNDS(movers + (before >> 16) < P / 2, status))
            src[movers + (before >> 16)] = p;
        if (in)
            remap[p] = p;
        holes += total & 0xFFFF;
        movers += total >> 16;
    }
    if (tid == 0)
        *count = movers;
    if (refs_out != refs)
        for (int p = tid; p < P; p += kPlanThreads)
            refs_out[p] = refs[p];
    __syncthreads();
    for (int i = tid; i < movers; i += kPlanThreads) {
        const int a = src[i], b = dst[i];
        if (!W4_IN_BOUNDS(a >= 0 && a < P && b >= 0 && b < P, status))
            continue;
        remap[a] = b;
        refs_out[b] = refs[a];
        refs_out[a] = 0;
    }
}

// ----------------------------------------------------------------- append
// CTA (b, y): sequence b's new tokens y, y + gridDim.y, ... eight at a time, a
// warp each.
struct AppendArgs {
    uint16_t *kp, *vp;
    const uint16_t *k, *v;
    const int32_t *table, *lens, *q_offsets;
    int32_t *status;
    int64_t page_stride, tok_stride, head_stride;
    int64_t k_tok, k_head, v_tok, v_head;
    int P, page, Hkv, D, B, W, T;
};

__global__ void __launch_bounds__(256) kv_append_kernel(const AppendArgs p)
{
    pdl_wait();
    pdl_trigger();
    const int b = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int t0 = p.q_offsets[b], t1 = p.q_offsets[b + 1], len = p.lens[b];
    if (t0 < 0 || t1 < t0 || t1 > p.T) {
        if (blockIdx.y == 0 && threadIdx.x == 0)
            raise_status(p.status, W4_DEV_BAD_SLOT);
        return;
    }
    const int vecs = p.D / 8;
    constexpr int kUnroll = 4;
    for (int t = t0 + blockIdx.y * 8 + warp; t < t1; t += gridDim.y * 8) {
        const int pos = len - (t1 - t);
        const int e = pos / p.page;
        const int pg = pos >= 0 && e < p.W ? p.table[static_cast<int64_t>(b) * p.W + e] : -1;
        if (pg < 0 || pg >= p.P) {
            if (lane == 0)
                raise_status(p.status, W4_DEV_BAD_PAGE);
            continue;
        }
        if (!W4_IN_BOUNDS(pos - e * p.page >= 0 && pos - e * p.page < p.page, p.status))
            continue;
        const int64_t to = pg * p.page_stride + (pos - e * p.page) * p.tok_stride;
        // kUnroll 16-byte values of k and of v in flight a lane
        for (int i0 = lane; i0 < p.Hkv * vecs; i0 += 32 * kUnroll) {
            int4 kv[kUnroll], vv[kUnroll];
            int64_t at[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; u++) {
                const int i = i0 + 32 * u, h = i / vecs, c = (i - h * vecs) * 8;
                at[u] = to + h * p.head_stride + c;
                if (i < p.Hkv * vecs) {
                    kv[u] = __ldcs(reinterpret_cast<const int4 *>(p.k + t * p.k_tok +
                                                                  h * p.k_head + c));
                    vv[u] = __ldcs(reinterpret_cast<const int4 *>(p.v + t * p.v_tok +
                                                                  h * p.v_head + c));
                }
            }
#pragma unroll
            for (int u = 0; u < kUnroll; u++)
                if (i0 + 32 * u < p.Hkv * vecs) {
                    *reinterpret_cast<int4 *>(p.kp + at[u]) = kv[u];
                    *reinterpret_cast<int4 *>(p.vp + at[u]) = vv[u];
                }
        }
    }
}

int sm_count()
{
    int dev = 0, sms = 0;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    return std::max(sms, 1);
}

cudaError_t raise_copy_limit()
{
    static std::atomic<uint64_t> raised{0};      // devices whose limit is raised already
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess || (raised.load(std::memory_order_relaxed) >> (dev & 63) & 1u))
        return err;
    err = cudaFuncSetAttribute(kv_copy_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               kSlots * kChunk);
    if (err == cudaSuccess)
        raised.fetch_or(1ull << (dev & 63), std::memory_order_relaxed);
    return err;
}

}  // namespace

cudaError_t launch_kv_reserve(int32_t *table, int B, int W, int32_t *lens, int32_t *refs, int P,
                              const int32_t *slots, const int32_t *new_lens, int n, int page,
                              int32_t *status, cudaStream_t stream)
{
    return launch_pdl(kv_reserve_kernel, dim3(1), dim3(kPlanThreads), 0, stream, table, B, W, lens,
                      refs, P, slots, new_lens, n, page, status);
}

cudaError_t launch_kv_free(int32_t *table, int B, int W, int32_t *lens, int32_t *refs, int P,
                           const int32_t *slots, int n, int32_t *status, cudaStream_t stream)
{
    const int y = std::min((W + 255) / 256, 64);
    return launch_pdl(kv_free_kernel, dim3(n, y), dim3(256), 0, stream, table, B, W, lens, refs, P,
                      slots, status);
}

cudaError_t launch_kv_fork(uint8_t *cache, int planes, int64_t page_bytes, int32_t *table, int B,
                           int W, int32_t *lens, int32_t *refs, int P, const int32_t *parents,
                           const int32_t *children, int n, int page, void *workspace,
                           int32_t *status, cudaStream_t stream)
{
    int2 *plan = static_cast<int2 *>(workspace);
    cudaError_t err =
        launch_pdl(kv_fork_plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, table, B, W, lens,
                   refs, P, parents, children, n, page, plan, status);
    if (err != cudaSuccess)
        return err;
    return launch_pdl(kv_fork_kernel, dim3(n, planes), dim3(256), 0, stream, cache, page_bytes,
                      table, W, static_cast<const int32_t *>(lens), refs, P, children, page,
                      static_cast<const int2 *>(plan), status);
}

cudaError_t launch_kv_copy(uint8_t *cache, int planes, int64_t page_bytes, int P,
                           const int32_t *src, const int32_t *dst, int n, int32_t *status,
                           cudaStream_t stream)
{
    const int64_t chunks = static_cast<int64_t>(n) * planes * ((page_bytes + kChunk - 1) / kChunk);
    cudaError_t err = raise_copy_limit();
    if (err != cudaSuccess)
        return err;
    const int grid = static_cast<int>(std::min<int64_t>(chunks, 2ll * sm_count()));
    return launch_pdl(kv_copy_kernel, dim3(grid), dim3(32), kSlots * kChunk, stream, cache, planes,
                      page_bytes, P, src, dst, static_cast<const int32_t *>(nullptr), n, status,
                      static_cast<const int32_t *>(nullptr), static_cast<int32_t *>(nullptr),
                      static_cast<int64_t>(0), static_cast<const int32_t *>(nullptr),
                      pipeline_test_hooks().wait_ns,
                      static_cast<int>(pipeline_test_hooks().withhold_sz));
}

cudaError_t launch_kv_compact(uint8_t *cache, int planes, int64_t page_bytes, const int32_t *table,
                              int64_t entries, const int32_t *refs, int P, int32_t *table_out,
                              int32_t *refs_out, void *workspace, int32_t *status,
                              cudaStream_t stream)
{
    int32_t *count = static_cast<int32_t *>(workspace), *src = count + 4;
    int32_t *dst = src + P / 2, *remap = dst + P / 2;
    cudaError_t err = launch_pdl(kv_compact_plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream,
                                 refs, refs_out, P, count, src, dst, remap, status);
    if (err != cudaSuccess)
        return err;
    err = raise_copy_limit();
    if (err != cudaSuccess)
        return err;
    return launch_pdl(kv_copy_kernel, dim3(2 * sm_count()), dim3(32), kSlots * kChunk, stream, cache,
                      planes, page_bytes, P, static_cast<const int32_t *>(src),
                      static_cast<const int32_t *>(dst), static_cast<const int32_t *>(count), 0,
                      status, table, table_out, entries, static_cast<const int32_t *>(remap),
                      pipeline_test_hooks().wait_ns,
                      static_cast<int>(pipeline_test_hooks().withhold_sz));
}

size_t kv_workspace_bytes(int P, int n)
{
    // compaction: a count, two lists of at most P / 2 pages, the map; fork: its plan
    return std::max(16 + 4 * (2 * static_cast<size_t>(P / 2) + P), 8 * static_cast<size_t>(n));
}

cudaError_t launch_kv_append(const KvAppend &q, cudaStream_t stream)
{
    AppendArgs a{};
    a.kp = q.k_pages;
    a.vp = q.v_pages;
    a.k = q.k;
    a.v = q.v;
    a.table = q.table;
    a.lens = q.lens;
    a.q_offsets = q.q_offsets;
    a.status = q.dev_status;
    a.page_stride = q.page_stride;
    a.tok_stride = q.tok_stride;
    a.head_stride = q.head_stride;
    a.k_tok = q.k_tok;
    a.k_head = q.k_head;
    a.v_tok = q.v_tok;
    a.v_head = q.v_head;
    a.P = q.P;
    a.page = q.page;
    a.Hkv = q.Hkv;
    a.D = q.D;
    a.B = q.B;
    a.W = q.W;
    a.T = q.T;
    // about one warp per token of an average sequence
    const int y = std::min(std::max((q.T / q.B + 7) / 8, 1), 1024);
    return launch_pdl(kv_append_kernel, dim3(q.B, y), dim3(256), 0, stream, a);
}

}  // namespace w4
