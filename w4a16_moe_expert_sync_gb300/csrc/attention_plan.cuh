// attention_plan.cuh -- how attention's work is split and where its pieces and
// fills are: pure index functions, which the kernels and a test on the host compile
// alike.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define W4_PLAN __host__ __device__ __forceinline__
#else
#define W4_PLAN inline
#endif

namespace w4 {
namespace plan {

constexpr int kRows = 128;                 // rows of a stream's tile
constexpr int kKeys = 128;                 // keys of a tile

// An item is kItemCost + its tiles long when the work is split: fetching its
// queries and storing its sums takes about as long as that many tiles.  (With 1
// and 3 instead of 2: 64 ragged sequences behind 8192 tokens 61.4 and 60.4 us
// against 58.6, four canvases of 256 queries 57.0 and 47.5 against 46.7, nine small
// groups 25.8 and 27.3 against 26.3.)
constexpr int kItemCost = 2;
// A CTA's time for a single tile in those of a pair's, as the CTAs are divided
// between the two.  (With 0.5, 0.7, 1.0: 120,000 shared tokens and short tails 84.6,
// 73.6 and 75.7 us, nine small groups 27.6, 26.2 and 27.4.  Both kinds on every CTA, the
// pairs first: 74.1 and 32.7.)
constexpr float kSingleWeight = 0.7f;

W4_PLAN int smaller(int a, int b) { return a < b ? a : b; }
W4_PLAN int larger(int a, int b) { return a > b ? a : b; }

// Worker w's share of a region's `all` begins here.
W4_PLAN int worker_begin(int all, int workers, int w)
{
    if (all < (1 << 22))                       // workers <= 512: 32 bits do
        return static_cast<int>(static_cast<uint32_t>(all) * w / workers);
    return static_cast<int>(static_cast<int64_t>(all) * w / workers);
}
// The worker whose share place x is in.
W4_PLAN int worker_of(int all, int workers, int x)
{
    if (all < (1 << 22))                       // workers <= 512: 32 bits do
        return static_cast<int>((static_cast<uint32_t>(x + 1) * workers - 1) / all);
    return static_cast<int>((static_cast<int64_t>(x + 1) * workers - 1) / all);
}
// How many CTAs take the pairs; the others, two streams each, take the single
// items.  No worker goes without a share.
W4_PLAN int pair_ctas(int singles, int pairs, int grid)
{
    if (pairs == 0 || singles == 0)
        return smaller(pairs, grid);
    const float part = pairs / (pairs + kSingleWeight * singles);
    return smaller(pairs,
                   larger(1, smaller(grid - 1, static_cast<int>(part * grid + 0.5f))));
}

// The tiles of an entry's keys k0 .. k1, which start where k0's page does.
W4_PLAN int key_tiles(int k0, int k1, int page_shift)
{
    return (k1 - (k0 >> page_shift << page_shift) + kKeys - 1) / kKeys;
}
// Whether an entry of `rows` rows is taken as pairs, and its items per kv head.
W4_PLAN bool is_pair(int rows) { return rows > kRows; }
W4_PLAN int row_tiles(int rows)
{
    return is_pair(rows) ? (rows + 2 * kRows - 1) / (2 * kRows) : 1;
}
// The tiles, from the first on, that a sequence's rows up to `last` see when causal:
// none sees beyond its own token's position.
W4_PLAN int causal_tiles(int k1, int tokens, int base, int last, int rep)
{
    const int limit = k1 - tokens + last / rep + 1;
    return (larger(limit - base, 0) + kKeys - 1) / kKeys;
}

// Which pair of fills (K, then V) a stream's tile r of its single items is: the loader
// takes the streams' tiles in turn, and a stream that has none left drops out.  A
// CTA has pairs, whose tile r is fill r, or single items.
W4_PLAN int fill_of(int tiles0, int tiles1, int which, int r)
{
    return which == 2 ? r : r + (which == 0 ? smaller(r, tiles1) : smaller(r + 1, tiles0));
}

// How many pieces a workspace holds: of pairs, of groups' single items, of all single
// items.  Each of up to `grid` CTAs (two workers each for single items) cuts at most
// one item more.  An entry of R > 128 rows has at most R / 128 pair items, and a row
// is in two entries; groups come first among the single items.
struct Caps {
    int pairs, groups, singles;
};
W4_PLAN Caps caps_of(int64_t T, int64_t rep, int B, int G, int Hkv, int grid)
{
    const int64_t pairs = 2 * T * rep / kRows * Hkv;
    Caps c;
    c.pairs = static_cast<int>(pairs < (1 << 24) ? pairs : 1 << 24) + grid;
    c.groups = G * Hkv + 2 * grid;
    c.singles = c.groups + B * Hkv;
    return c;
}

}  // namespace plan
}  // namespace w4
