// paged_chunk_attn.cu -- attention of chunks of new tokens over a paged cache
// whose K and V are e4m3 with one scale per (page, KV head): for row t and head
// h of group g, over the tokens j <= pos(t) of the blocks selected for (t, g)
// (or of every block),
//   l_j = scale ks <q, k_j>,  P = softmax(l),  o = sum_j P_j vs v_j,
//   lse = log sum_j exp(l_j).
//
// The rows of a chunk read the same pages, so the (row, head) pairs of a
// request and group are the rows of two products with a page,
//   S [128 pairs][128 tokens] = Q K^T,  O [128 pairs][d] += P V,
// and with a few hundred rows to a page the tensor cores bound it: 4 x 128 x 128
// x d operations a page and 128 pairs.  A tile has 256 pairs (256 / G rows): two
// halves, A and B, whose products alternate on the tensor cores while the other
// half's scores become probabilities.  2,048 rows of 64 heads over 32,768 tokens
// take this kernel 1,780 us (1,196 TFLOP/s; the call, with the tiles' plan and the
// joining, 1,866), where the tensor cores' rate gives 1,088: a page takes some
// 3,500 cycles, of which the products need 2,050 (the tensor pipe is 41% active,
// shared memory 27% busy); the conversion of the codes, 2,800 of its warps', and the
// softmax, 2,300 of each half's, share the issue slots and wait for one another, so
// that every handover between them counts.  The halves' issuers take turns: when
// both issue at once the products get in one another's way (2,240 us).
//
// Codes to 16 bits.  e4m3 products would need queries and probabilities as pairs
// of e4m3 terms, and small probabilities as several levels of those.  So four
// warps turn the codes into 16-bit tiles, once a page for both halves (one value
// converted to a probability computed): K to fp16, which is one instruction for
// two codes, against queries brought to fp16 by a power of two for each row and
// head; V to bf16, so that probabilities keep their 8 bits at any size, which
// takes five.  Those 8 bits put outputs 2.3e-3 off (relative, a whole tensor), where
// their own rounding to bf16 makes 1.7e-3; fp16 has 11, but down to 2^-14 only.
//
// Softmax.  With t_j = l_j log2 e + lv, 2^lv the page's V scale over that of the
// stretch's first page of the tile (2^base), the weight of token j's codes is
// P = 2^(t_j - m) and its part of the sum P 2^-lv, so one reference m per row does
// for both and P V adds up in TMEM across pages of different scales.  bf16 and fp32
// keep their bits at any size, so m need not be the largest t, only within 2^kFar
// of it: it is that of the row's first page, and the pages after it are searched for
// a larger one only if the codes' largest value, 448, times the row's sum of |q|
// could pass 2^kFar times the reference.  Otherwise the scores are read once.  P
// (bf16) takes their place in TMEM and is read from there as the A operand.
//
// What keeps the sums finite: with P up to 2^kFar and the 2^30 tokens that a table
// can name, P V ends below 2^(89 + 8.9 + 30), and the row's sum below
// 2^(89 + 30 + kBelow) if no lv is below -kBelow: a page whose scale is smaller than
// that, zeros for one (which are appended with 2^-112), has lv = -kBelow and what is
// left, pv < 1, on its P.  Scales above 2^(base + kAbove) leave a pv > 1: there the
// largest score is always looked for.  kAbove keeps the sum of a row that only sees
// such pages, and what other pages add to it, well inside fp32; the bounds on base
// leave pv at 2^67 at most, so that P V stays finite with it.
//
// A NaN code must not reach rows that do not see its token, and 0 x NaN does:
// NaNs of V enter the products as 0, and rows that see one (looked for only
// then) get theirs when they are written.
//
// With a selection, a tile walks the union of its rows' blocks (made by a kernel
// before, with a bit to each row that selected the block).  3,000 rows of 32 heads
// that selected 16 of up to 391 blocks each take this kernel 540 us (the call, with
// the plan, the unions and the joining, 607): the unions of 32 rows have
// 47 blocks, three times what a row selected.
// The work is one list of products, those of (tile 0, group 0), (tile 0, group 1)
// and so on, cut into equal stretches for persistent CTAs.  A stretch cuts at
// most two tiles; those pieces' states go to the workspace, and a kernel after
// joins them, in the order of their pages.  A tile of up to 128 pairs has only half
// A: its pages go to the two halves in turn, both with the same queries, and A joins them.
//   warps 0..3, 4..7   softmax of half A, B, a pair to a thread
//   warps 8..11        codes of K and V to 16-bit tiles in shared memory, loaded a tile ahead
//   warps 12, 13       tcgen05.mma issuers of half A, B
//   warp 14            planner: pages, scales and masks, through a ring
#include <algorithm>
#include <climits>
#include <type_traits>

#include "paged_chunk.h"
#include "tc.cuh"

namespace msa {

size_t paged_chunk_scores_scratch(const PagedProblem &p);

namespace {

using namespace tc;

constexpr int kSoftWarps = 8, kCodeWarps = 4;
constexpr int kCode0 = kSoftWarps, kMma = kCode0 + kCodeWarps, kPlanner = kMma + 2;
constexpr int kThreads = 32 * (kPlanner + 1);
constexpr int kStages = 2;                    // K and V tiles
constexpr int kRing = 8;                      // pages the planner is ahead
constexpr int kSub = 128 * 128;               // [128 rows][64 bf16], swizzled
constexpr int kLeast = 4;                     // products to a stretch at least, where an item has as many
// log2 of what a probability may outgrow its reference by where it has been looked at, and where it cannot by more.
constexpr float kLag = 8.f, kFar = 89.f;
// log2 of how far a page's V scale is taken into t below and above the first page's, and of the largest and least of that.
constexpr int kBelow = 8, kAbove = 90, kBase = 30;
constexpr int kMaskWords = kTileRows / 64;    // with a selection, a bit to each row of a tile (at most 128, with G = 1)
constexpr int kNoBlock = 1 << 23;             // behind any block of a table
constexpr int kWindow = 1 << 15;              // blocks whose union is taken in one go
constexpr int kListWarps = 4;

// mbar_wait_warp of tc.cuh with its failure out of line: it is in two dozen places, and the kernel's code has to stay in the
// instruction cache (at 180 KB every wait cost 400 cycles, and a page 12,000 instead of 3,000).
__device__ __forceinline__ void gave_up(DeviceStatus *st, int site, int parity, volatile int *abort_flag)
{
    report(st, kDevTimeout, site, parity);
    *abort_flag = 1;
}
__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, DeviceStatus *st, int site, volatile int *abort_flag)
{
    bool ok = mbar_try_wait(bar, parity);
    for (uint32_t it = 0; !ok; ++it) {
        ok = mbar_try_wait(bar, parity);
        if ((it & 1023u) != 1023u || ok) continue;
        if (*abort_flag) break;
        if (it >= (1u << 21)) {                // seconds
            gave_up(st, site, (int)parity, abort_flag);
            break;
        }
    }
    return __all_sync(0xffffffffu, ok);
}

enum Kind { kPageEntry = 0, kEndEntry = 1, kExit = 2 };

struct Entry {                 // a page of the ring
    int kind, item, page, block;
    int halves, first;         // bits of the halves that take it; of those whose first page it is
    float a, lv, il, pv;       // logits' factor, log2 of the V scale over 2^base (cut off), 2^-lv, and what lv leaves of it (1)
    uint32_t mask[kMaskWords];
};
struct Item {                  // a tile's piece
    int row, rows, req, group, part;    // part: the piece's place among the partial states; -1: a whole tile
    int split;                 // one half's pairs, pages in turn
    int c0, c1;
    int base;                  // log2 of the V scale that its sums are in
    long long at;              // of the tile's list
};

template <int D>
struct AttnSmem {
    static constexpr int KB = D / 64, TILE = KB * kSub;
    static constexpr int OFF_K = 2 * TILE, OFF_V = OFF_K + kStages * TILE, OFF_RING = OFF_V + kStages * TILE;
    static constexpr int OFF_ITEM = OFF_RING + kRing * (int)sizeof(Entry);
    static constexpr int OFF_STATE = OFF_ITEM + kRing * (int)sizeof(Item);      // half B's (m, z) of a split tile
    static constexpr int OFF_BAR = OFF_STATE + 128 * 8;
    static constexpr int BYTES = OFF_BAR + 512 + 1024;
    // one CTA, which takes all 512 TMEM columns, to an SM
    static constexpr int ALLOC = BYTES > 120 * 1024 ? BYTES : 120 * 1024;
};
static_assert(AttnSmem<128>::ALLOC <= 227 * 1024, "shared memory");
static_assert(sizeof(Entry) % 8 == 0 && sizeof(Item) % 8 == 0, "alignment of what follows");

// The plan's numbers for attention: with a selection, the work and pages of each (tile, group), and the unions.
struct AttnPlan {
    ChunkPlan tiles;
    long long *before;         // by item (tile, group), with a selection
    int *pages;                // of an item
    int *blocks;               // the items' unions, each at (row * Hkv + group * rows) * topk
    uint32_t *masks;
    float *part;               // partial states: [slot][256][D] sums, then [slot][256] (m, z)
    size_t bytes;
    __host__ __device__ AttnPlan(void *at, long long most, const PagedProblem &p, size_t plan_bytes, bool listed, int words, int ctas)
        : tiles(at, most)
    {
        char *c = static_cast<char *>(at) + plan_bytes;
        auto take = [&](size_t n) {
            char *r = c;
            c += (n + 255) / 256 * 256;
            return r;
        };
        const size_t items = (size_t)most * p.Hkv, entries = (size_t)p.T * p.Hkv * p.topk;
        before = reinterpret_cast<long long *>(take(listed ? (items + 1) * 8 : 0));
        pages = reinterpret_cast<int *>(take(listed ? items * 4 : 0));
        blocks = reinterpret_cast<int *>(take(listed ? entries * 4 : 0));
        masks = reinterpret_cast<uint32_t *>(take(listed ? entries * words * 4 : 0));
        part = reinterpret_cast<float *>(take((size_t)ctas * 2 * kTileRows * (p.d + 2) * 4));
        bytes = c - static_cast<char *>(at);
    }
    __host__ __device__ float2 *stats(int ctas, int d) const { return reinterpret_cast<float2 *>(part + (size_t)ctas * 2 * kTileRows * d); }
};

struct Args {
    PagedProblem p;
    const bf16 *q;
    const uint8_t *k8, *v8;
    const float *k_scale, *v_scale;
    const int32_t *block_table, *row_pos, *sel;
    bf16 *o;
    float *lse;
    int tokens, words, ctas;   // rows of a tile, mask words of an entry
    int shift;                 // log2 G
    DeviceStatus *st;
};

// ---------------------------------------------------------------- unions of a selection
// fn(block) for each entry of row t's selection that counts; returns false where one does not.
template <class F>
__device__ __forceinline__ bool selected(const PagedProblem &p, const int32_t *sel, int t, int g, int pos, F fn)
{
    const int32_t *s = sel + ((long long)t * p.Hkv + g) * p.topk;
    const int c_last = pos / kPage, entries = min(p.topk, c_last + 1);
    int prev = -1;
    bool fine = true;
    for (int i0 = 0; i0 < p.topk; i0 += 8) {
        int c[8];                              // eight loads in flight: one after another they were most of the kernel
#pragma unroll
        for (int j = 0; j < 8; ++j) c[j] = i0 + j < p.topk ? s[i0 + j] : -1;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (c[j] == -1) continue;
            if (i0 + j >= entries || c[j] <= prev || c[j] > c_last) {
                fine = false;
                continue;
            }
            prev = c[j];
            fn(c[j]);
        }
    }
    return fine;
}

// A warp to an item: a bitmap of the blocks, their numbers in order, then a bit to each row that has them.
__global__ void __launch_bounds__(32 * kListWarps)
chunk_list_kernel(Args a, AttnPlan plan)
{
    __shared__ uint32_t bits[kListWarps][kWindow / 32];
    __shared__ int rank[kListWarps][kWindow / 32];
    chain_next();
    chain_wait(a.row_pos, a.sel, a.o, a.lse);
    const PagedProblem &p = a.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long items = (long long)*plan.tiles.n_tiles * p.Hkv;
    for (long long it = (long long)blockIdx.x * kListWarps + warp; it < items; it += (long long)gridDim.x * kListWarps) {
        const int i = (int)(it / p.Hkv), g = (int)(it % p.Hkv);
        const ChunkTile t = plan.tiles.tiles[i];
        const long long at = ((long long)t.row * p.Hkv + (long long)g * t.rows) * p.topk;
        int n = 0;
        for (int w0 = 0; w0 < t.pages; w0 += kWindow) {
            const int words = min(kWindow, t.pages - w0 + 31) / 32;
            for (int w = lane; w < words; w += 32) bits[warp][w] = 0;
            __syncwarp();
            for (int j = lane; j < t.rows; j += 32) {
                const int pos = a.row_pos[t.row + j];
                if (pos < 0 || (long long)pos >= (long long)p.max_blocks * kPage) continue;
                const bool fine = selected(p, a.sel, t.row + j, g, pos, [&](int c) {
                    const int b = c - w0;
                    if (b >= 0 && b < words * 32) atomicOr(&bits[warp][b >> 5], 1u << (b & 31));
                });
                if (!fine && w0 == 0) report(a.st, kDevCheck, 180, t.row + j);
            }
            __syncwarp();
            for (int v0 = 0; v0 < words; v0 += 32) {
                uint32_t m = v0 + lane < words ? bits[warp][v0 + lane] : 0;
                int in = __popc(m);
                const int mine = in;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, in, o);
                    if (lane >= o) in += y;
                }
                int pos = n + in - mine;
                if (v0 + lane < words) rank[warp][v0 + lane] = pos;
                for (; m; m &= m - 1, ++pos) {
                    plan.blocks[at + pos] = w0 + (v0 + lane) * 32 + __ffs(m) - 1;
                    for (int w = 0; w < a.words; ++w) plan.masks[(at + pos) * a.words + w] = 0;
                }
                n += __shfl_sync(0xffffffffu, in, 31);
            }
            __threadfence();
            __syncwarp();
            for (int j = lane; j < t.rows; j += 32) {
                const int pos = a.row_pos[t.row + j];
                if (pos < 0 || (long long)pos >= (long long)p.max_blocks * kPage) continue;
                selected(p, a.sel, t.row + j, g, pos, [&](int c) {
                    const int b = c - w0;
                    if (b < 0 || b >= words * 32) return;
                    const int r = rank[warp][b >> 5] + __popc(bits[warp][b >> 5] & ((1u << (b & 31)) - 1));
                    atomicOr(&plan.masks[(at + r) * a.words + (j >> 5)], 1u << (j & 31));
                });
            }
            __syncwarp();
        }
        if (lane == 0) plan.pages[it] = n;
        // without any block: no work, and nobody else writes these rows
        for (int j = lane; n == 0 && j < t.rows * p.G; j += 32) {
            const int pos = a.row_pos[t.row + j / p.G];
            if (pos < 0 || (long long)pos >= (long long)p.max_blocks * kPage) continue;
            const long long row = (long long)(t.row + j / p.G) * p.Hq + g * p.G + j % p.G;
            for (int w = 0; w < p.d / 8; ++w) reinterpret_cast<uint4 *>(a.o + row * p.d)[w] = make_uint4(0, 0, 0, 0);
            a.lse[row] = -INFINITY;
        }
    }
}

// One CTA: the work before each item.
__global__ void __launch_bounds__(1024) chunk_sum_kernel(Args a, AttnPlan plan)
{
    __shared__ long long buf[32];
    chain_next();
    chain_wait(a.row_pos);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long items = (long long)*plan.tiles.n_tiles * a.p.Hkv;
    long long sum = 0;
    for (long long i0 = 0; i0 < items; i0 += 1024) {
        const long long i = i0 + tid;
        const long long x = i < items ? (long long)plan.pages[i] * tile_halves(plan.tiles.tiles[i / a.p.Hkv].rows * a.p.G) : 0;
        long long in = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, in, o);
            if (lane >= o) in += y;
        }
        __syncthreads();
        if (lane == 31) buf[warp] = in;
        __syncthreads();
        long long before = 0, all = 0;
        for (int w = 0; w < 32; ++w) {
            if (w < warp) before += buf[w];
            all += buf[w];
        }
        if (i < items) plan.before[i] = sum + before + in - x;
        sum += all;
    }
    if (tid == 0) plan.before[items] = sum;
}

// ---------------------------------------------------------------- stretches
// The pieces of a stretch.  Items are (tile, group), groups inside.
struct Pieces {
    const AttnPlan &plan;
    const Args &a;
    int n_items;                // at most rows x groups
    long long total;
    __device__ Pieces(const AttnPlan &pl, const Args &ar) : plan(pl), a(ar)
    {
        const int n = *pl.tiles.n_tiles;
        n_items = n * ar.p.Hkv;
        total = ar.sel ? pl.before[n_items] : pl.tiles.before[n] * ar.p.Hkv;
    }
    // Units of a stretch at least: an item costs as much as four to five pages to begin and end, and one that is cut has to be
    // joined, so items of a few pages stay whole, but no CTA takes a second one for having too little to do (13 rows over one
    // page, 8 items: 46 us in two CTAs, 18 in eight).
    __device__ int least() const { return (int)max(1ll, min((long long)kLeast, (total + n_items - 1) / max(n_items, 1))); }
    // the item that unit w is in, by a whole warp
    __device__ int find(long long w, int lane) const
    {
        if (a.sel) return chunk_find(plan.before, n_items, 1, w, lane);
        const int i = chunk_find(plan.tiles.before, *plan.tiles.n_tiles, a.p.Hkv, w, lane);
        const long long in = w - plan.tiles.before[i] * a.p.Hkv, one = plan.tiles.before[i + 1] - plan.tiles.before[i];
        return i * a.p.Hkv + (int)(in / one);
    }
    __device__ long long start(int item) const
    {
        if (a.sel) return plan.before[item];
        const int i = item / a.p.Hkv;
        const long long one = plan.tiles.before[i + 1] - plan.tiles.before[i];
        return plan.tiles.before[i] * a.p.Hkv + one * (item % a.p.Hkv);
    }
    __device__ int pages(int item) const { return a.sel ? plan.pages[item] : plan.tiles.tiles[item / a.p.Hkv].pages; }
};

// Pages [c0, c1) of an item of `pages` pages from unit `start` on that are [from, to)'s, a page where its first unit is.
__device__ __forceinline__ void cut(long long start, int pages, int mt, long long from, long long to, int &c0, int &c1)
{
    const long long off = max(0ll, from - start), stop = max(0ll, min((long long)pages * mt, to - start));
    c0 = (int)((off + mt - 1) >> (mt - 1));            // mt is 1 or 2
    c1 = (int)((stop + mt - 1) >> (mt - 1));
}

// ---------------------------------------------------------------- the kernel
// Two e4m3 codes to fp16, exactly (a NaN to a NaN).
__device__ __forceinline__ uint32_t widen(uint16_t codes)
{
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;\n" : "=r"(r) : "h"(codes));
    return r;
}
__device__ __forceinline__ uint32_t to_bf16(uint32_t h)
{
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
    return pack_bf16(f.x, f.y);
}
// The codes among four that are NaN (0x7F, 0xFF), bit 7 of each byte.
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }

// A tile's codes as the four warps take them: 16 at a time, eight tokens by 64 features to a warp's load, so that eight
// lanes store to eight different places of the swizzle.
template <int D>
struct Place {
    int token, feature;        // of a thread's first 16 codes; the next ones are kStep tokens on
    static constexpr int kStep = D == 128 ? 16 : 32;
    __device__ explicit Place(int tid)
    {
        const int w = tid >> 5, lane = tid & 31;
        token = (D == 128 ? w >> 1 : w) * 8 + (lane & 7);
        feature = (D == 128 ? (w & 1) * 64 : 0) + (lane >> 3) * 16;
    }
};
// Writes this thread's words of a tile of 128 tokens, K as fp16, V as bf16; of V, true where a code is NaN (to be mended).
template <int D, bool V>
__device__ __forceinline__ bool lay_down(uint8_t *tile, const uint4 (&u)[D / 16], const Place<D> &at)
{
    const int c = (at.feature & 63) >> 3, r = at.token & 7;
    uint8_t *row = tile + (at.feature >> 6) * kSub + at.token * 128;
    uint8_t *place[2] = {row + ((c ^ r) << 4), row + (((c + 1) ^ r) << 4)};
    __half2 sum = __float2half2_rn(0.f);           // at most 64 codes of at most 448
#pragma unroll
    for (int j = 0; j < D / 16; ++j) {
        const uint32_t w[4] = {u[j].x, u[j].y, u[j].z, u[j].w};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t x[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t y = w[2 * h + (k >> 1)];
                x[k] = widen((uint16_t)(k & 1 ? y >> 16 : y));
                if constexpr (V) {
                    sum = __hadd2(sum, *reinterpret_cast<const __half2 *>(&x[k]));
                    x[k] = to_bf16(x[k]);
                }
            }
            *reinterpret_cast<uint4 *>(place[h] + j * Place<D>::kStep * 128) = make_uint4(x[0], x[1], x[2], x[3]);
        }
    }
    return V && (__hisnan(__low2half(sum)) || __hisnan(__high2half(sum)));
}
// Its NaNs of V to 0.
template <int D>
__device__ __forceinline__ void mend(uint8_t *tile, const uint8_t *codes, const Place<D> &p)
{
#pragma unroll 1
    for (int j = 0; j < D / 16; ++j) {
#pragma unroll 1
        for (int k = 0; k < 16; ++k) {
            const int r = p.token + j * Place<D>::kStep, f = p.feature + k;
            if ((codes[r * D + f] & 0x7F) != 0x7F) continue;
            *reinterpret_cast<uint16_t *>(tile + (f >> 6) * kSub + r * 128 + ((((f & 63) >> 3) ^ (r & 7)) << 4) + (f & 7) * 2) = 0;
        }
    }
}

// The NaN features of the visible tokens' V codes into a row that has been written.
template <int D>
__device__ __forceinline__ void spoil(const Args &a, const AttnPlan &plan, const Item &it, int pos, int token, float *part, bf16 *o)
{
#pragma unroll 1
    for (int c = it.c0; c < it.c1; ++c) {
        const int block = a.sel ? plan.blocks[it.at + c] : c, page = a.block_table[(long long)it.req * a.p.max_blocks + block];
        if ((unsigned)page >= (unsigned)a.p.n_pages) continue;
        if (a.sel && !(plan.masks[(it.at + c) * a.words + (token >> 5)] >> (token & 31) & 1)) continue;
        const uint4 *row = reinterpret_cast<const uint4 *>(a.v8 + ((long long)page * a.p.Hkv + it.group) * kPage * D);
#pragma unroll 1
        for (int j = 0; j < kPage && block * kPage + j <= pos; ++j)
#pragma unroll 1
            for (int w = 0; w < D / 16; ++w) {
                const uint4 u = row[j * (D / 16) + w];
                if (!(nan_codes(u.x) | nan_codes(u.y) | nan_codes(u.z) | nan_codes(u.w))) continue;
                const uint8_t *codes = reinterpret_cast<const uint8_t *>(row + j * (D / 16) + w);
#pragma unroll 1
                for (int k = 0; k < 16; ++k) {
                    if ((codes[k] & 0x7F) != 0x7F) continue;
                    const int f = w * 16 + k;
                    if (part) part[f] = __uint_as_float(0x7FC00000u);
                    else o[f] = __ushort_as_bfloat16(0x7FC0);
                }
            }
    }
}

__device__ __forceinline__ uint64_t pair(float x, float y)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ void split(uint64_t v, float &x, float &y) { asm("mov.b64 {%0, %1}, %2;\n" : "=f"(x), "=f"(y) : "l"(v)); }
__device__ __forceinline__ uint64_t fma2(uint64_t x, uint64_t y, uint64_t z)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r) : "l"(x), "l"(y), "l"(z));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t x, uint64_t y)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(x), "l"(y));
    return r;
}
template <int D>
__global__ void __launch_bounds__(kThreads, 1)
chunk_attn_kernel(Args a, AttnPlan plan)
{
    using S = AttnSmem<D>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    Entry *ring = reinterpret_cast<Entry *>(sm + S::OFF_RING);
    Item *items = reinterpret_cast<Item *>(sm + S::OFF_ITEM);
    float2 *state = reinterpret_cast<float2 *>(sm + S::OFF_STATE);
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + S::OFF_BAR);
    uint64_t *ring_full = bars, *ring_empty = bars + kRing, *k_full = bars + 2 * kRing, *k_empty = k_full + kStages;
    uint64_t *v_full = k_empty + kStages, *v_empty = v_full + kStages, *q_full = v_empty + kStages;
    uint64_t *s_full = q_full + 2, *p_full = s_full + 2, *o_full = p_full + 2, *drained = o_full + 2;
    uint64_t *b_ready = drained + 1, *b_read = drained + 2, *turn = drained + 3;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drained + 5);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    volatile int *nan_item = reinterpret_cast<volatile int *>(tmem_slot + 2);     // by item: its number if a V code of it is NaN
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const PagedProblem &p = a.p;
    DeviceStatus *st = a.st;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kRing; ++i) {
            mbar_init(&ring_full[i], 1);
            mbar_init(&ring_empty[i], kSoftWarps + kCodeWarps + 2);
            nan_item[i] = -1;
        }
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&k_full[i], kCodeWarps);
            mbar_init(&k_empty[i], 2);
            mbar_init(&v_full[i], kCodeWarps);
            mbar_init(&v_empty[i], 2);
        }
        for (int h = 0; h < 2; ++h) {
            mbar_init(&q_full[h], 4);
            mbar_init(&s_full[h], 1);
            mbar_init(&p_full[h], 4);
            mbar_init(&o_full[h], 1);
            mbar_init(&turn[h], 1);
        }
        mbar_init(drained, 2);
        mbar_init(b_ready, 4);
        mbar_init(b_read, 4);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == kMma) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    chain_next();                 // behind the allocation: a successor that allocates too waits for this CTA to end
    const uint32_t tmem = *tmem_slot;
    chain_wait(a.q, a.k8, a.v8, a.k_scale, a.v_scale, a.block_table, a.row_pos, a.sel, a.o, a.lse);

    // the ring's next entry, for a consumer
    auto wait_entry = [&](int e) { return wait(&ring_full[e % kRing], (uint32_t)(e / kRing) & 1u, st, 181, abort_flag); };
    auto done_entry = [&](int e) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&ring_empty[e % kRing]);
    };

    if (warp == kPlanner) {
        const Pieces pieces(plan, a);
        const ChunkShare mine(pieces.total, gridDim.x, pieces.least(), blockIdx.x);
        int e = 0, seq = 0;
        bool ok = true;
        auto open = [&]() { return wait(&ring_empty[e % kRing], ((uint32_t)(e / kRing) & 1u) ^ 1u, st, 182, abort_flag); };
        auto push = [&](int kind) {        // an entry that is no page
            if (!(ok = open())) return;
            if (lane == 0) {
                ring[e % kRing].kind = kind;
                ring[e % kRing].item = seq;
                mbar_arrive(&ring_full[e % kRing]);
            }
            __syncwarp();
            ++e;
        };
        int item = mine.from < mine.to ? pieces.find(mine.from, lane) : 0;
        const float qk = p.scale * kLog2e;
        for (; ok && mine.from < mine.to && item < pieces.n_items; ++item) {
            const long long start = pieces.start(item);
            if (start >= mine.to) break;
            const int pages = pieces.pages(item), g = item % p.Hkv;
            const ChunkTile t = plan.tiles.tiles[item / p.Hkv];
            const int mt = tile_halves(t.rows * p.G);
            int c0, c1;
            cut(start, pages, mt, mine.from, mine.to, c0, c1);
            if (c0 >= c1) continue;
            const long long at = ((long long)t.row * p.Hkv + (long long)g * t.rows) * p.topk;
            if (!(ok = open())) break;
            if (lane == 0) {
                Item &i = items[seq % kRing];
                i.row = t.row;
                i.rows = t.rows;
                i.req = t.req;
                i.group = g;
                i.part = c0 == 0 && c1 == pages ? -1 : 2 * (int)blockIdx.x + (c0 == 0);
                i.split = mt == 1;
                i.c0 = c0;
                i.c1 = c1;
                i.base = 0;
                i.at = at;
            }
            __syncwarp();
            const int32_t *table = a.block_table + (long long)t.req * p.max_blocks;
            int turn = 0, base = 0;
            unsigned begun = 0;
            for (int c = c0; ok && c < c1; c += 32) {
                const int n = min(32, c1 - c);
                int block = 0, page = -1;
                uint32_t mask[kMaskWords];
                float ks = 0.f, vs = 0.f;
                if (lane < n) {
                    block = a.sel ? plan.blocks[at + c + lane] : c + lane;
                    for (int w = 0; w < kMaskWords; ++w) mask[w] = w < a.words && a.sel ? plan.masks[(at + c + lane) * a.words + w] : 0u;
                    page = table[block];
                    if ((unsigned)page < (unsigned)p.n_pages) {
                        ks = a.k_scale[(long long)page * p.Hkv + g];
                        vs = a.v_scale[(long long)page * p.Hkv + g];
                    } else {
                        report(st, kDevCheck, 173, page);
                        page = -1;
                    }
                }
                unsigned todo = __ballot_sync(0xffffffffu, page >= 0);
                // A piece none of whose pages is one gets a page that no row sees, so that every end follows a page of its item:
                // the warps that convert the codes look for the next page before they lay down a V, and the ends before it are
                // held until that V has been multiplied (eight in a row would fill the ring).
                if (!begun && !todo && c + 32 >= c1) {
                    if (lane == 0) {
                        page = 0;
                        block = kNoBlock;
                        vs = 1.f;
                        for (int w = 0; w < kMaskWords; ++w) mask[w] = 0;
                    }
                    todo = 1;
                }
                const int ev = (int)(__float_as_uint(vs) >> 23 & 255) - 127;
                if (!begun && todo) base = __shfl_sync(0xffffffffu, min(max(ev, -kBase), kBase), __ffs(todo) - 1);
                for (; ok && todo; todo &= todo - 1) {
                    const int j = __ffs(todo) - 1;
                    const int h = mt == 1 ? 1 + turn : 3;
                    turn ^= 1;
                    if (!(ok = open())) break;
                    if (lane == j) {
                        Entry &x = ring[e % kRing];
                        x.kind = kPageEntry;
                        x.item = seq;
                        x.page = page;
                        x.block = block;
                        x.halves = h;
                        x.first = h & ~begun;
                        x.a = qk * ks;
                        const int lv = min(max(ev - base, -kBelow), kAbove);
                        x.lv = (float)lv;
                        x.il = __uint_as_float((uint32_t)(127 - lv) << 23);
                        x.pv = vs * __uint_as_float((uint32_t)(127 - lv - base) << 23);
                        if (!begun) items[seq % kRing].base = base;      // read after the item's end, which this entry comes before
                        for (int w = 0; w < kMaskWords; ++w) x.mask[w] = mask[w];
                        mbar_arrive(&ring_full[e % kRing]);
                    }
                    __syncwarp();
                    begun |= h;
                    ++e;
                }
            }
            if (ok) push(kEndEntry);
            ++seq;
        }
        if (ok) push(kExit);
    } else if (warp >= kCode0 && warp < kMma) {
        // ------------------------------------------------ codes to bf16
        const Place<D> place(threadIdx.x - 32 * kCode0);
        uint4 k[D / 16], v[D / 16];
        int e = 0, n = 0;
        // the next page's codes' place and item; false at the end
        auto next = [&](long long &tile, int &item) {
            for (;; ++e) {
                if (!wait_entry(e)) return false;
                const Entry &x = ring[e % kRing];
                const int kind = x.kind;
                item = x.item;
                if (kind == kPageEntry) tile = ((long long)x.page * p.Hkv + items[item % kRing].group) * kPage * D;
                done_entry(e);
                if (kind == kPageEntry) break;
                if (kind == kExit) return false;
            }
            ++e;
            return true;
        };
        auto load = [&](uint4 (&u)[D / 16], const uint8_t *codes) {
#pragma unroll
            for (int j = 0; j < D / 16; ++j)
                u[j] = __ldg(reinterpret_cast<const uint4 *>(codes + (place.token + j * Place<D>::kStep) * D + place.feature));
        };
        long long tile = 0, tile2 = 0;
        int item = 0, item2 = 0;
        bool have = next(tile, item);
        if (have) load(k, a.k8 + tile);
        for (; have; ++n) {
            const int s = n % kStages;
            const uint32_t free = ((uint32_t)(n / kStages) & 1u) ^ 1u;
            load(v, a.v8 + tile);
            if (!wait(&k_empty[s], free, st, 183, abort_flag)) break;
            lay_down<D, false>(sm + S::OFF_K + s * S::TILE, k, place);
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(&k_full[s]);
            const bool more = next(tile2, item2);
            if (more) load(k, a.k8 + tile2);
            if (!wait(&v_empty[s], free, st, 184, abort_flag)) break;
            if (lay_down<D, true>(sm + S::OFF_V + s * S::TILE, v, place)) {
                mend<D>(sm + S::OFF_V + s * S::TILE, a.v8 + tile, place);
                nan_item[item % kRing] = item;
            }
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(&v_full[s]);
            have = more;
            tile = tile2;
            item = item2;
        }
    } else if (warp == kMma || warp == kMma + 1) {
        // ------------------------------------------------ MMA issuers, one for each half: a page's P V, then the next one's S
        constexpr uint32_t I_S = idesc_f16(128, kPage), I_O = idesc_bf16(128, D) | kBMajorMN;
        const int h = warp - kMma;
        const uint32_t tS = tmem + h * 128, tO = tmem + 256 + h * D;
        const uint64_t dQ = sdesc_k128(smem_u32(sm) + h * S::TILE), dK = sdesc_k128(smem_u32(sm + S::OFF_K));
        const uint64_t dV = sdesc_sw128(smem_u32(sm + S::OFF_V), kSub, 1024);
        uint32_t n = 0, ops = 0;
        int begun = -1;                        // the item whose queries are there
        int due = -1, left = -1;               // the page whose P V is due; the one whose V this half does not read
        bool due_first = false;
        bool ok = true;
        // the product due, once its P is there
        auto p_there = [&]() {
            return wait(&v_full[due % kStages], (uint32_t)(due / kStages) & 1u, st, 186, abort_flag) &&
                   wait(&p_full[h], ops++ & 1u, st, 185, abort_flag);
        };
        auto issue_o = [&]() {
            const uint64_t v = desc_adv(dV, due % kStages * S::TILE);
#pragma unroll
            for (int ks = 0; ks < kPage / 16; ++ks) mma_bf16_ts(tO, tS + ks * 8, desc_adv(v, ks * 2048), I_O, !due_first || ks > 0);
            mma_commit(&v_empty[due % kStages]);
        };
        for (int e = 0; ok; ++e) {
            if (!wait_entry(e)) break;
            const Entry &x = ring[e % kRing];
            const int kind = x.kind, item = x.item;
            const bool mine = kind == kPageEntry && (x.halves >> h & 1), first = x.first >> h & 1;
            done_entry(e);
            if (kind == kExit) break;
            const uint32_t s = n % kStages;
            // what this entry's products wait for
            if (kind == kPageEntry) {
                ok = wait(&k_full[s], n / kStages & 1u, st, 187, abort_flag);
                // (V of the page before was laid down before this K)
                if (left >= 0 && lane == 0) mbar_arrive(&v_empty[left % kStages]);
            } else if (left >= 0) {
                ok = wait(&v_full[left % kStages], (uint32_t)(left / kStages) & 1u, st, 186, abort_flag);
                if (ok && lane == 0) mbar_arrive(&v_empty[left % kStages]);
            }
            left = -1;
            if (!ok) break;
            if ((mine || kind == kEndEntry) && begun != item) {        // an item ends only after it has begun: never two ends ahead
                if (!(ok = wait(&q_full[h], (uint32_t)item & 1u, st, 188, abort_flag))) break;
                begun = item;
            }
            // its own next page, the end, or a page whose V waits for that one's place
            const bool o = due >= 0 && (mine || kind == kEndEntry || (int)n >= due + kStages);
            if (o && !(ok = p_there())) break;
            // the halves take turns
            if (!(ok = wait(&turn[h], ((uint32_t)e & 1u) ^ (h == 0), st, 193, abort_flag))) break;
            fence_after_sync();
            if (elect_one()) {
                if (o) issue_o();
                if (mine) {
                    const uint64_t k = desc_adv(dK, s * S::TILE);
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks) {
                        const uint32_t off = (ks >> 2) * kSub + (ks & 3) * 32;
                        mma_bf16(tS, desc_adv(dQ, off), desc_adv(k, off), I_S, ks > 0);
                    }
                    mma_commit(&s_full[h]);
                    mma_commit(&k_empty[s]);
                } else if (kind == kPageEntry) {
                    mbar_arrive(&k_empty[s]);
                } else {
                    mma_commit(&o_full[h]);
                }
                mbar_arrive(&turn[h ^ 1]);
            }
            __syncwarp();
            if (o) due = -1;
            if (mine) {
                due = (int)n;
                due_first = first;
            } else if (kind == kPageEntry) {
                left = (int)n;
            }
            n += kind == kPageEntry;
        }
        if (elect_one()) mma_commit(drained);
        __syncwarp();
        mbar_wait(drained, 0, nullptr, 0, nullptr);    // every product of both has ended
    } else if (warp < kSoftWarps) {
        // ------------------------------------------------ softmax: a (row, head) pair to a thread
        const int half = warp >> 2, r = (warp & 3) * 32 + lane;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + lanes + half * 128, tO = tmem + lanes + 256 + half * D;
        float m = -INFINITY, z = 0.f;          // reference (log2), sum
        float q_down = 1.f, q_sum = 0.f;       // the queries' factor, inverse; what their scores are bounded by
        int cur = -1, pos = -1, token = 0, ops = 0, splits = 0;
        bool used = false;

        auto begin = [&](int item) {
            cur = item;
            const Item &it = items[item % kRing];
            const int rho = it.split ? r : half * 128 + r, pairs = it.rows * p.G;
            token = rho >> a.shift;
            pos = rho < pairs ? a.row_pos[it.row + token] : -1;
            if ((long long)pos >= (long long)p.max_blocks * kPage) pos = -1;
            m = -INFINITY;
            z = 0.f;
            used = false;
            // this warp's 32 pairs of queries, as fp16: each times the power of two that brings its largest feature to 2^14 or above
            constexpr int CPR = D / 8, RPI = 32 / CPR, N = 32 / RPI;
            constexpr int ROUND = N < 8 ? N : 8;
            const int c = lane % CPR, first = (warp & 3) * 32 + lane / CPR;
            auto place = [&](int rr) { return reinterpret_cast<uint4 *>(sm + half * S::TILE + (c >> 3) * kSub + rr * 128 + (((c & 7) ^ (rr & 7)) << 4)); };
#pragma unroll 1
            for (int j0 = 0; j0 < N; j0 += ROUND) {
                uint4 u[ROUND];
#pragma unroll
                for (int j = 0; j < ROUND; ++j) {
                    const int rr = first + (j0 + j) * RPI, rh = it.split ? rr : half * 128 + rr;
                    u[j] = make_uint4(0, 0, 0, 0);
                    if (rh < pairs)
                        u[j] = __ldg(reinterpret_cast<const uint4 *>(a.q + ((long long)(it.row + (rh >> a.shift)) * p.Hq + it.group * p.G + (rh & (p.G - 1))) * D) + c);
                }
#pragma unroll
                for (int j = 0; j < ROUND; ++j) *place(first + (j0 + j) * RPI) = u[j];
            }
#pragma unroll 1
            for (int j = 0; j < N; ++j) {
                const int rr = first + j * RPI;
                const uint4 q = *place(rr);
                uint32_t w[4] = {q.x, q.y, q.z, q.w};
                float top = 0.f, sum = 0.f;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 f = unpack_bf16(w[k]);
                    top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
                    sum += fabsf(f.x) + fabsf(f.y);
                }
#pragma unroll
                for (int o = 1; o < CPR; o <<= 1) {
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                    sum += __shfl_xor_sync(0xffffffffu, sum, o);
                }
                const int ex = top > 0.f ? min(14 - ((int)(__float_as_uint(top) >> 23) - 127), 126) : 0;   // 126 falls short below 2^-112
                const float up = __uint_as_float((uint32_t)(127 + ex) << 23), down = __uint_as_float((uint32_t)(127 - ex) << 23);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 f = unpack_bf16(w[k]);
                    const __half2 h = __floats2half2_rn(f.x * up, f.y * up);
                    w[k] = *reinterpret_cast<const uint32_t *>(&h);
                }
                *place(rr) = make_uint4(w[0], w[1], w[2], w[3]);
                // 452: the largest code, 448, and what the sum's roundings could lack
                const float of_row = __shfl_sync(0xffffffffu, down, (lane % RPI) * CPR), its_sum = __shfl_sync(0xffffffffu, sum * up * 452.f, (lane % RPI) * CPR);
                if (lane / RPI == j) {
                    q_down = of_row;
                    q_sum = its_sum;
                }
            }
            fence_proxy_async();
            fence_before_sync();                              // the item before has read its sums
            __syncwarp();
            if (lane == 0) mbar_arrive(&q_full[half]);
        };

        // Scores to probabilities, in their place.
        auto page = [&](int lim, bool first, float fa, float lv, float il, float pv) {
            if (!wait(&s_full[half], (uint32_t)ops++ & 1u, st, 189, abort_flag)) return false;
            fence_after_sync();
            used = true;
            if (!__any_sync(0xffffffffu, lim >= 0)) {
                const uint32_t none[16] = {};
#pragma unroll 1
                for (int c = 0; c < 64; c += 16) tmem_st16(tS + c, none);
            } else {
                uint32_t x[32], y[32];
                // rows that see nothing of the page: their probabilities are put to 0
                const bool mixed = !__all_sync(0xffffffffu, lim >= 0);
                const uint32_t seen = lim >= 0 ? ~0u : 0u;
                // rows that see a part of it: masked scores are minus infinity from here on
                if (__builtin_expect(__any_sync(0xffffffffu, lim >= 0 && lim < kPage - 1), 0)) {
#pragma unroll 1
                    for (int c = 0; c < kPage; c += 32) {
                        tmem_ld32_nowait(tS + c, x);
                        tmem_wait32(x);
#pragma unroll
                        for (int j = 0; j < 32; ++j) x[j] = c + j <= lim ? x[j] : 0xFF800000u;
                        tmem_st16(tS + c, x);
                        tmem_st16(tS + c + 16, x + 16);
                    }
                    tmem_wait_st();
                }
                // the largest score is looked for where one could lie too far above the reference
                const bool far = (!(q_sum * fa + lv <= m + kFar) || pv > 1.f) && lim >= 0;
                if (__any_sync(0xffffffffu, far)) {
                    float top = -INFINITY;
#pragma unroll 1
                    for (int c = 0; c < kPage; c += 64) {
                        tmem_ld32_nowait(tS + c, x);
                        tmem_ld32_nowait(tS + c + 32, y);
                        tmem_wait32(x);
                        tmem_wait32(y);
#pragma unroll
                        for (int j = 0; j < 32; ++j) top = fmaxf(top, fmaxf(__uint_as_float(x[j]), __uint_as_float(y[j])));
                    }
                    const float t = top * fa + lv;
                    const bool up = far && t > m + kLag;
                    if (__any_sync(0xffffffffu, up)) {
                        const float keep = up ? ex2(m - t) : 1.f;
                        if (!first && __any_sync(0xffffffffu, up && m != -INFINITY)) {      // (rows that see their first page have no sums)
#pragma unroll 1
                            for (int c = 0; c < D; c += 16) {
                                uint32_t o[16];
                                tmem_ld16_nowait(tO + c, o);
                                tmem_wait16(o);
#pragma unroll
                                for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * keep);
                                tmem_st16(tO + c, o);
                            }
                        }
                        z *= keep;
                        m = up ? t : m;
                    }
                }
                tmem_ld32_nowait(tS, x);
                const float c0 = m == -INFINITY ? lv : lv - m;
                const uint64_t fa2 = pair(fa, fa), c02 = pair(c0, c0);
                uint64_t zp[2] = {0, 0};
                auto powers = [&](const uint32_t (&v)[32], int c) {
                    uint32_t pk[16];
#pragma unroll
                    for (int j = 0; j < 32; j += 2) {
                        float e0, e1;
                        split(fma2(pair(__uint_as_float(v[j]), __uint_as_float(v[j + 1])), fa2, c02), e0, e1);
                        e0 = ex2(e0);
                        e1 = ex2(e1);
                        zp[j >> 1 & 1] = add2(zp[j >> 1 & 1], pair(e0, e1));
                        pk[j / 2] = pack_bf16(e0, e1);
                    }
                    if (__builtin_expect(pv != 1.f, 0)) {               // exact: a power of two
                        const __nv_bfloat162 pv2 = __float2bfloat162_rn(pv);
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const __nv_bfloat162 q = __hmul2(*reinterpret_cast<__nv_bfloat162 *>(&pk[j]), pv2);
                            pk[j] = *reinterpret_cast<const uint32_t *>(&q);
                        }
                    }
                    if (mixed) {
#pragma unroll
                        for (int j = 0; j < 16; ++j) pk[j] &= seen;
                    }
                    tmem_st16(tS + c / 2, pk);
                };
#pragma unroll 1
                for (int c = 0; c < kPage; c += 64) {
                    tmem_wait32(x);
                    tmem_ld32_nowait(tS + c + 32, y);
                    powers(x, c);                  // P takes the columns from half of the scores' on: behind what was read
                    tmem_wait32(y);
                    if (c + 64 < kPage) tmem_ld32_nowait(tS + c + 64, x);
                    powers(y, c + 32);
                }
                float z0, z1;
                split(add2(zp[0], zp[1]), z0, z1);
                if (seen) z += (z0 + z1) * il;
            }
            tmem_wait_st();
            fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[half]);
            return true;
        };

        auto finish = [&](int item) {
            const Item &it = items[item % kRing];
            if (!wait(&o_full[half], (uint32_t)item & 1u, st, 190, abort_flag)) return false;
            fence_after_sync();
            const int rho = it.split ? r : half * 128 + r;
            const bool mine = rho < it.rows * p.G && pos >= 0;
            float wa = used ? 1.f : 0.f, wb = 0.f;
            if (it.split) {
                const uint32_t turn = splits++ & 1u;
                if (half == 1) {
                    state[r] = make_float2(used ? m : -INFINITY, used ? z : 0.f);
                    fence_before_sync();                      // A reads the sums that this half's products left
                    __syncwarp();
                    if (lane == 0) mbar_arrive(b_ready);
                    return wait(b_read, turn, st, 191, abort_flag);   // A has read this half's sums
                }
                if (!wait(b_ready, turn, st, 192, abort_flag)) return false;
                fence_after_sync();
                const float2 b = state[r];
                const bool none = b.y == 0.f;                 // nothing visible on B's pages
                const float top = none ? m : fmaxf(m, b.x);
                wa = !used || z == 0.f ? 0.f : m == top ? 1.f : ex2(m - top);
                wb = none ? 0.f : b.x == top ? 1.f : ex2(b.x - top);
                z = (wa == 0.f ? 0.f : z * wa) + (wb == 0.f ? 0.f : b.y * wb);
                m = top;
            }
            const bool any_a = __any_sync(0xffffffffu, wa != 0.f), any_b = __any_sync(0xffffffffu, wb != 0.f);
            // z = f 2^k, f below 1.  A whole tile's outputs are O 2^base / z.  A piece's state is (m + k, f) and O 2^(base - k), no
            // larger than outputs, so that pieces in different bases join.  2^(base - k) in two steps: what is between them is no larger
            // than the larger end.  (A sum that is NaN stays in f.)
            const int ez = (int)(__float_as_uint(z) >> 23 & 255), k = ez == 0 || ez == 255 ? 0 : min(ez - 126, 126);
            const float f = z * __uint_as_float((uint32_t)(127 - k) << 23);
            const int by = it.base - k, half_by = by >> 1;
            const float by0 = z == 0.f ? 0.f : __uint_as_float((uint32_t)(127 + half_by) << 23);
            const float by1 = __uint_as_float((uint32_t)(127 + by - half_by) << 23), inv = it.part >= 0 || z == 0.f ? by1 : by1 / f;
            const long long row = (long long)(it.row + token) * p.Hq + it.group * p.G + (rho & (p.G - 1));
            float *part = it.part >= 0 ? plan.part + ((long long)it.part * kTileRows + rho) * D : nullptr;
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
                float x[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) x[j] = 0.f;
                uint32_t o[16];
                if (any_a) {
                    tmem_ld16_nowait(tO + c, o);
                    tmem_wait16(o);
#pragma unroll
                    for (int j = 0; j < 16; ++j) x[j] = wa == 0.f ? 0.f : __uint_as_float(o[j]) * wa;
                }
                if (any_b) {
                    tmem_ld16_nowait(tO + D + c, o);
                    tmem_wait16(o);
#pragma unroll
                    for (int j = 0; j < 16; ++j) x[j] += wb == 0.f ? 0.f : __uint_as_float(o[j]) * wb;
                }
#pragma unroll
                for (int j = 0; j < 16; ++j) x[j] = x[j] * by0 * inv;
                if (mine && part) {
#pragma unroll
                    for (int j = 0; j < 16; j += 4) *reinterpret_cast<float4 *>(part + c + j) = make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]);
                } else if (mine) {
#pragma unroll
                    for (int j = 0; j < 16; j += 8)
                        *reinterpret_cast<uint4 *>(a.o + row * D + c + j) =
                            make_uint4(pack_bf16(x[j], x[j + 1]), pack_bf16(x[j + 2], x[j + 3]), pack_bf16(x[j + 4], x[j + 5]), pack_bf16(x[j + 6], x[j + 7]));
                }
                __syncwarp();
            }
            if (mine) {
                if (part) plan.stats(a.ctas, D)[(long long)it.part * kTileRows + rho] = make_float2(z == 0.f ? -INFINITY : m + (float)k, f);
                else a.lse[row] = z == 0.f ? -INFINITY : (m + (float)k + log2f(f)) * kLn2;
                if (nan_item[item % kRing] == item) spoil<D>(a, plan, it, pos, token, part, a.o + row * D);
            }
            __syncwarp();
            if (it.split) {
                fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(b_read);
            }
            return true;
        };

        for (int e = 0;; ++e) {
            if (!wait_entry(e)) break;
            const Entry &x = ring[e % kRing];
            const int kind = x.kind, item = x.item;
            if (kind == kExit) break;
            if (item != cur) begin(item);
            if (kind == kPageEntry && (x.halves >> half & 1)) {
                const bool seen = !a.sel || x.mask[token >> 5] >> (token & 31) & 1;
                const int lim = seen ? min(pos - x.block * kPage, kPage - 1) : -1;
                const bool first = x.first >> half & 1;
                float fa = x.a * q_down;
                if (fa == 0.f) fa = 0x1p-126f;                    // so that masked scores stay minus infinity
                const float lv = x.lv, il = x.il, pv = x.pv;
                done_entry(e);
                if (!page(lim, first, fa, lv, il, pv)) break;
            } else {
                if (kind == kEndEntry && !finish(item)) break;
                done_entry(e);                     // not before: the item's place may be taken once its end is let go
            }
        }
    }
    fence_before_sync();
    __syncthreads();
    if (warp == kMma) {
        fence_after_sync();
        tmem_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------- cut tiles
// CTAs of 64 pairs for each stretch: those of the item that ends in it and was begun before.  A warp takes eight, whose
// states it loads at once: finding the item is a chain of loads as long as the rest (a pair to a warp: 35 us instead of
// 21 for the tiles of 256 that 152 stretches cut).
constexpr int kJoin = 8;
template <int D>
__global__ void __launch_bounds__(256) chunk_join_kernel(Args a, AttnPlan plan)
{
    chain_next();
    chain_wait(a.row_pos, a.sel, a.o, a.lse);
    const PagedProblem &p = a.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, cta = blockIdx.x;
    const Pieces pieces(plan, a);
    const ChunkShare mine(pieces.total, a.ctas, pieces.least(), cta);
    if (mine.from >= mine.to) return;
    const int item = pieces.find(mine.from, lane);
    const long long start = pieces.start(item);
    if (start >= mine.from) return;
    const ChunkTile t = plan.tiles.tiles[item / p.Hkv];
    const int pages = pieces.pages(item), mt = tile_halves(t.rows * p.G), g = item % p.Hkv;
    int c0, c1;
    cut(start, pages, mt, mine.from, mine.to, c0, c1);
    if (c0 == 0 || c0 >= c1 || c1 != pages) return;
    const int rho0 = (blockIdx.y * 8 + warp) * kJoin, pairs = t.rows * p.G;
    if (rho0 >= pairs) return;
    const float2 *stats = plan.stats(a.ctas, D);
    const bool has = lane * 4 < D;
    float m[kJoin], z[kJoin], x[kJoin][4];
#pragma unroll
    for (int i = 0; i < kJoin; ++i) {
        m[i] = -INFINITY;
        z[i] = x[i][0] = x[i][1] = x[i][2] = x[i][3] = 0.f;
    }
    for (int k = (int)(start / mine.share); k <= cta; ++k) {
        int b0, b1;
        cut(start, pages, mt, mine.share * k, min(pieces.total, mine.share * (k + 1)), b0, b1);
        if (b0 >= b1) continue;
        const long long s = ((long long)2 * k + (b0 == 0)) * kTileRows + rho0;      // (a slot has 256 pairs, whatever the tile's)
        float2 b[kJoin];
        float4 y[kJoin];
#pragma unroll
        for (int i = 0; i < kJoin; ++i) {
            b[i] = stats[s + i];
            y[i] = has ? *reinterpret_cast<const float4 *>(plan.part + (s + i) * D + lane * 4) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int i = 0; i < kJoin; ++i) {
            if (b[i].y == 0.f) continue;                       // none of its pages visible
            // (2^-10: sums of values near the largest that there are stay finite)
            const float top = fmaxf(m[i], b[i].x), wa = m[i] == top ? 1.f : ex2(m[i] - top), wb = (b[i].x == top ? 1.f : ex2(b[i].x - top)) * 0x1p-10f;
            z[i] = z[i] * wa + b[i].y * wb;
            x[i][0] = x[i][0] * wa + y[i].x * wb;
            x[i][1] = x[i][1] * wa + y[i].y * wb;
            x[i][2] = x[i][2] * wa + y[i].z * wb;
            x[i][3] = x[i][3] * wa + y[i].w * wb;
            m[i] = top;
        }
    }
#pragma unroll
    for (int i = 0; i < kJoin; ++i) {
        const int rho = rho0 + i;
        const int pos = rho < pairs ? a.row_pos[t.row + rho / p.G] : -1;
        if (pos < 0 || (long long)pos >= (long long)p.max_blocks * kPage) continue;
        const long long row = (long long)(t.row + rho / p.G) * p.Hq + g * p.G + rho % p.G;
        const float inv = z[i] == 0.f ? 0.f : 1.f / z[i];
        if (has)
            *reinterpret_cast<uint2 *>(a.o + row * D + lane * 4) =
                make_uint2(pack_bf16(x[i][0] * inv, x[i][1] * inv), pack_bf16(x[i][2] * inv, x[i][3] * inv));
        if (lane == 0) a.lse[row] = z[i] == 0.f ? -INFINITY : (m[i] + log2f(z[i] * 0x1p10f)) * kLn2;
    }
}

// Rows of a tile: 256 pairs, or 128 with a selection.  Fewer rows have fewer blocks in their union, and the two halves
// take them in turn, where the halves of 256 pairs would wait for each other at blocks that only one of them has.
int attn_tokens(const PagedProblem &p, bool listed) { return (listed ? kTileRows / 2 : kTileRows) / p.G; }
int mask_words(const PagedProblem &p) { return std::max(1, attn_tokens(p, true) / 32); }
AttnPlan attn_plan(const PagedProblem &p, void *scratch, bool listed)
{
    const long long most = chunk_tiles(p, attn_tokens(p, listed));
    return AttnPlan(scratch, most, p, ChunkPlan::bytes(most), listed, mask_words(p), p.num_sms);
}

}  // namespace

size_t paged_chunk_scratch_bytes(const PagedProblem &p, bool attention)
{
    return attention ? std::max(attn_plan(p, nullptr, true).bytes, attn_plan(p, nullptr, false).bytes) : paged_chunk_scores_scratch(p);
}

cudaError_t launch_paged_chunk_attn(const PagedProblem &p, const bf16 *q, const uint8_t *k8, const uint8_t *v8, const float *k_scale,
                                    const float *v_scale, const int32_t *block_table, const int32_t *q_starts, const int32_t *row_pos,
                                    const int32_t *sel, bf16 *o, float *lse, void *scratch, DeviceStatus *st, cudaStream_t s)
{
    const int tokens = attn_tokens(p, sel != nullptr);
    cudaError_t e = launch_chunk_plan(p, q_starts, row_pos, tokens, p.G, scratch, st, s);
    if (e != cudaSuccess) return e;
    const AttnPlan plan = attn_plan(p, scratch, sel != nullptr);
    const Args a{p, q, k8, v8, k_scale, v_scale, block_table, row_pos, sel, o, lse, tokens, mask_words(p), p.num_sms, p.G == 8 ? 3 : p.G / 2, st};
    if (sel) {
        const long long items = chunk_tiles(p, tokens) * p.Hkv, ctas = std::min((items + kListWarps - 1) / kListWarps, 8LL * p.num_sms);
        if ((e = launch_chained("paged_chunk_list_kernel", chunk_list_kernel, dim3((unsigned)ctas), 32 * kListWarps, 0, s, a, plan)) != cudaSuccess) return e;
        if ((e = launch_chained("paged_chunk_sum_kernel", chunk_sum_kernel, dim3(1), 1024, 0, s, a, plan)) != cudaSuccess) return e;
    }
    auto run = [&](auto dtag) {
        constexpr int D = decltype(dtag)::value;
        static std::atomic<unsigned long long> allowed{0};
        if ((e = allow_smem(chunk_attn_kernel<D>, AttnSmem<D>::ALLOC, allowed)) != cudaSuccess) return e;
        e = launch_chained("paged_chunk_attn_kernel", chunk_attn_kernel<D>, dim3(p.num_sms), kThreads, AttnSmem<D>::ALLOC, s, a, plan);
        if (e != cudaSuccess) return e;
        return launch_chained("paged_chunk_join_kernel", chunk_join_kernel<D>, dim3(p.num_sms, (sel ? kTileRows / 2 : kTileRows) / (8 * kJoin)), 256, 0, s, a, plan);
    };
    return p.d == 128 ? run(std::integral_constant<int, 128>{}) : run(std::integral_constant<int, 64>{});
}

}  // namespace msa
