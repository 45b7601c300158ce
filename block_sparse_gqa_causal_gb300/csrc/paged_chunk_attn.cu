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
// half's scores become probabilities.
//
// Codes to bf16.  e4m3 products would need queries and probabilities as pairs
// of e4m3 terms, and small probabilities as several levels of those; as bf16
// everything is exact but the probabilities' own 8 bits, at any size.  An
// e4m3 value is a bf16 with its exponent moved: the code's bits shifted into
// place, times 2^120, exact for subnormal codes too.  Four warps do that once a
// page for both halves (one value converted to a probability computed); they
// keep the order 0, 2, 1, 3 of each four features, in which two pairs of bytes
// come out of a word without being sorted.  The queries are laid down in that
// order, and O's columns are put right when they are written.
//
// Softmax.  With t_j = l_j log2 e + log2 vs, the weight of token j's codes is
// 2^t_j and that of the sum 2^t_j / vs, so one reference m per row bounds both
// and P V adds up in TMEM across pages of different scales.  m is the largest t
// so far, or up to kLag less: only then are the sums rescaled.  P (bf16) takes
// the place of its scores in TMEM and is read from there as the A operand.
//
// A NaN code must not reach rows that do not see its token, and 0 x NaN does:
// NaNs of V enter the products as 0, and rows that see one (looked for only
// then) get theirs when they are written.
//
// With a selection, a tile walks the union of its rows' blocks (made by a kernel
// before, with a bit to each row that selected the block); a half without any
// such row is passed over.
// The work is one list of products, those of (tile 0, group 0), (tile 0, group 1)
// and so on, cut into equal stretches for persistent CTAs.  A stretch cuts at
// most two tiles; those pieces' states go to the workspace, and a kernel after
// joins them, in the order of their pages.  A tile of up to 128 pairs has only half
// A: its pages go to the two halves in turn, both with the same queries, and A joins them.
//   warps 0..3, 4..7   softmax of half A, B, a pair to a thread
//   warps 8..11        codes of K and V to bf16 tiles in shared memory, loaded a tile ahead
//   warp 12            tcgen05.mma issuer
//   warp 13            planner: pages, scales and masks, through a ring
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
constexpr int kCode0 = kSoftWarps, kMma = kCode0 + kCodeWarps, kPlanner = kMma + 1;
constexpr int kThreads = 32 * (kPlanner + 1);
constexpr int kStages = 2;                    // K and V tiles
constexpr int kRing = 8;                      // pages the planner is ahead
constexpr int kSub = 128 * 128;               // [128 rows][64 bf16], swizzled
constexpr int kLeast = 4;                     // products to a stretch at least
constexpr float kLag = 8.f;                   // log2 of what a probability may outgrow its reference by
constexpr int kMaskWords = kTileRows / 32;    // a bit to each row of a tile (at most 256, with G = 1)
constexpr int kWindow = 1 << 15;              // blocks whose union is taken in one go
constexpr int kListWarps = 4;

enum Kind { kPageEntry = 0, kEndEntry = 1, kExit = 2 };

struct Entry {                 // a page of the ring
    int kind, item, page, block;
    int halves, first;         // bits of the halves that take it; of those whose first page it is
    float a, lv, il, pv;       // logits' factor, log2 of the V scale (-100 at least), 2^-lv, what lv leaves of the scale (1)
    uint32_t mask[kMaskWords];
};
struct Item {                  // a tile's piece
    int row, rows, req, group, part;    // part: the piece's place among the partial states; -1: a whole tile
    int split;                 // one half's pairs, pages in turn
    int c0, c1;
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
    for (int i = 0; i < p.topk; ++i) {
        const int c = s[i];
        if (c == -1) continue;
        if (i >= entries || c <= prev || c > c_last) {
            fine = false;
            continue;
        }
        prev = c;
        fn(c);
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
    long long n_items, total;
    __device__ Pieces(const AttnPlan &pl, const Args &ar) : plan(pl), a(ar)
    {
        const int n = *pl.tiles.n_tiles;
        n_items = (long long)n * ar.p.Hkv;
        total = ar.sel ? pl.before[n_items] : pl.tiles.before[n] * ar.p.Hkv;
    }
    // the item that unit w is in, by a whole warp
    __device__ long long find(long long w, int lane) const
    {
        if (a.sel) return chunk_find(plan.before, (int)n_items, 1, w, lane);
        const int i = chunk_find(plan.tiles.before, *plan.tiles.n_tiles, a.p.Hkv, w, lane);
        const long long in = w - plan.tiles.before[i] * a.p.Hkv, one = plan.tiles.before[i + 1] - plan.tiles.before[i];
        return (long long)i * a.p.Hkv + in / one;
    }
    __device__ long long start(long long item) const
    {
        if (a.sel) return plan.before[item];
        const long long i = item / a.p.Hkv, one = plan.tiles.before[i + 1] - plan.tiles.before[i];
        return plan.tiles.before[i] * a.p.Hkv + one * (item % a.p.Hkv);
    }
    __device__ int pages(long long item) const { return a.sel ? plan.pages[item] : plan.tiles.tiles[item / a.p.Hkv].pages; }
};

// Pages [c0, c1) of an item of `pages` pages from unit `start` on that are [from, to)'s, a page where its first unit is.
__device__ __forceinline__ void cut(long long start, int pages, int mt, long long from, long long to, int &c0, int &c1)
{
    const long long off = max(0ll, from - start), stop = min((long long)pages * mt, to - start);
    c0 = (int)((off + mt - 1) / mt);
    c1 = stop > 0 ? (int)((stop + mt - 1) / mt) : 0;
}

// ---------------------------------------------------------------- the kernel
// Four e4m3 codes to bf16: features 0 and 2, then 1 and 3.
__device__ __forceinline__ uint2 widen(uint32_t w)
{
    const __nv_bfloat162 up = __halves2bfloat162(__ushort_as_bfloat16(0x7B80), __ushort_as_bfloat16(0x7B80));   // 2^120
    uint32_t even = ((w << 4) & 0x07F007F0u) | ((w << 8) & 0x80008000u), odd = ((w >> 4) & 0x07F007F0u) | (w & 0x80008000u);
    const __nv_bfloat162 e = __hmul2(*reinterpret_cast<__nv_bfloat162 *>(&even), up), o = __hmul2(*reinterpret_cast<__nv_bfloat162 *>(&odd), up);
    return make_uint2(*reinterpret_cast<const uint32_t *>(&e), *reinterpret_cast<const uint32_t *>(&o));
}
// The codes among four that are NaN (0x7F, 0xFF), bit 7 of each byte.
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }

// Writes the tile of 128 tokens that this thread's words `u` are part of.  NaNs stay (K) or become 0 and are told (V).
template <int D, bool V>
__device__ __forceinline__ bool lay_down(uint8_t *tile, const uint4 (&u)[D / 16], int tid)
{
    constexpr int CPR = D / 16;           // 16-code words of a token
    bool nan = false;
#pragma unroll
    for (int j = 0; j < D / 16; ++j) {
        const int i = tid + 128 * j, r = i / CPR, c = i % CPR;
        uint32_t w[4] = {u[j].x, u[j].y, u[j].z, u[j].w};
        uint32_t x[8];
        const uint32_t bad = nan_codes(w[0]) | nan_codes(w[1]) | nan_codes(w[2]) | nan_codes(w[3]);
        if (V && bad) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t b = nan_codes(w[k]);
                w[k] &= ~(b | (b - (b >> 7)));
            }
            nan = true;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint2 v = widen(w[k]);
            x[2 * k] = v.x;
            x[2 * k + 1] = v.y;
            if (!V && bad) {
                const uint32_t b = nan_codes(w[k]);
                if (b & 0x80u) x[2 * k] |= 0x00007FC0u;
                if (b & 0x800000u) x[2 * k] |= 0x7FC00000u;
                if (b & 0x8000u) x[2 * k + 1] |= 0x00007FC0u;
                if (b & 0x80000000u) x[2 * k + 1] |= 0x7FC00000u;
            }
        }
        // the 32 bytes' two halves in an order that keeps eight lanes on different banks
        uint8_t *row = tile + (c >> 2) * kSub + r * 128;
        const int at = 2 * (c & 3), turn = (c >> 2) & 1;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int k = h ^ turn;
            const uint4 y = k ? make_uint4(x[4], x[5], x[6], x[7]) : make_uint4(x[0], x[1], x[2], x[3]);
            *reinterpret_cast<uint4 *>(row + (((at + k) ^ (r & 7)) << 4)) = y;
        }
    }
    return nan;
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
    uint64_t *b_ready = drained + 1, *b_read = drained + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drained + 3);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    volatile int *nan_item = reinterpret_cast<volatile int *>(tmem_slot + 2);     // by item: its number if a V code of it is NaN
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const PagedProblem &p = a.p;
    DeviceStatus *st = a.st;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kRing; ++i) {
            mbar_init(&ring_full[i], 1);
            mbar_init(&ring_empty[i], kSoftWarps + kCodeWarps + 1);
            nan_item[i] = -1;
        }
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&k_full[i], kCodeWarps);
            mbar_init(&k_empty[i], 1);
            mbar_init(&v_full[i], kCodeWarps);
            mbar_init(&v_empty[i], 1);
        }
        for (int h = 0; h < 2; ++h) {
            mbar_init(&q_full[h], 4);
            mbar_init(&s_full[h], 1);
            mbar_init(&p_full[h], 4);
            mbar_init(&o_full[h], 1);
        }
        mbar_init(drained, 1);
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
    auto wait_entry = [&](int e) { return mbar_wait_warp(&ring_full[e % kRing], (uint32_t)(e / kRing) & 1u, st, 181, abort_flag); };
    auto done_entry = [&](int e) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&ring_empty[e % kRing]);
    };

    if (warp == kPlanner) {
        const Pieces pieces(plan, a);
        const ChunkShare mine(pieces.total, gridDim.x, kLeast, blockIdx.x);
        int e = 0, seq = 0;
        bool ok = true;
        auto open = [&]() { return mbar_wait_warp(&ring_empty[e % kRing], ((uint32_t)(e / kRing) & 1u) ^ 1u, st, 182, abort_flag); };
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
        long long item = mine.from < mine.to ? pieces.find(mine.from, lane) : 0;
        const float qk = p.scale * kLog2e;
        for (; ok && mine.from < mine.to && item < pieces.n_items; ++item) {
            const long long start = pieces.start(item);
            if (start >= mine.to) break;
            const int pages = pieces.pages(item), g = (int)(item % p.Hkv);
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
                i.at = at;
            }
            __syncwarp();
            const int32_t *table = a.block_table + (long long)t.req * p.max_blocks;
            int turn = 0;
            unsigned begun = 0;
            for (int c = c0; ok && c < c1; c += 32) {
                const int n = min(32, c1 - c);
                int block = 0, page = -1;
                uint32_t mask[kMaskWords];
                float ks = 0.f, vs = 0.f;
                if (lane < n) {
                    block = a.sel ? plan.blocks[at + c + lane] : c + lane;
                    for (int w = 0; w < kMaskWords; ++w) mask[w] = a.sel ? w < a.words ? plan.masks[(at + c + lane) * a.words + w] : 0u : ~0u;
                    page = table[block];
                    if ((unsigned)page < (unsigned)p.n_pages) {
                        ks = a.k_scale[(long long)page * p.Hkv + g];
                        vs = a.v_scale[(long long)page * p.Hkv + g];
                    } else {
                        report(st, kDevCheck, 173, page);
                        page = -1;
                    }
                }
                // half A's rows are those of the first 128 / G tokens
                int halves = 3;
                if (a.sel && mt == 2 && lane < n) {
                    const int half = kTileRows / 2 / p.G;
                    uint32_t lo = 0, hi = 0;
                    if (half >= 32) {
                        for (int w = 0; w < kMaskWords; ++w) (w < half / 32 ? lo : hi) |= mask[w];
                    } else {
                        lo = mask[0] & ((1u << half) - 1);
                        hi = mask[0] >> half;
                    }
                    halves = (lo ? 1 : 0) | (hi || !lo ? 2 : 0);
                }
                unsigned todo = __ballot_sync(0xffffffffu, page >= 0);
                for (; ok && todo; todo &= todo - 1) {
                    const int j = __ffs(todo) - 1;
                    int h = __shfl_sync(0xffffffffu, halves, j);
                    if (mt == 1) {
                        h = 1 + turn;
                        turn ^= 1;
                    }
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
                        const int ex = max((int)(__float_as_uint(vs) >> 23 & 255) - 127, -100);
                        x.lv = (float)ex;
                        x.il = ldexpf(1.f, -ex);
                        x.pv = ldexpf(vs, -ex);
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
        const int tid = threadIdx.x - 32 * kCode0;
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
            for (int j = 0; j < D / 16; ++j) u[j] = __ldg(reinterpret_cast<const uint4 *>(codes) + tid + 128 * j);
        };
        long long tile = 0, tile2 = 0;
        int item = 0, item2 = 0;
        bool have = next(tile, item);
        if (have) load(k, a.k8 + tile);
        for (; have; ++n) {
            const int s = n % kStages;
            const uint32_t free = ((uint32_t)(n / kStages) & 1u) ^ 1u;
            load(v, a.v8 + tile);
            if (!mbar_wait_warp(&k_empty[s], free, st, 183, abort_flag)) break;
            lay_down<D, false>(sm + S::OFF_K + s * S::TILE, k, tid);
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(&k_full[s]);
            const bool more = next(tile2, item2);
            if (more) load(k, a.k8 + tile2);
            if (!mbar_wait_warp(&v_empty[s], free, st, 184, abort_flag)) break;
            if (lay_down<D, true>(sm + S::OFF_V + s * S::TILE, v, tid)) nan_item[item % kRing] = item;
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(&v_full[s]);
            have = more;
            tile = tile2;
            item = item2;
        }
    } else if (warp == kMma) {
        // ------------------------------------------------ MMA issuer: a half's scores, then the half before's P V
        constexpr uint32_t I_S = idesc_bf16(128, kPage), I_O = idesc_bf16(128, D) | kBMajorMN;
        const uint64_t dQ = sdesc_k128(smem_u32(sm)), dK = sdesc_k128(smem_u32(sm + S::OFF_K));
        const uint64_t dV = sdesc_sw128(smem_u32(sm + S::OFF_V), kSub, 1024);
        int n = 0, e = 0;
        uint32_t done[2] = {0, 0};             // products with P of each half
        struct {
            int half, page;
            bool first, last;                  // of the half's pages; half of the page
        } due{-1, 0, false, false};
        bool ok = true;
        auto issue_o = [&]() {
            const int h = due.half, s = due.page % kStages;
            due.half = -1;
            ok = mbar_wait_warp(&p_full[h], done[h]++ & 1u, st, 185, abort_flag) &&
                 mbar_wait_warp(&v_full[s], (uint32_t)(due.page / kStages) & 1u, st, 186, abort_flag);
            if (!ok) return;
            fence_after_sync();
            if (elect_one()) {
#pragma unroll
                for (int ks = 0; ks < kPage / 16; ++ks)
                    mma_bf16_ts(tmem + 256 + h * D, tmem + h * 128 + ks * 8, desc_adv(dV, s * S::TILE + ks * 2048), I_O, !due.first || ks > 0);
                if (due.last) mma_commit(&v_empty[s]);
            }
            __syncwarp();
        };
        while (ok) {
            if (!(ok = wait_entry(e))) break;
            const Entry &x = ring[e % kRing];
            const int kind = x.kind, item = x.item, halves = x.halves, first = x.first;
            done_entry(e);
            ++e;
            if (kind == kExit) break;
            if (kind == kEndEntry) {
                if (due.half >= 0) issue_o();
                if (!ok) break;
                if (elect_one()) {
                    mma_commit(&o_full[0]);
                    mma_commit(&o_full[1]);
                }
                __syncwarp();
                continue;
            }
            const int s = n % kStages;
            if (!(ok = mbar_wait_warp(&k_full[s], (uint32_t)(n / kStages) & 1u, st, 187, abort_flag))) break;
            for (int h = 0; ok && h < 2; ++h) {
                if (!(halves >> h & 1)) continue;
                if (first >> h & 1 && !(ok = mbar_wait_warp(&q_full[h], (uint32_t)item & 1u, st, 188, abort_flag))) break;
                if (due.half == h) issue_o();          // its P is where the scores go
                if (!ok) break;
                fence_after_sync();
                if (elect_one()) {
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks) {
                        const uint32_t off = (ks >> 2) * kSub + (ks & 3) * 32;
                        mma_bf16(tmem + h * 128, desc_adv(dQ, h * S::TILE + off), desc_adv(dK, s * S::TILE + off), I_S, ks > 0);
                    }
                    mma_commit(&s_full[h]);
                    if (halves >> (h + 1) == 0) mma_commit(&k_empty[s]);
                }
                __syncwarp();
                if (due.half >= 0) issue_o();
                due = {h, n, (first >> h & 1) != 0, halves >> (h + 1) == 0};
            }
            ++n;
        }
        if (elect_one()) mma_commit(drained);
        __syncwarp();
        mbar_wait(drained, 0, nullptr, 0, nullptr);    // every product has ended
    } else if (warp < kSoftWarps) {
        // ------------------------------------------------ softmax: a (row, head) pair to a thread
        const int half = warp >> 2, r = (warp & 3) * 32 + lane;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + lanes + half * 128, tO = tmem + lanes + 256 + half * D;
        float m = -INFINITY, z = 0.f;          // reference (log2), sum
        int cur = -1, pos = -1, token = 0, ops = 0, splits = 0;
        bool used = false;
        Item it{};

        auto begin = [&](int item) {
            cur = item;
            it = items[item % kRing];
            const int rho = it.split ? r : half * 128 + r, pairs = it.rows * p.G;
            token = rho / p.G;
            pos = rho < pairs ? a.row_pos[it.row + token] : -1;
            if ((long long)pos >= (long long)p.max_blocks * kPage) pos = -1;
            m = -INFINITY;
            z = 0.f;
            used = false;
            // this warp's 32 pairs of queries, features in the order of the codes'
            constexpr int CPR = D / 8, RPI = 32 / CPR, N = 32 / RPI;
            uint4 u[N];
            const int c = lane % CPR;
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const int rr = (warp & 3) * 32 + j * RPI + lane / CPR, rh = it.split ? rr : half * 128 + rr;
                u[j] = make_uint4(0, 0, 0, 0);
                if (rh < pairs)
                    u[j] = __ldg(reinterpret_cast<const uint4 *>(a.q + ((long long)(it.row + rh / p.G) * p.Hq + it.group * p.G + rh % p.G) * D) + c);
            }
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const int rr = (warp & 3) * 32 + j * RPI + lane / CPR;
                const uint4 y = make_uint4(__byte_perm(u[j].x, u[j].y, 0x5410), __byte_perm(u[j].x, u[j].y, 0x7632),
                                           __byte_perm(u[j].z, u[j].w, 0x5410), __byte_perm(u[j].z, u[j].w, 0x7632));
                *reinterpret_cast<uint4 *>(sm + half * S::TILE + (c >> 3) * kSub + rr * 128 + (((c & 7) ^ (rr & 7)) << 4)) = y;
            }
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(&q_full[half]);
        };

        // Scores to probabilities, in their place.
        auto page = [&](int lim, bool first, float fa, float lv, float il, float pv) {
            if (!mbar_wait_warp(&s_full[half], (uint32_t)ops++ & 1u, st, 189, abort_flag)) return false;
            fence_after_sync();
            const bool all = __all_sync(0xffffffffu, lim >= kPage - 1);
            if (!__any_sync(0xffffffffu, lim >= 0)) {
                const uint32_t none[16] = {};
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_st16(tS + c * 16, none);
            } else {
                float mq[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int c64 = 0; c64 < 2; ++c64) {
                    uint32_t s0[32], s1[32];
                    tmem_ld32_nowait(tS + c64 * 64, s0);
                    tmem_ld32_nowait(tS + c64 * 64 + 32, s1);
                    tmem_wait32(s0);
                    tmem_wait32(s1);
                    if (all) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) mq[j & 3] = fmaxf(mq[j & 3], fmaxf(__uint_as_float(s0[j]), __uint_as_float(s1[j])));
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            if (c64 * 64 + j <= lim) mq[j & 3] = fmaxf(mq[j & 3], __uint_as_float(s0[j]));
                            if (c64 * 64 + 32 + j <= lim) mq[j & 3] = fmaxf(mq[j & 3], __uint_as_float(s1[j]));
                        }
                    }
                }
                const float t = fmaxf(fmaxf(mq[0], mq[1]), fmaxf(mq[2], mq[3])) * fa + lv;
                const bool up = t > m + kLag;
                const float keep = up ? ex2(m - t) : 1.f;
                if (!first && __any_sync(0xffffffffu, up && m != -INFINITY)) {
#pragma unroll
                    for (int c = 0; c < D; c += 32) {
                        uint32_t o[32];
                        tmem_ld32_nowait(tO + c, o);
                        tmem_wait32(o);
#pragma unroll
                        for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * keep);
                        tmem_st16(tO + c, o);
                        tmem_st16(tO + c + 16, o + 16);
                    }
                }
                z *= keep;
                m = up ? t : m;
                const float c0 = m == -INFINITY ? lv : lv - m;
                float zp[4] = {0.f, 0.f, 0.f, 0.f};
                auto powers = [&](auto plain_tag) {
                    constexpr bool kPlain = decltype(plain_tag)::value;    // no token is masked, no factor
#pragma unroll
                    for (int c64 = 0; c64 < 2; ++c64) {
                        uint32_t sr[2][32];
                        tmem_ld32_nowait(tS + c64 * 64, sr[0]);
                        tmem_ld32_nowait(tS + c64 * 64 + 32, sr[1]);
                        tmem_wait32(sr[0]);
                        tmem_wait32(sr[1]);
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            uint32_t pk[16];
#pragma unroll
                            for (int j = 0; j < 32; j += 2) {
                                const int at = c64 * 64 + x * 32 + j;
                                float e0 = ex2(fmaf(__uint_as_float(sr[x][j]), fa, c0)), e1 = ex2(fmaf(__uint_as_float(sr[x][j + 1]), fa, c0));
                                if constexpr (!kPlain) {
                                    e0 = at <= lim ? e0 : 0.f;
                                    e1 = at + 1 <= lim ? e1 : 0.f;
                                }
                                zp[(j >> 1) & 3] += e0 + e1;
                                pk[j / 2] = kPlain ? pack_bf16(e0, e1) : pack_bf16(at <= lim ? e0 * pv : 0.f, at + 1 <= lim ? e1 * pv : 0.f);
                            }
                            tmem_st16(tS + c64 * 32 + x * 16, pk);
                        }
                    }
                };
                if (all && pv == 1.f) powers(std::true_type{});
                else powers(std::false_type{});
                z += ((zp[0] + zp[1]) + (zp[2] + zp[3])) * il;
            }
            tmem_wait_st();
            fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[half]);
            used = true;
            return true;
        };

        // The features of a visible token's V codes that are NaN.
        auto spoiled = [&](uint32_t (&bad)[D / 32]) {
            for (int w = 0; w < D / 32; ++w) bad[w] = 0;
            for (int c = it.c0; c < it.c1; ++c) {
                const int block = a.sel ? plan.blocks[it.at + c] : c, page = a.block_table[(long long)it.req * p.max_blocks + block];
                if ((unsigned)page >= (unsigned)p.n_pages) continue;
                if (a.sel && !(plan.masks[(it.at + c) * a.words + (token >> 5)] >> (token & 31) & 1)) continue;
                const uint4 *row = reinterpret_cast<const uint4 *>(a.v8 + ((long long)page * p.Hkv + it.group) * kPage * D);
                for (int j = 0; j < kPage && block * kPage + j <= pos; ++j)
                    for (int w = 0; w < D / 16; ++w) {
                        const uint4 u = row[j * (D / 16) + w];
                        const uint32_t x[4] = {nan_codes(u.x), nan_codes(u.y), nan_codes(u.z), nan_codes(u.w)};
                        for (int k = 0; k < 4; ++k)
                            bad[w / 2] |= ((x[k] >> 7 & 1) | (x[k] >> 14 & 2) | (x[k] >> 21 & 4) | (x[k] >> 28 & 8)) << ((w & 1) * 16 + k * 4);
                    }
            }
        };

        auto finish = [&](int item) {
            if (!mbar_wait_warp(&o_full[half], (uint32_t)item & 1u, st, 190, abort_flag)) return false;
            fence_after_sync();
            const int rho = it.split ? r : half * 128 + r;
            const bool mine = rho < it.rows * p.G && pos >= 0;
            float wa = used ? 1.f : 0.f, wb = 0.f;
            if (it.split) {
                const uint32_t turn = splits++ & 1u;
                if (half == 1) {
                    state[r] = make_float2(used ? m : -INFINITY, used ? z : 0.f);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(b_ready);
                    return mbar_wait_warp(b_read, turn, st, 191, abort_flag);   // A has read this half's sums
                }
                if (!mbar_wait_warp(b_ready, turn, st, 192, abort_flag)) return false;
                const float2 b = state[r];
                const bool none = b.y == 0.f;                 // nothing visible on B's pages
                const float top = none ? m : fmaxf(m, b.x);
                wa = !used || z == 0.f ? 0.f : m == top ? 1.f : ex2(m - top);
                wb = none ? 0.f : b.x == top ? 1.f : ex2(b.x - top);
                z = (wa == 0.f ? 0.f : z * wa) + (wb == 0.f ? 0.f : b.y * wb);
                m = top;
            }
            const bool any_a = __any_sync(0xffffffffu, wa != 0.f), any_b = __any_sync(0xffffffffu, wb != 0.f);
            const float inv = it.part >= 0 ? 1.f : z == 0.f ? 0.f : 1.f / z;
            uint32_t bad[D / 32];
            const bool look = nan_item[item % kRing] == item;
            if (look && mine) spoiled(bad);
            __syncwarp();
            const long long row = (long long)(it.row + token) * p.Hq + it.group * p.G + rho % p.G;
            float *part = plan.part + ((long long)it.part * kTileRows + rho) * D;
#pragma unroll
            for (int c = 0; c < D; c += 32) {
                float x[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) x[j] = 0.f;
                uint32_t o[32];
                if (any_a) {
                    tmem_ld32_nowait(tO + c, o);
                    tmem_wait32(o);
#pragma unroll
                    for (int j = 0; j < 32; ++j) x[j] = wa == 0.f ? 0.f : __uint_as_float(o[j]) * wa;
                }
                if (any_b) {
                    tmem_ld32_nowait(tO + D + c, o);
                    tmem_wait32(o);
#pragma unroll
                    for (int j = 0; j < 32; ++j) x[j] += wb == 0.f ? 0.f : __uint_as_float(o[j]) * wb;
                }
                if (look && mine) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        const int f = (j & ~3) | (j & 3) >> 1 | (j & 1) << 1;       // column j is feature f
                        if (bad[c / 32] >> f & 1) x[j] = __uint_as_float(0x7FC00000u);
                    }
                }
                if (mine && it.part >= 0) {
#pragma unroll
                    for (int j = 0; j < 32; j += 4) *reinterpret_cast<float4 *>(part + c + j) = make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]);
                } else if (mine) {
#pragma unroll
                    for (int j = 0; j < 32; j += 8)
                        *reinterpret_cast<uint4 *>(a.o + row * D + c + j) =
                            make_uint4(pack_bf16(x[j] * inv, x[j + 2] * inv), pack_bf16(x[j + 1] * inv, x[j + 3] * inv),
                                       pack_bf16(x[j + 4] * inv, x[j + 6] * inv), pack_bf16(x[j + 5] * inv, x[j + 7] * inv));
                }
                __syncwarp();
            }
            if (mine) {
                if (it.part >= 0) plan.stats(a.ctas, D)[(long long)it.part * kTileRows + rho] = make_float2(z == 0.f ? -INFINITY : m, z);
                else a.lse[row] = z == 0.f ? -INFINITY : (m + log2f(z)) * kLn2;
            }
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
                const bool seen = x.mask[token >> 5] >> (token & 31) & 1;
                const int lim = seen ? min(pos - x.block * kPage, kPage - 1) : -1;
                const bool first = x.first >> half & 1;
                const float fa = x.a, lv = x.lv, il = x.il, pv = x.pv;
                done_entry(e);
                if (!page(lim, first, fa, lv, il, pv)) break;
            } else {
                done_entry(e);
                if (kind == kEndEntry && !finish(item)) break;
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
// A CTA of 8 rows for each stretch: those of the item that ends in it and was begun before.
template <int D>
__global__ void __launch_bounds__(256) chunk_join_kernel(Args a, AttnPlan plan)
{
    chain_next();
    chain_wait(a.row_pos, a.sel, a.o, a.lse);
    const PagedProblem &p = a.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, cta = blockIdx.x;
    const Pieces pieces(plan, a);
    const ChunkShare mine(pieces.total, a.ctas, kLeast, cta);
    if (mine.from >= mine.to) return;
    const long long item = pieces.find(mine.from, lane), start = pieces.start(item);
    if (start >= mine.from) return;
    const ChunkTile t = plan.tiles.tiles[item / p.Hkv];
    const int pages = pieces.pages(item), mt = tile_halves(t.rows * p.G), g = (int)(item % p.Hkv);
    int c0, c1;
    cut(start, pages, mt, mine.from, mine.to, c0, c1);
    if (c0 == 0 || c0 >= c1 || c1 != pages) return;
    const int rho = blockIdx.y * 8 + warp;
    if (rho >= t.rows * p.G) return;
    const int pos = a.row_pos[t.row + rho / p.G];
    if (pos < 0 || (long long)pos >= (long long)p.max_blocks * kPage) return;
    const float2 *stats = plan.stats(a.ctas, D);
    const int from = (int)(start / mine.share);
    auto slot = [&](int k) -> long long {
        int b0, b1;
        cut(start, pages, mt, mine.share * k, min(pieces.total, mine.share * (k + 1)), b0, b1);
        return b0 < b1 ? ((long long)2 * k + (b0 == 0)) * kTileRows + rho : -1;
    };
    float m = -INFINITY, z = 0.f, x[4] = {0.f, 0.f, 0.f, 0.f};
    for (int k = from; k <= cta; ++k) {
        const long long s = slot(k);
        if (s < 0) continue;
        const float2 b = stats[s];
        if (b.y == 0.f) continue;                              // none of its pages visible
        const float top = fmaxf(m, b.x), wa = m == top ? 1.f : ex2(m - top), wb = b.x == top ? 1.f : ex2(b.x - top);
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
        if (lane * 4 < D) y = *reinterpret_cast<const float4 *>(plan.part + s * D + lane * 4);
        z = z * wa + b.y * wb;
        x[0] = x[0] * wa + y.x * wb;
        x[1] = x[1] * wa + y.y * wb;
        x[2] = x[2] * wa + y.z * wb;
        x[3] = x[3] * wa + y.w * wb;
        m = top;
    }
    const long long row = (long long)(t.row + rho / p.G) * p.Hq + g * p.G + rho % p.G;
    const float inv = z == 0.f ? 0.f : 1.f / z;
    if (lane * 4 < D)
        *reinterpret_cast<uint2 *>(a.o + row * D + lane * 4) = make_uint2(pack_bf16(x[0] * inv, x[2] * inv), pack_bf16(x[1] * inv, x[3] * inv));
    if (lane == 0) a.lse[row] = z == 0.f ? -INFINITY : (m + log2f(z)) * kLn2;
}

int mask_words(const PagedProblem &p) { return std::max(1, kTileRows / p.G / 32); }
AttnPlan attn_plan(const PagedProblem &p, void *scratch, bool listed)
{
    const long long most = chunk_tiles(p, kTileRows / p.G);
    return AttnPlan(scratch, most, p, ChunkPlan::bytes(most), listed, mask_words(p), p.num_sms);
}

}  // namespace

size_t paged_chunk_scratch_bytes(const PagedProblem &p, bool attention)
{
    return attention ? attn_plan(p, nullptr, true).bytes : paged_chunk_scores_scratch(p);
}

cudaError_t launch_paged_chunk_attn(const PagedProblem &p, const bf16 *q, const uint8_t *k8, const uint8_t *v8, const float *k_scale,
                                    const float *v_scale, const int32_t *block_table, const int32_t *q_starts, const int32_t *row_pos,
                                    const int32_t *sel, bf16 *o, float *lse, void *scratch, DeviceStatus *st, cudaStream_t s)
{
    const int tokens = kTileRows / p.G;
    cudaError_t e = launch_chunk_plan(p, q_starts, row_pos, tokens, p.G, scratch, st, s);
    if (e != cudaSuccess) return e;
    const AttnPlan plan = attn_plan(p, scratch, sel != nullptr);
    const Args a{p, q, k8, v8, k_scale, v_scale, block_table, row_pos, sel, o, lse, tokens, mask_words(p), p.num_sms, st};
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
        return launch_chained("paged_chunk_join_kernel", chunk_join_kernel<D>, dim3(p.num_sms, kTileRows / 8), 256, 0, s, a, plan);
    };
    return p.d == 128 ? run(std::integral_constant<int, 128>{}) : run(std::integral_constant<int, 64>{});
}

}  // namespace msa
