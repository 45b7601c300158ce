// paged_fork.cu -- block tables of a paged cache whose requests go on from one
// another's pages, and the moving of the pages in use to the pool's front.
//
// Forking.  A table entry is a reference to a page; shares[p] is one less than
// the references to p.  Slot r with a source s != r drops the references of its
// row and takes some of s's: whole pages as they are, a page of its own for a
// last one that is only partly filled (the caller's copies, `moves`).  All
// slots change at once (beams trade places), so all that is taken and dropped is
// summed into shares first, and shares[p] < 0 then says that nobody holds p any
// more.  Several slots may drop the same page; one of them, the first in the
// order of (slot, block), stands for it (owner[p], a minimum over keys, the same
// whatever the order of the atomics) and gives it back, so that the ring's order
// does not depend on timing.
//
// Compaction.  A bitmap of the pages in use; u of them.  The i-th one at or
// above u moves to the i-th hole below u: both lists are sums of bits over the
// bitmap's words.
//
// Both are phases over a few thousand table entries, each a handful of dependent
// reads, with a barrier between them: latency is all there is.  One cluster of
// eight CTAs runs all phases in one launch, its barrier in hardware.  A warp takes
// 256 entries of a row, eight loads of a thread in flight.  Sixteen CTAs were
// no faster.  8 beams of 1,000 tokens fork in 10 us, 256 requests of up to 32,120
// in 17; the plan of a compaction of 4,300 pages takes 14.
#include <algorithm>

#include "paged.h"

namespace msa {
namespace {

constexpr int kCtas = 8;
constexpr int kThreads = 1024;
constexpr int kWarps = kCtas * kThreads / 32;

using u64 = unsigned long long;

__device__ __forceinline__ int pages_of(int n) { return (int)(((unsigned)n + kPage - 1) / kPage); }
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}

struct Sum {
    long long a;
    int bad;
};

// The sum of a over the CTA and whether any thread is bad, on every thread.
__device__ Sum cta_sum(Sum v, Sum *buf)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v.a += __shfl_xor_sync(0xffffffffu, v.a, o);
    v.bad = __any_sync(0xffffffffu, v.bad);
    __syncthreads();
    if (lane == 0) buf[warp] = v;
    __syncthreads();
    v = buf[lane];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v.a += __shfl_xor_sync(0xffffffffu, v.a, o);
    v.bad = __any_sync(0xffffffffu, v.bad);
    return v;
}

// The largest x >= 0 of the CTA, on every thread.
__device__ int cta_max(int x, int *buf)
{
    x = __reduce_max_sync(0xffffffffu, x);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = x;
    __syncthreads();
    return __reduce_max_sync(0xffffffffu, buf[threadIdx.x & 31]);
}

// Exclusive sums of one int a thread over the CTA; total on every thread.
__device__ int cta_scan(int x, int *buf, int &total)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int in = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, in, o);
        if (lane >= o) in += y;
    }
    __syncthreads();
    if (lane == 31) buf[warp] = in;
    __syncthreads();
    int w = buf[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += y;
    }
    total = __shfl_sync(0xffffffffu, w, 31);
    const int before = warp ? __shfl_sync(0xffffffffu, w, warp - 1) : 0;
    return before + in - x;
}

// A warp's share of a row.
constexpr int kDeep = 8, kPiece = 32 * kDeep;

// scratch of a fork: by page the key of the slot and block that give it back; by request {tokens, pages before, page taken};
// by piece of a row the pages given back; the rows as they were
struct ForkScratch {
    u64 *owner;
    int32_t *new_len, *had, *take_at, *back_at, *old;
    __host__ __device__ ForkScratch(void *at, const PagedProblem &p)
    {
        owner = static_cast<u64 *>(at);
        new_len = reinterpret_cast<int32_t *>(owner + p.n_pages);
        had = new_len + p.R;
        take_at = had + p.R;
        back_at = take_at + p.R;
        old = back_at + (size_t)p.R * ((p.max_blocks + kPiece - 1) / kPiece);
    }
};

__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(kCtas, 1, 1)
fork_kernel(PagedProblem p, ForkArgs a, void *scratch, DeviceStatus *st)
{
    __shared__ Sum sums[32];
    __shared__ int ints[32];
    chain_next();
    chain_wait(a.src, a.lens, a.held, a.block_table, a.free_pages, a.free_state, a.shares, scratch);
    const ForkScratch x(scratch, p);
    const int tid = threadIdx.x, lane = tid & 31, cta = blockIdx.x;
    const int gwarp = (cta * kThreads + tid) >> 5;
    const int R = p.R, nb = p.max_blocks;
    auto row = [&](int r) { return a.block_table + (long long)r * nb; };
    auto is_page = [&](int page) { return (unsigned)page < (unsigned)p.n_pages; };

    // ---- what each slot becomes; every CTA looks at all of them, the first writes it down
    const int head = a.free_state[0], count = a.free_state[1];
    Sum total{0, 0};
    int taken = 0, most = 0;
    for (int r0 = 0; r0 < R; r0 += kThreads) {
        const int r = r0 + tid;
        int take = 0;
        if (r < R) {
            const int s = a.src[r], len = a.lens[r];
            const int had = a.held ? a.held[r] : len >= 0 ? pages_of(len) : 0;
            bool fine = s >= -1 && s < R && len >= 0 && (long long)len <= (long long)nb * kPage && had >= pages_of(len) && had <= nb;
            int n = fine && s == r ? len : 0;
            if (fine && s >= 0 && s != r) {
                const int most = a.lens[s];
                n = a.fork_lens ? a.fork_lens[r] : most;
                fine = n >= 0 && n <= most;
                take = fine && n % kPage != 0;
            }
            total.bad |= !fine;
            total.a += take;
            most = max(most, s == r ? 0 : max(had, n / kPage));
            if (cta == 0) {
                x.new_len[r] = n;
                x.had[r] = had;
            }
        }
        if (cta == 0) {                        // uniform over the CTA
            int all;
            const int before = cta_scan(take, ints, all);
            if (r < R) x.take_at[r] = taken + before;
            taken += all;
        }
    }
    total = cta_sum(total, sums);
    const bool fits = !total.bad && head >= 0 && head < p.n_pages && count >= 0 && count <= p.n_pages && total.a <= count;
    if (!fits) {
        if (cta == 0 && tid == 0) report(st, kDevCheck, 160, 0);
        for (int i = cta * kThreads + tid; i < R; i += kCtas * kThreads) {
            a.moves[3 * i] = a.moves[3 * i + 1] = -1;
            a.moves[3 * i + 2] = 0;
        }
        cluster_sync();
        return;
    }
    cluster_sync();

    // The rows' pieces that change, warp by warp: fn(r, s, first block, pages before, whole pages taken, piece).
    const int pieces = (cta_max(most, ints) + kPiece - 1) / kPiece;
    const long long items = (long long)R * pieces;
    auto each = [&](auto fn) {
        for (long long i = gwarp; i < items; i += kWarps) {
            const int r = (int)(i / pieces), s = a.src[r];
            if (s != r) fn(r, s, (int)(i % pieces) * kPiece, x.had[r], s >= 0 ? x.new_len[r] / kPage : 0, i);
        }
    };
    auto load = [&](int (&to)[kDeep], const int32_t *from, int first, int n) {
#pragma unroll
        for (int j = 0; j < kDeep; ++j) to[j] = first + 32 * j + lane < n ? from[first + 32 * j + lane] : -1;
    };
    // whether a row drops and takes a page (or the same entry that is none) at block b; outside of a row there is neither
    auto same = [&](int drop, int take, int b, int had, int full) { return drop == take && b < had && b < full; };
    auto key_of = [&](int r, int b) { return (u64)r * (u64)nb + (u64)b; };

    // A page that a row drops and takes at the same block, as beams of one prompt do with nearly all of theirs, stays held:
    // there is nothing to count, and nobody else gives it back either (256 requests of four prompts: 39 -> 21 us).

    // ---- the rows as they are; nobody gives a page back yet
    each([&](int r, int s, int b0, int had, int full, long long) {
        int drop[kDeep], take[kDeep];
        load(drop, row(r), b0, had);
        load(take, s >= 0 ? row(s) : row(r), b0, full);
#pragma unroll
        for (int j = 0; j < kDeep; ++j) {
            const int b = b0 + 32 * j + lane;
            if (b >= had) continue;
            x.old[(long long)r * nb + b] = drop[j];
            if (!is_page(drop[j])) report(st, kDevCheck, 161, r);
            else if (!same(drop[j], take[j], b, had, full)) x.owner[drop[j]] = ~0ull;
        }
    });
    cluster_sync();
    each([&](int r, int s, int b0, int had, int full, long long) {
        int drop[kDeep], take[kDeep];
        load(drop, row(r), b0, had);
        load(take, s >= 0 ? row(s) : row(r), b0, full);
#pragma unroll
        for (int j = 0; j < kDeep; ++j) {
            const int b = b0 + 32 * j + lane;
            if (same(drop[j], take[j], b, had, full)) continue;
            if (is_page(drop[j])) {
                atomicAdd(&a.shares[drop[j]], -1);
                atomicMin(&x.owner[drop[j]], key_of(r, b));
            }
            if (is_page(take[j])) atomicAdd(&a.shares[take[j]], 1);
            else if (b < full) report(st, kDevCheck, 161, r);
        }
    });
    cluster_sync();
    // Whether (r, b) gives its page back, for each of a thread's blocks.
    auto frees = [&](bool (&is)[kDeep], const int (&drop)[kDeep], const int (&take)[kDeep], int r, int b0, int had, int full) {
        u64 key[kDeep];
        int left[kDeep];
#pragma unroll
        for (int j = 0; j < kDeep; ++j) {
            const bool fine = is_page(drop[j]) && !same(drop[j], take[j], b0 + 32 * j + lane, had, full);
            key[j] = fine ? x.owner[drop[j]] : ~0ull;
            left[j] = fine ? a.shares[drop[j]] : 0;
        }
#pragma unroll
        for (int j = 0; j < kDeep; ++j) is[j] = left[j] < 0 && key[j] == key_of(r, b0 + 32 * j + lane);
    };
    // ---- pages given back, piece by piece
    for (long long i = cta * kThreads + tid; i < items; i += kCtas * kThreads) {
        const int r = (int)(i / pieces);
        if (a.src[r] == r) x.back_at[i] = 0;
    }
    each([&](int r, int s, int b0, int had, int full, long long i) {
        int drop[kDeep], take[kDeep], back = 0;
        bool is[kDeep];
        load(drop, row(r), b0, had);
        load(take, s >= 0 ? row(s) : row(r), b0, full);
        frees(is, drop, take, r, b0, had, full);
#pragma unroll
        for (int j = 0; j < kDeep; ++j) back += __popc(__ballot_sync(0xffffffffu, is[j]));
        if (lane == 0) x.back_at[i] = back;
    });
    cluster_sync();
    int given = 0;
    if (cta == 0) {
        for (long long i0 = 0; i0 < items; i0 += kThreads) {
            const long long i = i0 + tid;
            int all;
            const int before = cta_scan(i < items ? x.back_at[i] : 0, ints, all);
            if (i < items) x.back_at[i] = given + before;
            given += all;
        }
    }
    cluster_sync();
    // ---- the ring, the tables and the moves
    // s's row as it was: its copy where s changes too
    auto source = [&](int s) { return a.src[s] != s ? x.old + (long long)s * nb : row(s); };
    each([&](int r, int s, int b0, int had, int full, long long i) {
        int drop[kDeep], take[kDeep];
        bool is[kDeep];
        int back = x.back_at[i];
        load(drop, x.old + (long long)r * nb, b0, had);
        load(take, s >= 0 ? source(s) : row(r), b0, full);
        frees(is, drop, take, r, b0, had, full);
#pragma unroll
        for (int j = 0; j < kDeep; ++j) {
            const int b = b0 + 32 * j + lane;
            const unsigned all = __ballot_sync(0xffffffffu, is[j]);
            if (is[j]) {
                a.free_pages[((long long)head + count + back + __popc(all & ((1u << lane) - 1))) % p.n_pages] = drop[j];
                a.shares[drop[j]] = 0;                 // nobody but this block's thread looks at it
            }
            back += __popc(all);
            if (b < full && !same(drop[j], take[j], b, had, full)) row(r)[b] = take[j];
        }
    });
    for (int r = cta * kThreads + tid; r < R; r += kCtas * kThreads) {
        const int s = a.src[r];
        int from = -1, to = -1, rows = 0;
        if (s != r) {
            const int n = x.new_len[r], full = n / kPage, rest = s >= 0 ? n % kPage : 0;
            if (rest) {
                const int page = a.free_pages[((long long)head + x.take_at[r]) % p.n_pages];
                from = source(s)[full];
                const bool fine = is_page(page);
                row(r)[full] = fine ? page : -1;
                if (fine) a.shares[page] = 0;
                if (fine && is_page(from)) {
                    to = page;
                    rows = rest;
                } else {
                    report(st, kDevCheck, 162, r);
                    from = -1;
                }
            }
            a.lens[r] = n;
            if (a.held) a.held[r] = pages_of(n);
        }
        a.moves[3 * (long long)r] = from;
        a.moves[3 * (long long)r + 1] = to;
        a.moves[3 * (long long)r + 2] = rows;
    }
    if (cta == 0 && tid == 0) {
        a.free_state[0] = (int)((head + total.a) % p.n_pages);
        a.free_state[1] = (int)(count - total.a + given);
    }
}

// scratch of a compaction: the bitmap, the pages to move, the holes, each moved page's new number
struct CompactScratch {
    uint32_t *bits;
    int32_t *movers, *holes, *to;
    __host__ __device__ CompactScratch(void *at, const PagedProblem &p)
    {
        bits = static_cast<uint32_t *>(at);
        movers = reinterpret_cast<int32_t *>(bits + (p.n_pages + 31) / 32);
        holes = movers + p.n_pages / 2 + 1;
        to = holes + p.n_pages / 2 + 1;
    }
};

__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(kCtas, 1, 1)
compact_kernel(PagedProblem p, CompactArgs a, void *scratch, DeviceStatus *st)
{
    __shared__ Sum sums[32];
    __shared__ int ints[32];
    chain_next();
    chain_wait(a.lens, a.held, a.block_table, a.shares, scratch);
    const CompactScratch x(scratch, p);
    const int tid = threadIdx.x, lane = tid & 31, cta = blockIdx.x;
    const int gtid = cta * kThreads + tid, gwarp = gtid >> 5, all_threads = kCtas * kThreads;
    const int R = p.R, nb = p.max_blocks, N = p.n_pages, words = (N + 31) / 32;

    for (int w = gtid; w < words; w += all_threads) x.bits[w] = 0;
    cluster_sync();
    auto held_of = [&](int r, bool &fine) {
        const int len = a.lens[r];
        const long long need = len < 0 ? 0 : min((long long)pages_of(len), (long long)nb);
        const long long had = a.held ? a.held[r] : need;
        fine = len >= 0 && (long long)len <= (long long)nb * kPage && had >= need && had <= nb;
        return (int)min(max(had, need), (long long)nb);
    };
    for (int r = gwarp; r < R; r += kWarps) {
        bool fine;
        const int had = held_of(r, fine);
        if (!fine && lane == 0) report(st, kDevCheck, 163, r);
        for (int b = lane; b < had; b += 32) {
            const int page = a.block_table[(long long)r * nb + b];
            if ((unsigned)page < (unsigned)N) atomicOr(&x.bits[page >> 5], 1u << (page & 31));
            else report(st, kDevCheck, 164, r);
        }
    }
    cluster_sync();
    Sum used{0, 0};
    for (int w = tid; w < words; w += kThreads) used.a += __popc(x.bits[w]);
    const int u = (int)cta_sum(used, sums).a;
    // pages in use at or above u (CTA 0), holes below it (CTA 1): as many
    int n = 0;
    if (cta < 2) {
        const int first = cta == 0 ? u >> 5 : 0, last = cta == 0 ? words : (u + 31) >> 5;
        int32_t *out = cta == 0 ? x.movers : x.holes;
        for (int w0 = first; w0 < last; w0 += kThreads) {
            const int w = w0 + tid;
            uint32_t m = 0;
            if (w < last) {
                const uint32_t low = u - w * 32 >= 32 ? ~0u : u - w * 32 <= 0 ? 0u : (1u << (u - w * 32)) - 1;   // pages below u
                m = cta == 0 ? x.bits[w] & ~low : ~x.bits[w] & low;
            }
            int total;
            int at = n + cta_scan(__popc(m), ints, total);
            for (; m; m &= m - 1) out[at++] = w * 32 + __ffs(m) - 1;
            n += total;
        }
    }
    // the others count for themselves
    Sum above{0, 0};
    for (int w = (u >> 5) + tid; w < words; w += kThreads) {
        const uint32_t m = x.bits[w];
        above.a += __popc(w == u >> 5 ? m & ~((1u << (u & 31)) - 1) : m);
    }
    const int moved = (int)cta_sum(above, sums).a;
    cluster_sync();
    const int most = max(1, N / 2);
    for (int i = gtid; i < most; i += all_threads) {
        const bool is = i < moved;
        const int from = is ? x.movers[i] : -1, to = is ? x.holes[i] : -1;
        a.moves[3 * (long long)i] = from;
        a.moves[3 * (long long)i + 1] = to;
        a.moves[3 * (long long)i + 2] = is ? kPage : 0;
        if (is) {
            x.to[from] = to;
            if (a.shares) a.shares_out[to] = a.shares[from];      // `to` was a hole: nobody else reads its count
        }
    }
    cluster_sync();
    for (int i = gtid; i < N; i += all_threads) {
        a.free_pages[i] = i < N - u ? u + i : -1;
        if (a.shares) {
            if (i >= u) a.shares_out[i] = 0;
            else if (x.bits[i >> 5] >> (i & 31) & 1) a.shares_out[i] = a.shares[i];
        }
    }
    for (int r = gwarp; r < R; r += kWarps) {
        bool fine;
        const int had = held_of(r, fine);
        const long long at = (long long)r * nb;
        for (int b = lane; b < nb; b += 32) {
            const int page = a.block_table[at + b];
            a.block_table_out[at + b] = b < had && page >= u && page < N ? x.to[page] : page;
        }
    }
    if (gtid == 0) {
        a.free_state[0] = 0;
        a.free_state[1] = N - u;
    }
}

// ---------------------------------------------------------------- copies
// Work comes in pieces: one head's K or V codes of a move, or its index keys (and the scales).  A CTA looks at 256 pieces
// at a time, a thread to each, and copies those that are any: a 16-KB tile in one go, five CTAs to an SM.  The memory
// bounds it: a compaction's 630 MB, read and written, take 100 us (93 at the copy rate).
constexpr int kCopyThreads = 256;

__global__ void __launch_bounds__(kCopyThreads, 5)
copy_kernel(PagedProblem p, const int32_t *moves, int n_moves, uint8_t *k8, uint8_t *v8, float *k_scale, float *v_scale, bf16 *k_idx,
            DeviceStatus *st)
{
    __shared__ int4 todo[kCopyThreads];       // {from, to, rows, part}
    __shared__ int n_todo[kCopyThreads / 32];
    chain_next();
    chain_wait(moves, k8, v8, k_scale, v_scale, k_idx);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int heads = k8 ? 2 * p.Hkv : 0, parts = heads + 1;
    const long long pieces = (long long)n_moves * parts;
    for (long long base = blockIdx.x; base < pieces; base += (long long)gridDim.x * kCopyThreads) {
        const long long piece = base + (long long)tid * gridDim.x;
        int4 me = make_int4(-1, -1, 0, 0);
        if (piece < pieces) {
            const int m = (int)(piece / parts);
            me = make_int4(moves[3 * (long long)m], moves[3 * (long long)m + 1], moves[3 * (long long)m + 2], (int)(piece % parts));
            if (me.x >= 0 && (me.x >= p.n_pages || (unsigned)me.y >= (unsigned)p.n_pages || (unsigned)me.z > (unsigned)kPage)) {
                report(st, kDevCheck, 165, m);
                me.x = -1;
            }
        }
        const unsigned any = __ballot_sync(0xffffffffu, me.x >= 0);
        if (lane == 0) n_todo[warp] = __popc(any);
        __syncthreads();
        int at = 0, n = 0;
        for (int w = 0; w < kCopyThreads / 32; ++w) {
            if (w < warp) at += n_todo[w];
            n += n_todo[w];
        }
        if (me.x >= 0) todo[at + __popc(any & ((1u << lane) - 1))] = me;
        __syncthreads();
        for (int i = 0; i < n; ++i) {
            const int4 t = todo[i];
            const uint4 *src;
            uint4 *dst;
            int words;
            if (t.w < heads) {
                uint8_t *cache = t.w < p.Hkv ? k8 : v8;
                const int h = t.w < p.Hkv ? t.w : t.w - p.Hkv;
                const long long tile = (long long)kPage * p.d;
                src = reinterpret_cast<const uint4 *>(cache + ((long long)t.x * p.Hkv + h) * tile);
                dst = reinterpret_cast<uint4 *>(cache + ((long long)t.y * p.Hkv + h) * tile);
                words = t.z * p.d / 16;
            } else {
                if (k8)
                    for (int h = tid; h < p.Hkv; h += kCopyThreads) {
                        k_scale[(long long)t.y * p.Hkv + h] = k_scale[(long long)t.x * p.Hkv + h];
                        v_scale[(long long)t.y * p.Hkv + h] = v_scale[(long long)t.x * p.Hkv + h];
                    }
                if (!k_idx) continue;
                const long long tile = (long long)kPage * p.d_idx;
                src = reinterpret_cast<const uint4 *>(k_idx + t.x * tile);
                dst = reinterpret_cast<uint4 *>(k_idx + t.y * tile);
                words = t.z * p.d_idx / 8;
            }
            for (int w0 = 0; w0 < words; w0 += 4 * kCopyThreads) {
                uint4 v[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (w0 + j * kCopyThreads + tid < words) v[j] = src[w0 + j * kCopyThreads + tid];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (w0 + j * kCopyThreads + tid < words) dst[w0 + j * kCopyThreads + tid] = v[j];
            }
        }
        __syncthreads();
    }
}

}  // namespace

size_t paged_fork_scratch_bytes(const PagedProblem &p)
{
    return (size_t)p.n_pages * 8 + 4 * (size_t)p.R * (3 + (size_t)(p.max_blocks + kPiece - 1) / kPiece + p.max_blocks);
}

cudaError_t launch_paged_fork(const PagedProblem &p, const ForkArgs &a, void *scratch, DeviceStatus *st, cudaStream_t s)
{
    return launch_chained("paged_fork_kernel", fork_kernel, dim3(kCtas), kThreads, 0, s, p, a, scratch, st);
}

size_t paged_compact_scratch_bytes(const PagedProblem &p)
{
    return 4 * ((size_t)(p.n_pages + 31) / 32 + 2 * ((size_t)p.n_pages / 2 + 1) + p.n_pages);
}

cudaError_t launch_paged_compact(const PagedProblem &p, const CompactArgs &a, void *scratch, DeviceStatus *st, cudaStream_t s)
{
    return launch_chained("paged_compact_kernel", compact_kernel, dim3(kCtas), kThreads, 0, s, p, a, scratch, st);
}

cudaError_t launch_paged_copy(const PagedProblem &p, const int32_t *moves, int n_moves, uint8_t *k8, uint8_t *v8, float *k_scale,
                              float *v_scale, bf16 *k_idx, DeviceStatus *st, cudaStream_t s)
{
    const long long pieces = (long long)n_moves * ((k8 ? 2 * p.Hkv : 0) + 1);
    return launch_chained("paged_copy_kernel", copy_kernel, dim3((unsigned)std::min(pieces, 5LL * p.num_sms)), kCopyThreads, 0, s, p, moves,
                          n_moves, k8, v8, k_scale, v_scale, k_idx, st);
}

}  // namespace msa
