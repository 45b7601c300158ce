// paged_chunk.cu -- chunks of new tokens over a paged cache: the plan of their
// tiles, and the index branch's block scores,
//   block_scores[t, g, c] = max over visible tokens j of block c of
//                           scale_idx <q_idx[t, g], k_idx[j]>.
//
// Scores.  The index keys are shared by all groups, so a request's (row, group)
// pairs are the rows of one product with its pages: tiles of 256 pairs (two of
// M = 128) against one 128-token page, whose scores land in TMEM and are reduced
// there to their maxima; token scores never leave the SM.  The tensor cores bound
// it (2 x 128 x 128 x d_idx to a page and tile half); the maxima, 128 a row and page
// from TMEM, run beside the next page's products on the other accumulators.
// The work is one list of pages, those of (tile 0, head part 0), (tile 0, head
// part 1) and so on, cut into equal stretches for persistent CTAs, whatever the
// requests' lengths.  Pages and queries come by TMA; the queries have two
// buffers, so that a tile's first product does not wait for them.
// Each half has an issuer of its own: issuing blocks until the tensor cores take the
// instruction, so one warp's waits for the next page and accumulator came on top of
// its products (116 us for 2,048 rows of 8 groups over 32,768 tokens, against 101;
// the tensor cores' rate gives 68).  With the queries in TMEM instead, which leaves
// three accumulators, one issuer took 115: it was not shared memory that it waited for.
// Of the 101, 77 are pages (1,400 cycles each, of which the products need 1,024), the
// rest the start, the first queries and the blocks past the rows.
//   warp 0      TMA producer
//   warps 1, 2  tcgen05.mma issuers of the halves; TMEM
//   warps 3..10 one (row, group) to a thread: TMEM -> registers, causal mask, maximum, store
#include <algorithm>
#include <climits>

#include "paged_chunk.h"
#include "tc.cuh"

namespace msa {
namespace {

using namespace tc;

constexpr int kPlanThreads = 1024;

__device__ long long plan_scan(long long x, long long *buf, long long &total)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    long long in = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, in, o);
        if (lane >= o) in += y;
    }
    __syncthreads();
    if (lane == 31) buf[warp] = in;
    __syncthreads();
    long long w = buf[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += y;
    }
    total = __shfl_sync(0xffffffffu, w, 31);
    const long long before = __shfl_sync(0xffffffffu, w, warp ? warp - 1 : 0);
    return (warp ? before : 0) + in - x;
}

// The largest x of the threads before this one and of all, at least `least`.
__device__ int plan_max(int x, int least, int *buf, int &all)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto up_to = [&](int v) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v = max(v, y);
        }
        return v;
    };
    const int in = up_to(max(x, least));
    __syncthreads();
    if (lane == 31) buf[warp] = in;
    __syncthreads();
    const int w = up_to(buf[lane]);
    all = __shfl_sync(0xffffffffu, w, 31);
    const int warps = __shfl_sync(0xffffffffu, w, warp ? warp - 1 : 0), lanes = __shfl_up_sync(0xffffffffu, in, 1);
    return max(warp ? warps : least, lane ? lanes : least);
}

// One CTA: a request to a thread, then a tile to a thread, then a tile to a warp for the furthest position of its rows.
__global__ void __launch_bounds__(kPlanThreads)
chunk_plan_kernel(PagedProblem p, const int32_t *q_starts, const int32_t *row_pos, int tokens, int pairs, int most, void *at, DeviceStatus *st)
{
    __shared__ int first[kPlanThreads], start[kPlanThreads], rows[kPlanThreads];
    __shared__ long long buf[32];
    chain_next();
    chain_wait(q_starts, row_pos, at);
    const ChunkPlan plan(at, most);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int n = 0, left_out = 0, end = 0;              // end: of the requests so far
    for (int r0 = 0; r0 < p.R; r0 += kPlanThreads) {
        const int r = r0 + tid;
        int a = 0, b = 0;
        bool fine = true;
        if (r < p.R) {
            a = q_starts[r];
            b = q_starts[r + 1];
            fine = a >= 0 && a <= b && b <= p.T;
        }
        left_out |= __syncthreads_or(!fine);
        if (left_out) {                            // a request behind one that does not fit may begin in rows of those before it
            int all;
            const int before = plan_max(fine ? b : 0, end, first, all);
            fine = fine && (r >= p.R || a >= before);
            end = all;
        } else {
            end = q_starts[min(r0 + kPlanThreads, p.R)];
        }
        if (!fine) report(st, kDevCheck, 170, r);
        const int m = fine ? b - a : 0;
        long long all;
        const int mine = (int)plan_scan((m + tokens - 1) / tokens, buf, all);
        first[tid] = mine;
        start[tid] = a;
        rows[tid] = m;
        __syncthreads();
        for (int i = tid; i < (int)all; i += kPlanThreads) {
            int lo = 0, hi = kPlanThreads;               // the last request with first <= i: the one that has tile i
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (first[mid] <= i) lo = mid;
                else hi = mid;
            }
            const int off = (i - first[lo]) * tokens;
            plan.tiles[n + i] = ChunkTile{start[lo] + off, min(tokens, rows[lo] - off), r0 + lo, 0};      // no two tiles have a row
        }
        n += (int)all;
        __syncthreads();
    }
    for (int i = warp; i < n; i += kPlanThreads / 32) {
        const ChunkTile t = plan.tiles[i];
        int far = -1;
        for (int j = lane; j < t.rows; j += 32) {
            const int pos = row_pos[t.row + j];
            if ((long long)pos >= (long long)p.max_blocks * kPage) report(st, kDevCheck, 171, t.row + j);
            else far = max(far, pos);
        }
        far = __reduce_max_sync(0xffffffffu, far);
        if (lane == 0) plan.tiles[i].pages = far < 0 ? 0 : far / kPage + 1;
    }
    __syncthreads();
    long long sum = 0;
    for (int i0 = 0; i0 < n; i0 += kPlanThreads) {
        const int i = i0 + tid;
        long long all;
        const long long mine = plan_scan(i < n ? plan.tiles[i].pages * tile_halves(plan.tiles[i].rows * pairs) : 0, buf, all);
        if (i < n) plan.before[i] = sum + mine;
        sum += all;
    }
    if (tid == 0) {
        plan.before[n] = sum;
        plan.n_tiles[0] = n;
        plan.n_tiles[1] = left_out;
    }
}

// ---------------------------------------------------------------- scores
constexpr int kStages = 3;
constexpr int kLeast = 2;                      // units of work to a stretch at least
constexpr int kEpiWarps = 8;
constexpr int kThreads = 32 * (3 + kEpiWarps);
constexpr int kSub = 128 * 128;               // [128 rows][64 bf16], swizzled

template <int DI>
struct ScoresSmem {
    static constexpr int KB = DI / 64;
    static constexpr int Q = 2 * KB * kSub, K = KB * kSub;
    static constexpr int OFF_K = 2 * Q, OFF_BAR = OFF_K + kStages * K;
    // one CTA, which takes all 512 TMEM columns, to an SM
    static constexpr int BYTES = (OFF_BAR + 256 > 120 * 1024 ? OFF_BAR + 256 : 120 * 1024) + 1024;
};

// One stretch's walk over its tiles; every warp has its own.  A page belongs to the stretch that its first unit is in.
struct Walk {
    ChunkPlan plan;
    int parts, pairs;               // head parts of a tile, pairs of a token
    long long at, end;
    int i, part, c0, c1, mt;        // tile, head part, pages [c0, c1), halves
    ChunkTile t;
    __device__ Walk(const ChunkPlan &pl, int parts_, int pairs_, long long from, long long to, int tile)
        : plan(pl), parts(parts_), pairs(pairs_), at(from), end(to), i(tile)
    {
    }
    __device__ bool next()
    {
        do {
            if (at >= end) return false;
            while (at >= plan.before[i + 1] * parts) ++i;    // tiles without pages are passed over
            t = plan.tiles[i];
            mt = tile_halves(t.rows * pairs);
            const long long in = at - plan.before[i] * parts, whole = (long long)t.pages * mt;
            part = (int)(in / whole);
            const long long off = in - part * whole, stop = min(whole, off + (end - at));
            c0 = (int)((off + mt - 1) / mt);
            c1 = (int)((stop + mt - 1) / mt);
            at += stop - off;
        } while (c0 >= c1);
        return true;
    }
};

template <int DI>
__global__ void __launch_bounds__(kThreads, 1)
chunk_scores_kernel(PagedProblem p, const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                    const int32_t *block_table, const int32_t *q_starts, const int32_t *row_pos, float *scores, void *plan_at, int most,
                    int parts, DeviceStatus *st)
{
    using S = ScoresSmem<DI>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t *sK = smem + S::OFF_K;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + S::OFF_BAR);
    uint64_t *full = bars, *empty = bars + kStages, *q_full = bars + 2 * kStages, *q_empty = q_full + 2;
    uint64_t *acc_full = q_full + 4, *acc_empty = q_full + 8;      // [half][2]
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(q_full + 12);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    __shared__ int sh_tile;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 2);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&q_full[a], 1);
            mbar_init(&q_empty[a], 2);
        }
        for (int a = 0; a < 4; ++a) {
            mbar_init(&acc_full[a], 1);
            mbar_init(&acc_empty[a], kEpiWarps / 2);
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    chain_next();                 // behind the allocation: a successor that allocates too waits for this CTA to end
    const uint32_t tmem = *tmem_slot;
    chain_wait(block_table, q_starts, row_pos, scores, plan_at);

    const ChunkPlan plan(plan_at, most);
    const int n_tiles = *plan.n_tiles;
    const ChunkShare mine(plan.before[n_tiles] * parts, gridDim.x, kLeast, blockIdx.x);
    const long long from = mine.from, to = mine.to;
    if (warp == 0) {
        const int i = from < to ? chunk_find(plan.before, n_tiles, parts, from, lane) : 0;
        if (lane == 0) sh_tile = i;
    }
    __syncthreads();
    Walk walk(plan, parts, p.Hkv, from, to, sh_tile);

    if (warp == 0) {
        int n = 0, qn = 0, q_issued = 0, issued = 0;
        bool ok = true;
        while (ok && walk.next()) {
            const int a = qn & 1;
            if (!(ok = mbar_wait_warp(&q_empty[a], ((uint32_t)(qn >> 1) & 1u) ^ 1u, st, 172, abort_flag))) break;
            const long long first = (long long)walk.t.row * p.Hkv + walk.part * kTileRows;
            const int mt = walk.mt;
            if (elect_one()) {
                mbar_arrive_expect_tx(&q_full[a], mt * S::KB * kSub);
                for (int m = 0; m < mt; ++m)
                    for (int kb = 0; kb < S::KB; ++kb)
                        tma_load_3d(smem + a * S::Q + (m * S::KB + kb) * kSub, &tmap_q, &q_full[a], kb * 64, (int)(first + m * 128), 0);
            }
            __syncwarp();
            ++qn;
            q_issued = qn;
            const int32_t *table = block_table + (long long)walk.t.req * p.max_blocks;
            for (int c = walk.c0; ok && c < walk.c1; c += 32) {
                int page = c + lane < walk.c1 ? table[c + lane] : 0;
                if ((unsigned)page >= (unsigned)p.n_pages) {
                    report(st, kDevCheck, 173, page);
                    page = 0;                            // its maxima are passed over
                }
                for (int j = 0; j < 32 && c + j < walk.c1; ++j, ++n) {
                    const int s = n % kStages, z = __shfl_sync(0xffffffffu, page, j);
                    if (!(ok = mbar_wait_warp(&empty[s], ((uint32_t)(n / kStages) & 1u) ^ 1u, st, 174, abort_flag))) break;
                    if (elect_one()) {
                        mbar_arrive_expect_tx(&full[s], S::K);
                        for (int kb = 0; kb < S::KB; ++kb) tma_load_3d(sK + s * S::K + kb * kSub, &tmap_k, &full[s], kb * 64, 0, z);
                    }
                    __syncwarp();
                    issued = n + 1;
                }
            }
        }
        if (*abort_flag) {
            // this CTA's own copies land before it ends (bounded waits)
            for (int i = max(0, q_issued - 2); i < q_issued; ++i) mbar_wait(&q_full[i & 1], (uint32_t)(i >> 1) & 1u, nullptr, 0, nullptr);
            for (int i = max(0, issued - kStages); i < issued; ++i)
                mbar_wait(&full[i % kStages], (uint32_t)(i / kStages) & 1u, nullptr, 0, nullptr);
        }
    } else if (warp <= 2) {
        constexpr uint32_t kIdesc = idesc_bf16(128, 128);
        const int m = warp - 1;
        uint64_t *my_full = acc_full + 2 * m, *my_empty = acc_empty + 2 * m;
        int n = 0, unit = 0, qn = 0;
        bool ok = true;
        while (ok && walk.next()) {
            const int aq = qn & 1;
            const bool part_of = m < walk.mt;         // a tile of one half passes the second's issuer by
            if (!(ok = mbar_wait_warp(&q_full[aq], (uint32_t)(qn >> 1) & 1u, st, 175, abort_flag))) break;
            const uint64_t dq = sdesc_k128(smem_u32(smem + aq * S::Q + m * S::KB * kSub));
            for (int c = walk.c0; c < walk.c1; ++c, ++n) {
                const int s = n % kStages, a = unit & 1;
                if (part_of && !(ok = mbar_wait_warp(&my_empty[a], ((uint32_t)(unit >> 1) & 1u) ^ 1u, st, 176, abort_flag))) break;
                if (!(ok = mbar_wait_warp(&full[s], (uint32_t)(n / kStages) & 1u, st, 177, abort_flag))) break;
                fence_after_sync();
                const uint64_t dk = sdesc_k128(smem_u32(sK + s * S::K));
                if (elect_one()) {
                    if (part_of) {
#pragma unroll
                        for (int ks = 0; ks < DI / 16; ++ks) {
                            const uint32_t off = (ks >> 2) * kSub + (ks & 3) * 32;
                            mma_bf16(tmem + (uint32_t)((m * 2 + a) * 128), desc_adv(dq, off), desc_adv(dk, off), kIdesc, ks > 0);
                        }
                        mma_commit(&my_full[a]);
                        mma_commit(&empty[s]);
                        if (c + 1 == walk.c1) mma_commit(&q_empty[aq]);
                    } else {
                        mbar_arrive(&empty[s]);
                        if (c + 1 == walk.c1) mbar_arrive(&q_empty[aq]);
                    }
                }
                __syncwarp();
                unit += part_of;
            }
            ++qn;
        }
        if (*abort_flag && unit > 0)    // MMAs end in order: the last batch's end is that of all
            mbar_wait(&my_full[(unit - 1) & 1], (uint32_t)((unit - 1) >> 1) & 1u, nullptr, 0, nullptr);
    } else {
        const int m = (warp - 3) >> 2, quarter = warp & 3;
        const int row = m * 128 + quarter * 32 + lane;          // of the tile
        const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
        int unit = 0;
        bool ok = true;
        while (ok && walk.next()) {
            if (m >= walk.mt) continue;
            const int here = parts > 1 ? min(kTileRows, p.Hkv - walk.part * kTileRows) : walk.t.rows * p.Hkv;
            const long long rho = (long long)walk.t.row * p.Hkv + walk.part * kTileRows + row;
            const bool mine = row < here;
            int pos = mine ? row_pos[rho / p.Hkv] : -1;
            if ((long long)pos >= (long long)p.max_blocks * kPage) pos = -1;
            const int c_last = pos < 0 ? -1 : pos / kPage;
            const int first_pos = __reduce_min_sync(0xffffffffu, mine ? pos : INT_MAX);
            float *out = scores + rho * p.max_blocks;
            const int32_t *table = block_table + (long long)walk.t.req * p.max_blocks;
            for (int c8 = walk.c0; c8 < walk.c1; c8 += 8) {
                const int pages = min(8, walk.c1 - c8);
                const unsigned good = __ballot_sync(0xffffffffu, lane < pages && (unsigned)table[c8 + lane] < (unsigned)p.n_pages);
                float grp[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) grp[k] = -INFINITY;
                // (rolled: eight copies of this do not stay in the instruction cache)
#pragma unroll 1
                for (int u = 0; u < pages; ++u, ++unit) {
                    const int a = m * 2 + (unit & 1);
                    if (!mbar_wait_warp(&acc_full[a], (uint32_t)(unit >> 1) & 1u, st, 178, abort_flag)) {
                        ok = false;
                        break;
                    }
                    fence_after_sync();
                    const uint32_t base = tmem + lane_base + (uint32_t)(a * 128);
                    uint32_t v[4][32];
#pragma unroll
                    for (int k = 0; k < 4; ++k) tmem_ld32_nowait(base + k * 32, v[k]);
#pragma unroll
                    for (int k = 0; k < 4; ++k) tmem_wait32(v[k]);
                    fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&acc_empty[a]);
                    const int j0 = (c8 + u) * kPage;
                    if (j0 + kPage - 1 > first_pos) {
                        const int lim = min(pos - j0, kPage - 1);      // last visible token of the page for this row
#pragma unroll
                        for (int k = 0; k < 4; ++k)
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                if (k * 32 + j > lim) v[k][j] = __float_as_uint(-INFINITY);
                    }
                    float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int k = 0; k < 4; k += 2)
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            m4[j & 3] = fmaxf(m4[j & 3], fmaxf(__uint_as_float(v[k][j]), __uint_as_float(v[k + 1][j])));
                    const float most = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * p.scale_idx;
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (k == u && (good >> u & 1)) grp[k] = most;
                }
                if (!ok) break;
                const int last = min(c8 + pages - 1, c_last);
                if (last == c8 + 7 && ((reinterpret_cast<uintptr_t>(out + c8) & 15) == 0)) {
                    reinterpret_cast<float4 *>(out + c8)[0] = make_float4(grp[0], grp[1], grp[2], grp[3]);
                    reinterpret_cast<float4 *>(out + c8)[1] = make_float4(grp[4], grp[5], grp[6], grp[7]);
                } else {
#pragma unroll
                    for (int u = 0; u < 8; ++u)
                        if (c8 + u <= last) out[c8 + u] = grp[u];
                }
            }
        }
    }
    // the blocks past each row's own, a warp to a (row, group); tile by tile where a request was left out
    auto past = [&](long long i, int pos) {
        float *dst = scores + i * p.max_blocks;
        for (int c = min(pos / kPage + 1, p.max_blocks) + lane; pos >= 0 && c < p.max_blocks; c += 32) dst[c] = -INFINITY;
    };
    const int me = (int)blockIdx.x * (kThreads / 32) + warp, all = (int)gridDim.x * (kThreads / 32);
    if (!plan.n_tiles[1]) {
        for (long long i = (long long)q_starts[0] * p.Hkv + me; i < (long long)q_starts[p.R] * p.Hkv; i += all) past(i, row_pos[i / p.Hkv]);
    } else {
        for (int n = me; n < n_tiles; n += all)
            for (int j = 0; j < plan.tiles[n].rows * p.Hkv; ++j) past((long long)plan.tiles[n].row * p.Hkv + j, row_pos[plan.tiles[n].row + j / p.Hkv]);
    }
    fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        fence_after_sync();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace

cudaError_t launch_chunk_plan(const PagedProblem &p, const int32_t *q_starts, const int32_t *row_pos, int tokens, int pairs, void *plan,
                              DeviceStatus *st, cudaStream_t s)
{
    return launch_chained("paged_chunk_plan_kernel", chunk_plan_kernel, dim3(1), kPlanThreads, 0, s, p, q_starts, row_pos, tokens,
                          pairs, (int)chunk_tiles(p, tokens), plan, st);
}

// Rows of a tile: as many as make 256 (row, group) pairs; a row with more groups than that is cut into parts.
static int score_tokens(const PagedProblem &p) { return p.Hkv > kTileRows ? 1 : kTileRows / p.Hkv; }

size_t paged_chunk_scores_scratch(const PagedProblem &p) { return ChunkPlan::bytes(chunk_tiles(p, score_tokens(p))); }

cudaError_t launch_paged_chunk_scores(const PagedProblem &p, const bf16 *q_idx, const bf16 *k_idx, const int32_t *block_table,
                                      const int32_t *q_starts, const int32_t *row_pos, float *scores, void *scratch, DeviceStatus *st,
                                      cudaStream_t s)
{
    const int tokens = score_tokens(p), parts = p.Hkv > kTileRows ? (p.Hkv + kTileRows - 1) / kTileRows : 1;
    cudaError_t e = launch_chunk_plan(p, q_starts, row_pos, tokens, p.Hkv, scratch, st, s);
    if (e != cudaSuccess) return e;
    CUtensorMap tq, tk;
    const unsigned long long pairs = (unsigned long long)p.T * p.Hkv;
    if ((e = make_tmap_bf16_3d(&tq, q_idx, p.d_idx, pairs, 1, p.d_idx * 2ull, pairs * p.d_idx * 2, 64, 128)) != cudaSuccess) return e;
    if ((e = make_tmap_bf16_3d(&tk, k_idx, p.d_idx, kPage, p.n_pages, p.d_idx * 2ull, (unsigned long long)kPage * p.d_idx * 2, 64, kPage)) != cudaSuccess)
        return e;
    auto run = [&](auto kernel, int smem, std::atomic<unsigned long long> &allowed) {
        if ((e = allow_smem(kernel, smem, allowed)) != cudaSuccess) return e;
        return launch_chained("paged_chunk_scores_kernel", kernel, dim3(p.num_sms), kThreads, smem, s, p, tq, tk, block_table, q_starts, row_pos,
                              scores, scratch, (int)chunk_tiles(p, tokens), parts, st);
    };
    static std::atomic<unsigned long long> allowed64{0}, allowed128{0};
    return p.d_idx == 128 ? run(chunk_scores_kernel<128>, ScoresSmem<128>::BYTES, allowed128) : run(chunk_scores_kernel<64>, ScoresSmem<64>::BYTES, allowed64);
}

}  // namespace msa
