// paged_plan.cu -- the plan of a serving step over a paged cache: which pages
// the step's new tokens take, each row's request, position and cache slot.
//
// Request r holds ceil(l/128) pages for its l tokens and brings n new ones; it
// takes ceil((l+n)/128) - ceil(l/128) pages from the front of a ring of free
// pages, requests in order.  Where lengths may be lowered between steps, the
// pages held are told apart from them: those past the length are filled again
// before any is taken.  A request that ended gives its pages back behind
// the ring's free ones, so a step's releases never meet its takes and the two
// need no order.  Everything else is exclusive sums over the requests: first
// row, first page taken, first segment.
//
// One CTA sums (the work is a few thousand integers; latency is all there is)
// and decides whether the step fits before anything is written.  Rows are
// independent after that: a row finds its request by bisection of q_starts.
// Up to kFusedRows rows (one to a thread) the same CTA fills them, a launch
// fewer; above that a second kernel does (4,000 rows: 5 us against 8).  64 decoding requests take 3 us; 256 requests with
// 32,768 new tokens in tables of 1,024 columns, some ending, 10 us.
#include <algorithm>

#include "paged.h"

namespace msa {
namespace {

constexpr int kFusedRows = 1024;
constexpr int kFillThreads = 256;
constexpr int kCopied = 2048;            // requests whose first rows a CTA copies

// scratch: {ring head, segments, -, -}, then per request {first page taken,
// first segment, length before, pages held before}
__device__ __forceinline__ int pages_of(int n) { return (n + kPage - 1) / kPage; }

__device__ __forceinline__ void fill_entry(const PagedProblem &p, const PlanArgs &a, const int32_t *scratch, int S,
                                           const int32_t *starts, int n_rows, int n_segs, int head, int i, DeviceStatus *st)
{
    if (i >= n_segs && i <= S) a.segs[i] = n_rows;
    if (i >= p.T) return;
    if (i >= n_rows) {
        a.row_req[i] = -1;
        a.row_pos[i] = -1;
        a.slots[i] = -1;
        return;
    }
    int lo = 0, hi = p.R;                       // the last r with q_starts[r] <= i
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (starts[mid] <= i) lo = mid;
        else hi = mid;
    }
    const int4 rq = reinterpret_cast<const int4 *>(scratch)[1 + lo];
    const int q0 = starts[lo];
    const int pos = rq.z + (i - q0), blk = pos / kPage, off = pos % kPage;
    int32_t *entry = a.block_table + (long long)lo * p.max_blocks + blk;
    int page;
    if (blk >= rq.w) {
        const int at = head + rq.x + (blk - rq.w);   // under twice the ring: its takes are at most its pages
        page = a.free_pages[at < p.n_pages ? at : at - p.n_pages];
        if (off == 0) *entry = (unsigned)page < (unsigned)p.n_pages ? page : -1;   // every page taken is opened by one row of the step
    } else {
        page = *entry;                          // the partly filled last page
    }
    a.row_req[i] = lo;
    a.row_pos[i] = pos;
    if ((unsigned)page < (unsigned)p.n_pages) {
        a.slots[i] = page * kPage + off;
    } else {
        a.slots[i] = -1;
        report(st, kDevCheck, 102, page);
    }
    if (i == q0 || off == 0) a.segs[rq.y + blk - rq.z / kPage] = i;
}

struct Sums {
    long long rows, take, gone, segs;
};
__device__ __forceinline__ Sums operator+(const Sums &x, const Sums &y)
{
    return {x.rows + y.rows, x.take + y.take, x.gone + y.gone, x.segs + y.segs};
}
__device__ __forceinline__ Sums shfl_up(const Sums &x, int d)
{
    return {__shfl_up_sync(0xffffffffu, x.rows, d), __shfl_up_sync(0xffffffffu, x.take, d),
            __shfl_up_sync(0xffffffffu, x.gone, d), __shfl_up_sync(0xffffffffu, x.segs, d)};
}

__global__ void __launch_bounds__(1024) plan_kernel(PagedProblem p, PlanArgs a, int32_t *scratch, int S, int fused,
                                                    DeviceStatus *st)
{
    __shared__ Sums warp_sum[32];
    __shared__ int bad, n_ended, lost;
    __shared__ int3 ended[1024];
    chain_next();
    chain_wait(a.new_lens, a.lens_in, a.ended, a.free_in, a.held, a.block_table, a.free_pages, scratch);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nthr = blockDim.x, nwarp = nthr >> 5;
    const int head = a.free_in[0], count = a.free_in[1];
    const int most = p.max_blocks * kPage;
    if (tid == 0) bad = lost = 0;
    __syncthreads();

    struct Req {
        int had, old, n, held, after;
        Sums s;
    };
    auto load = [&](int r) {
        Req q{};
        if (r < p.R) {
            q.had = a.lens_in[r];
            q.n = a.new_lens[r];
            const bool ended = a.ended && a.ended[r] != 0;
            int pages = pages_of(q.had);                         // in the slot's row of the table
            if (q.had < 0 || q.had > most || q.n < 0 || q.n > most - (ended ? 0 : q.had)) {
                bad = 1;
                return q;
            }
            if (a.held) {
                const int h = a.held[r];
                if (h < pages || h > p.max_blocks) {
                    bad = 1;
                    return q;
                }
                pages = h;
            }
            q.old = ended ? 0 : q.had;
            q.held = ended ? 0 : pages;
            const int last = pages_of(q.old + q.n);
            q.after = max(q.held, last);
            q.s = {q.n, q.after - q.held, ended ? pages : 0, q.n > 0 ? last - q.old / kPage : 0};
        }
        return q;
    };
    // exclusive sum over the CTA's requests of one pass; the pass's total too
    auto scan = [&](const Sums &x, Sums &total) {
        Sums inc = x;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const Sums o = shfl_up(inc, d);
            if (lane >= d) inc = inc + o;
        }
        __syncthreads();
        if (lane == 31) warp_sum[warp] = inc;
        __syncthreads();
        if (warp == 0) {                                         // the warps' sums, summed up in turn
            Sums w = lane < nwarp ? warp_sum[lane] : Sums{};
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const Sums o = shfl_up(w, d);
                if (lane >= d) w = w + o;
            }
            warp_sum[lane] = w;
        }
        __syncthreads();
        const Sums before = warp ? warp_sum[warp - 1] : Sums{};
        total = warp_sum[31];
        return Sums{before.rows + inc.rows - x.rows, before.take + inc.take - x.take, before.gone + inc.gone - x.gone,
                    before.segs + inc.segs - x.segs};
    };

    // the step's totals decide whether it fits; nothing is written before that
    Sums total{};
    Req one{};
    Sums one_at{};
    for (int base = 0; base < p.R; base += nthr) {
        const Req q = load(base + tid);
        Sums t;
        const Sums at = scan(q.s, t);
        one = q;
        one_at = {total.rows + at.rows, total.take + at.take, total.gone + at.gone, total.segs + at.segs};
        total = total + t;
    }
    const bool ring_ok = head >= 0 && head < p.n_pages && count >= 0 && count <= p.n_pages;
    int why = 0;
    if (bad) why = 1;                                            // a length out of range
    else if (!ring_ok || total.gone + count > p.n_pages) why = 2;  // the ring's state
    else if (total.rows > p.T) why = 3;                          // more rows than T
    else if (total.take > count) why = 4;                        // too few free pages; those that come back do not count
    if (why) {
        if (tid == 0) report(st, kDevCheck, 101, why);
        total = Sums{};
    }
    if (tid == 0) {
        scratch[0] = head;
        scratch[1] = (int)total.segs;
    }
    const bool single = p.R <= nthr;                             // the scan above already is the whole one
    Sums run{};
    for (int base = 0; base < p.R; base += nthr) {
        const int r = base + tid;
        Req q;
        Sums at;
        if (single) {
            q = one;
            at = one_at;
        } else {
            q = load(r);
            Sums t;
            at = scan(q.s, t);
            at = at + run;
            run = run + t;
        }
        if (r < p.R) {
            a.q_starts[r] = why ? 0 : (int)at.rows;
            a.lens_out[r] = why ? a.lens_in[r] : q.old + q.n;
            if (a.held && !why) a.held[r] = q.after;
            if (!why) reinterpret_cast<int4 *>(scratch)[1 + r] = make_int4((int)at.take, (int)at.segs, q.old, q.held);
        }
        // pages of ended requests go behind the free ones, a warp to a request
        if (!why && total.gone > 0) {
            if (tid == 0) n_ended = 0;
            __syncthreads();
            if (q.s.gone > 0) ended[atomicAdd(&n_ended, 1)] = make_int3(r, (int)q.s.gone, (int)at.gone);
            __syncthreads();
            for (int i = warp; i < n_ended; i += nwarp) {
                const int3 e = ended[i];
                const int32_t *row = a.block_table + (long long)e.x * p.max_blocks;
                const int first = (int)(((long long)head + count + e.z) % p.n_pages);
                auto place = [&](int j) { return first + j < p.n_pages ? first + j : first + j - p.n_pages; };
                unsigned top = 0;
                constexpr int U = 16;                            // loads in flight before the stores they may not pass
                for (int j0 = lane; j0 < e.y; j0 += 32 * U) {
                    int32_t page[U];
#pragma unroll
                    for (int u = 0; u < U; ++u) page[u] = j0 + 32 * u < e.y ? row[j0 + 32 * u] : 0;
#pragma unroll
                    for (int u = 0; u < U; ++u)
                        if (j0 + 32 * u < e.y) a.free_pages[place(j0 + 32 * u)] = page[u];
#pragma unroll
                    for (int u = 0; u < U; ++u) top = max(top, (unsigned)page[u]);
                }
                if (top >= (unsigned)p.n_pages) {
                    report(st, kDevCheck, 103, (int)top);
                    lost = 1;
                }
            }
            __syncthreads();
        }
    }
    long long back = total.gone;
    if (total.gone > 0 && warp == 0 && lost) {                 // entries that are no pages do not enter the ring: the others move up
        back = 0;
        for (long long j0 = 0; j0 < total.gone; j0 += 32) {
            const int page = j0 + lane < total.gone ? a.free_pages[((long long)head + count + j0 + lane) % p.n_pages] : -1;
            const unsigned fine = __ballot_sync(0xffffffffu, (unsigned)page < (unsigned)p.n_pages);
            if (fine >> lane & 1) a.free_pages[((long long)head + count + back + __popc(fine & ((1u << lane) - 1))) % p.n_pages] = page;
            back += __popc(fine);
            __syncwarp();
        }
    }
    if (tid == 0) {
        a.q_starts[p.R] = (int)total.rows;
        a.free_out[0] = why ? head : (int)((head + total.take) % p.n_pages);
        a.free_out[1] = why ? count : (int)(count - total.take + back);
    }
    if (!fused) return;
    __syncthreads();
    const int n = max(p.T, S + 1);
    for (int i = tid; i < n; i += nthr)
        fill_entry(p, a, scratch, S, a.q_starts, (int)total.rows, (int)total.segs, head, i, st);
}

__global__ void __launch_bounds__(kFillThreads) plan_fill_kernel(PagedProblem p, PlanArgs a, const int32_t *scratch, int S,
                                                                 DeviceStatus *st)
{
    chain_next();
    chain_wait(a.q_starts, a.block_table, a.free_pages, scratch);
    // the bisection's steps depend on one another: a copy in shared memory answers them ten times sooner
    __shared__ int32_t copy[kCopied + 1];
    const bool small = p.R <= kCopied;
    if (small)
        for (int r = threadIdx.x; r <= p.R; r += kFillThreads) copy[r] = a.q_starts[r];
    __syncthreads();
    const int i = blockIdx.x * kFillThreads + threadIdx.x;
    fill_entry(p, a, scratch, S, small ? copy : a.q_starts, a.q_starts[p.R], scratch[1], scratch[0], i, st);
}

}  // namespace

size_t paged_plan_scratch_ints(const PagedProblem &p) { return 4 + 4 * (size_t)p.R; }

cudaError_t launch_paged_plan(const PagedProblem &p, const PlanArgs &a, int32_t *scratch, DeviceStatus *st, cudaStream_t s)
{
    const int S = paged_segments(p);
    const bool fused = p.T <= kFusedRows;
    const int want = a.ended ? 1024 : std::max(p.R, fused ? p.T : 1);
    const int threads = std::min(1024, std::max(64, (want + 31) / 32 * 32));
    cudaError_t e = launch_chained("paged_plan_kernel", plan_kernel, dim3(1), threads, 0, s, p, a, scratch, S, fused ? 1 : 0, st);
    if (e != cudaSuccess || fused) return e;
    const int n = std::max(p.T, S + 1);
    return launch_chained("paged_plan_fill_kernel", plan_fill_kernel, dim3((n + kFillThreads - 1) / kFillThreads), kFillThreads, 0,
                          s, p, a, (const int32_t *)scratch, S, st);
}

}  // namespace msa
