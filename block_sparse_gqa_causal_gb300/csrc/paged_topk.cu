// paged_topk.cu -- the block selection of a ragged batch, from block scores:
// per (row, group) the row's own block and the topk - 1 earlier ones of
// largest score, ties to the lower block.
//
// Candidates are ranked by 64-bit keys (score, then lower block), all
// distinct, so the order is total and the result does not depend on how the
// work is split.  A warp keeps its 32 best, one to a lane, in descending order.
// A tile of 32 candidates is sorted and merged in only when one of them beats
// the (topk-1)-th best so far, which for scores in random order stops
// happening soon.  Rows of many blocks are cut over the CTA's warps, whose
// lists the first warp merges.
#include <algorithm>

#include "paged.h"

namespace msa {
namespace {

constexpr int kWarps = 8;

__device__ __forceinline__ unsigned long long merged(unsigned long long best, unsigned long long more, int lane)
{
    const unsigned long long o = shfl64(more, 31 - lane);     // both descending: the larger halves are bitonic
    return merge_desc64(best > o ? best : o, lane);
}

// W: warps of a row (1: a CTA takes eight rows, 8: one)
template <int W>
__global__ void __launch_bounds__(32 * kWarps)
topk_kernel(PagedProblem p, const float *__restrict__ scores, const int32_t *__restrict__ row_pos,
            int32_t *__restrict__ sel, DeviceStatus *st)
{
    __shared__ unsigned long long lists[kWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long row = W == 1 ? (long long)blockIdx.x * kWarps + warp : blockIdx.x;
    if (row >= (long long)p.T * p.Hkv) return;
    const int pos = row_pos[row / p.Hkv];
    if (pos < 0) return;                                      // a row behind the last request
    const int c0 = pos / kPage, k = p.topk;
    if (c0 >= p.max_blocks) {
        if (lane == 0) report(st, kDevCheck, 131, pos);
        return;
    }
    const float *sc = scores + row * p.max_blocks;
    unsigned long long best = 0;                              // 0: none
    if (c0 >= k && k > 1) {
        const int w = W == 1 ? 0 : warp;
        unsigned long long bar = 0;
        for (int base = w * 32; base < c0; base += 32 * W) {
            const int c = base + lane;
            float s = c < c0 ? sc[c] : 0.f;
            if (s != s) s = -INFINITY;                        // a NaN ranks last
            const unsigned long long key = c < c0 ? block_key(s, c) : 0ull;
            if (__ballot_sync(0xffffffffu, key > bar) == 0) continue;
            best = merged(best, sort_desc64(key, lane), lane);
            bar = shfl64(best, k - 2);
        }
        if (W > 1) {
            lists[warp][lane] = best;
            __syncthreads();
            if (warp != 0) return;
            for (int w2 = 1; w2 < W; ++w2) {
                const unsigned long long more = lists[w2][lane];
                if (__ballot_sync(0xffffffffu, more > shfl64(best, k - 2)) == 0) continue;
                best = merged(best, more, lane);
            }
        }
    } else if (W > 1 && warp != 0) {
        return;
    }
    // ascending blocks, then -1: sorted as 2^32 - 1 - block, none as 0
    uint32_t c = 0xFFFFFFFFu;
    if (c0 < k) {
        if (lane <= c0) c = (uint32_t)lane;
    } else if (lane < k - 1) {
        c = 0xFFFFFFFFu - (uint32_t)best;
    } else if (lane == k - 1) {
        c = (uint32_t)c0;
    }
    const unsigned long long asc = sort_desc64(c == 0xFFFFFFFFu ? 0ull : 0xFFFFFFFFull - c, lane);
    if (lane < k) sel[row * k + lane] = asc ? (int32_t)(0xFFFFFFFFu - (uint32_t)asc) : -1;
}

}  // namespace

cudaError_t launch_paged_block_topk(const PagedProblem &p, const float *scores, const int32_t *row_pos, int32_t *sel,
                                    DeviceStatus *st, cudaStream_t s)
{
    const long long rows = (long long)p.T * p.Hkv;
    const bool wide = p.max_blocks > 64 && rows < 8LL * p.num_sms * kWarps;
    {
        TimedLaunch timed_("paged_block_topk_kernel", s);
        if (wide) topk_kernel<kWarps><<<(unsigned)rows, 32 * kWarps, 0, s>>>(p, scores, row_pos, sel, st);
        else topk_kernel<1><<<(unsigned)((rows + kWarps - 1) / kWarps), 32 * kWarps, 0, s>>>(p, scores, row_pos, sel, st);
    }
    note_launch();
    return cudaGetLastError();
}

}  // namespace msa
