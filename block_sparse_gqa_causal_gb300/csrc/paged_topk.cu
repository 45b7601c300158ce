// paged_topk.cu -- the block selection of a ragged batch, from block scores:
// per (row, group) the row's own block and the topk - 1 earlier ones of
// largest score, ties to the lower block.
//
// The order is total (score, then lower block), so the result does not depend
// on how the work is split.  A warp takes 1,024 blocks at a time, 32 to a lane,
// in registers.  The (topk-1)-th largest of the 32 lanes' maxima is a lower
// bound of the (topk-1)-th best score, and only about twenty of 1,024 scores in
// random order reach it: these alone are listed.  Where they are at most 32,
// one to a lane, and the row has no other tile, one sort of their scores gives
// the last score that is in, and the equals of it that fit are found apart.
// Else (scores that tie make the list longer, not wrong) they are ranked by
// 64-bit keys and merged into the warp's 32 best, and rows of more than 1,024
// blocks are cut over a CTA's warps, whose lists the first warp merges.  8,000
// rows over 1,024 blocks take 8 us (the sorting networks' shuffles; reading
// the scores takes 2.5; 9 with a 64-bit sort of every list), 512 rows of 256
// blocks 3 us.
#include <algorithm>

#include "paged.h"

namespace msa {
namespace {

constexpr int kPer = 32;                 // scores of a lane
constexpr int kTile = 32 * kPer;         // blocks a warp takes at a time

__device__ __forceinline__ unsigned long long merged(unsigned long long best, unsigned long long more, int lane)
{
    const unsigned long long o = shfl64(more, 31 - lane);     // both descending: the larger halves are bitonic
    return merge_desc64(best > o ? best : o, lane);
}

// descending bitonic sort of one value per lane
template <class T>
__device__ __forceinline__ T sort_desc(T v, int lane)
{
#pragma unroll
    for (int size = 2; size <= 32; size <<= 1) {
#pragma unroll
        for (int stride = size >> 1; stride > 0; stride >>= 1) {
            const T o = __shfl_xor_sync(0xffffffffu, v, stride);
            const bool desc = (lane & size) == 0 || size == 32;
            v = ((lane & stride) == 0) == desc ? max(v, o) : min(v, o);
        }
    }
    return v;
}

// the score of a ranking key; -inf of none
__device__ __forceinline__ float worst(unsigned long long key)
{
    const uint32_t u = (uint32_t)(key >> 32);
    return key == 0 ? -INFINITY : __uint_as_float(u & 0x80000000u ? u ^ 0x80000000u : ~u);
}

// W: warps of a row; R: rows of a CTA
template <int W, int R>
__global__ void __launch_bounds__(32 * W * R)
topk_kernel(PagedProblem p, const float *__restrict__ scores, const int32_t *__restrict__ row_pos,
            int32_t *__restrict__ sel, DeviceStatus *st)
{
    static_assert(W == 1 || R == 1, "a row's warps fill the CTA");
    __shared__ int list[W * R][kTile];                        // the blocks of a tile that reach the bound
    __shared__ unsigned long long lists[W][32];
    chain_next();
    chain_wait(scores, row_pos);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long row = W == 1 ? (long long)blockIdx.x * R + warp : blockIdx.x;
    if (row >= (long long)p.T * p.Hkv) return;
    const int pos = row_pos[row / p.Hkv];
    if (pos < 0) return;                                      // a row behind the last request
    const int c0 = pos / kPage, k = p.topk;
    if (c0 >= p.max_blocks) {
        if (lane == 0) report(st, kDevCheck, 131, pos);
        return;
    }
    const float *sc = scores + row * p.max_blocks;
    unsigned long long best = 0;                              // this lane's of the warp's 32 best; 0: none
    uint32_t picked = 0;                                      // or the selection itself, 2^32 - 1 - block; 0: none
    bool done = false;
    if (c0 >= k && k > 1) {
        int *mine = list[warp];
        for (int base = (W == 1 ? 0 : warp) * kTile; base < c0; base += W * kTile) {
            const int n = min(kTile, c0 - base), mine_n = (n - lane + 31) / 32;   // this lane's: blocks base + lane + 32 i
            float v[kPer], top = -INFINITY;
#pragma unroll
            for (int g = 0; g < kPer; g += 8) {
                if (g * 32 < n) {                             // the warp's eights that hold blocks at all
#pragma unroll
                    for (int i = g; i < g + 8; ++i) v[i] = i < mine_n ? sc[base + i * 32 + lane] : -INFINITY;
                }
            }
#pragma unroll
            for (int g = 0; g < kPer; g += 8)
                if (g * 32 < n) {
#pragma unroll
                    for (int i = g; i < g + 8; ++i) top = fmaxf(top, v[i]);   // passes NaN over
                }
            const float bound = fmaxf(__shfl_sync(0xffffffffu, sort_desc(top, lane), k - 2), worst(shfl64(best, k - 2)));
            uint32_t in = 0;
#pragma unroll
            for (int g = 0; g < kPer; g += 8)
                if (g * 32 < n) {
#pragma unroll
                    for (int i = g; i < g + 8; ++i)
                        if (v[i] >= bound) in |= 1u << i;
                }
            if (bound == -INFINITY) in = ~0u;                 // a NaN ranks last: with -inf
            in &= mine_n >= 32 ? ~0u : mine_n > 0 ? (1u << mine_n) - 1 : 0u;
            int at = __popc(in), m = at;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int o = __shfl_up_sync(0xffffffffu, at, d);
                if (lane >= d) at += o;
            }
            m = __shfl_sync(0xffffffffu, at, 31);
            at -= __popc(in);
            for (; in; in &= in - 1) mine[at++] = base + lane + 32 * (__ffs(in) - 1);
            __syncwarp();
            if (W == 1 && m <= 32 && c0 <= kTile) {
                // all of the row's candidates, one to a lane: those above the (topk-1)-th score, and of its equals the
                // lowest blocks
                int c = lane < m ? mine[lane] : 0;
                float x = lane < m ? fmaxf(sc[c], -INFINITY) : -INFINITY;
                const float last = __shfl_sync(0xffffffffu, sort_desc(x, lane), k - 2);
                bool take = lane < m && x > last;
                const bool equal = lane < m && x == last;
                const int room = k - 1 - __popc(__ballot_sync(0xffffffffu, take));
                if (__popc(__ballot_sync(0xffffffffu, equal)) > room) {
                    const uint32_t order = sort_desc(equal ? 0xFFFFFFFFu - (uint32_t)c : 0u, lane);
                    const uint32_t least = __shfl_sync(0xffffffffu, order, room - 1);
                    take = take || (equal && 0xFFFFFFFFu - (uint32_t)c >= least);
                } else {
                    take = take || equal;
                }
                picked = take ? 0xFFFFFFFFu - (uint32_t)c : 0u;
                done = true;
                break;
            }
            for (int i = 0; i < m; i += 32) {
                unsigned long long key = 0;
                if (i + lane < m) {
                    const int c = mine[i + lane];
                    const float s = sc[c];
                    key = block_key(s != s ? -INFINITY : s, c);
                }
                if (__ballot_sync(0xffffffffu, key > shfl64(best, k - 2)) == 0) continue;
                key = sort_desc64(key, lane);
                best = base == 0 && i == 0 ? key : merged(best, key, lane);
            }
            __syncwarp();
        }
        if (W > 1) {
            lists[warp][lane] = best;
            __syncthreads();
            if (warp != 0) return;
            for (int w = 1; w < W; ++w) {
                const unsigned long long more = lists[w][lane];
                if (__ballot_sync(0xffffffffu, more > shfl64(best, k - 2)) == 0) continue;
                best = merged(best, more, lane);
            }
        }
    } else if (W > 1 && warp != 0) {
        return;
    }
    // ascending blocks, then -1: sorted as 2^32 - 1 - block, none as 0
    uint32_t c = 0;
    if (c0 < k) {
        if (lane <= c0) c = 0xFFFFFFFFu - (uint32_t)lane;
    } else {
        // the row's own block is the last: it needs no place in the sort
        c = done ? picked : lane < k - 1 ? (uint32_t)best : 0u;   // a key's low half
    }
    c = sort_desc(c, lane);
    if (c0 >= k && lane == k - 1) c = 0xFFFFFFFFu - (uint32_t)c0;
    if (lane < k) sel[row * k + lane] = c ? (int32_t)(0xFFFFFFFFu - c) : -1;
}

}  // namespace

cudaError_t launch_paged_block_topk(const PagedProblem &p, const float *scores, const int32_t *row_pos, int32_t *sel,
                                    DeviceStatus *st, cudaStream_t s)
{
    constexpr int W = 8, R = 4;
    const long long rows = (long long)p.T * p.Hkv;
    const bool wide = p.max_blocks > kTile;
    return launch_chained("paged_block_topk_kernel", wide ? topk_kernel<W, 1> : topk_kernel<1, R>,
                          dim3((unsigned)(wide ? rows : (rows + R - 1) / R)), 32 * (wide ? W : R), 0, s, p, scores, row_pos, sel, st);
}

}  // namespace msa
