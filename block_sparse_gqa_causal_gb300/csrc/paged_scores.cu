// paged_scores.cu -- the index branch over a ragged batch with paged index
// keys: for every row t, group g and block c of the row's request,
//   bs[t, g, c] = scale_idx * max over the block's tokens j <= pos(t) of
//                 <q_idx[t, g, :], k_idx[j, :]>,
// -inf for blocks past the row's own.
//
// In decoding every key is read once for a handful of queries (the groups of
// one row), so the keys' bytes bound the call: 32 KB a page at d_idx = 128
// against 128 small MMAs.  A producer warp streams pages through a ring of
// shared-memory stages by TMA; each of three consumer warps takes a whole page
// (no reduction across warps), always in the same stage, so that it sees every
// phase of that stage's barriers, and multiplies it with the queries it keeps
// in registers: a tile of 16 or 32 (row, group) pairs of one request.  The
// scale, a positive factor, is applied after the maximum.
//
// The tiles' pages, one tile after another, are cut into equal stretches for
// the two CTAs that each SM holds, whatever the requests' lengths: at four
// caches of 131,072 to 1,048,576 tokens (605 MB) 93 us, 96% of the copy rate,
// against 100 for a grid of (tile, share) CTAs.  With more rows than
// kPrefixRows, whole tiles are dealt out.
#include <limits.h>

#include <algorithm>
#include <type_traits>

#include "paged.h"
#include "tc.cuh"

namespace msa {
namespace {

using namespace tc;

constexpr int kConsumers = 3;
constexpr int kThreads = 32 * (kConsumers + 1);
constexpr int kStages = 3;
static_assert(kStages % kConsumers == 0, "a stage has one consumer");

template <int DI>
struct ScoreSmem {
    static constexpr int HALF = kPage * 128;          // 128 tokens x 64 features
    static constexpr int STAGE = HALF * (DI / 64);
    static constexpr int BYTES = kStages * STAGE + 1024;   // + alignment
};

constexpr int kPrefixRows = 512;       // most rows whose pages are cut evenly

struct PageMeta {
    int t, h0, c;      // the tile's first row and group, the block; t < 0 after the last
    int valid;
};

template <int DI, int MT>
__global__ void __launch_bounds__(kThreads, 2)
scores_kernel(PagedProblem p, const bf16 *__restrict__ q_idx, const __grid_constant__ CUtensorMap tm_k,
              const int32_t *__restrict__ block_table, const int32_t *__restrict__ q_starts,
              const int32_t *__restrict__ row_req, const int32_t *__restrict__ row_pos, float *__restrict__ scores,
              int rows_per_tile, int head_tiles, DeviceStatus *st)
{
    using S = ScoreSmem<DI>;
    constexpr int M = 16 * MT;
    extern __shared__ uint8_t raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
    __shared__ uint64_t full[kStages], empty[kStages];
    __shared__ PageMeta meta[kStages];
    __shared__ long long before[kPrefixRows + 1];      // pages of the tiles before each row's
    __shared__ int abort_flag;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const bool even = p.T <= kPrefixRows;
    chain_next();
    if (tid == 0) {
        abort_flag = 0;
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        fence_mbar_init();
    }
    chain_wait(q_idx, block_table, q_starts, row_req, row_pos);

    // the rows of the tile that row t begins (a tile is up to rows_per_tile rows of one request); 0: t begins none
    auto tile_rows = [&](int t) {
        const int req = row_req[t];
        if (req < 0) return 0;                         // a row behind the last request
        if (req >= p.R) {
            report(st, kDevCheck, 121, req);
            return 0;
        }
        const int first = q_starts[req], end = min(q_starts[req + 1], p.T);
        return t < first || t >= end || (t - first) % rows_per_tile != 0 ? 0 : min(rows_per_tile, end - t);
    };
    // pages that some row of the tile sees (positions in any order)
    auto tile_pages = [&](int t) {
        int last = row_pos[t];
        const int n = tile_rows(t);
        if (n == 0) last = -1;
        for (int u = 1; u < n; ++u) last = max(last, row_pos[t + u]);
        if (last >= 0 && last / kPage >= p.max_blocks) report(st, kDevCheck, 122, last);
        return last < 0 ? 0 : min(last / kPage + 1, p.max_blocks);
    };
    if (even)
        for (int t = tid; t < p.T; t += kThreads) before[t] = (long long)tile_pages(t) * head_tiles;
    __syncthreads();
    if (even && warp == 0) {
        long long sum = 0;
        for (int t0 = 0; t0 < p.T; t0 += 32) {
            const long long n = t0 + lane < p.T ? before[t0 + lane] : 0;
            long long inc = n;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const long long v = __shfl_up_sync(0xffffffffu, inc, d);
                if (lane >= d) inc += v;
            }
            if (t0 + lane < p.T) before[t0 + lane] = sum + inc - n;
            sum += __shfl_sync(0xffffffffu, inc, 31);
        }
        if (lane == 0) before[p.T] = sum;
    }
    __syncthreads();

    if (warp == kConsumers) {
        int step = 0, copied = 0;
        bool live = true;
        auto next = [&](const PageMeta &m, int page) {
            const int s = step % kStages;
            if (step >= kStages && !mbar_wait_warp(&empty[s], (step / kStages - 1) & 1, st, 123, &abort_flag)) {
                live = false;
                return;
            }
            if (lane == 0) {
                meta[s] = m;
                if (m.valid) {
                    mbar_arrive_expect_tx(&full[s], S::STAGE);
                    for (int h = 0; h < DI / 64; ++h)
                        tma_load_3d(smem + s * S::STAGE + h * S::HALF, &tm_k, &full[s], h * 64, 0, page);
                } else {
                    if (m.t >= 0) report(st, kDevCheck, 124, page);
                    mbar_arrive(&full[s]);
                }
            }
            ++step;
        };
        auto piece = [&](int t, int h0, int c_lo, int c_hi) {
            const int32_t *row = block_table + (long long)row_req[t] * p.max_blocks;
            for (int base = c_lo; base < c_hi && live; base += 32) {
                const int mine = base + lane < c_hi ? row[base + lane] : -1;
                for (int i = 0; i < 32 && base + i < c_hi && live; ++i) {
                    const int page = __shfl_sync(0xffffffffu, mine, i);
                    next(PageMeta{t, h0, base + i, (unsigned)page < (unsigned)p.n_pages}, page);
                }
            }
        };
        const long long me = blockIdx.x;
        if (even) {
            const long long W = before[p.T], n = gridDim.x;
            long long x = W * me / n;
            const long long x1 = W * (me + 1) / n;
            int t = 0, hi = p.T;
            while (hi - t > 1) {                       // the last row that starts at or before x
                const int mid = (t + hi) >> 1;
                if (before[mid] <= x) t = mid;
                else hi = mid;
            }
            while (x < x1 && live) {
                const long long y = x - before[t], all = before[t + 1] - before[t];
                if (y >= all) {
                    ++t;
                    continue;
                }
                const int seen = (int)(all / head_tiles), c = (int)(y % seen);
                const int m = (int)min((long long)(seen - c), x1 - x);
                piece(t, (int)(y / seen) * M, c, c + m);
                x += m;
            }
        } else {
            for (long long i = me; i < (long long)p.T * head_tiles && live; i += gridDim.x) {
                const int t = (int)(i / head_tiles), n = tile_pages(t);
                if (n) piece(t, (int)(i % head_tiles) * M, 0, n);
            }
        }
        copied = step;
        for (int i = 0; i < kConsumers && live; ++i) next(PageMeta{-1, 0, 0, 0}, -1);   // every consumer's end
        // stay until the last copies have landed (a stage with an end mark has been read)
        for (int k = max(0, step - kStages); k < copied; ++k) mbar_wait_warp(&full[k % kStages], (k / kStages) & 1, st, 125, nullptr);
        return;
    }

    // this lane's pairs of the tile: accumulator rows g and g + 8 of each 16 rows, groups fastest
    const int g = lane >> 2, q4 = lane & 3;
    uint32_t a[MT][DI / 16][4];
    int pos[MT][2], first_pos = 0, t = -1, h0 = 0;
    for (int step = warp;; step += kConsumers) {
        const int s = step % kStages;
        if (!mbar_wait_warp(&full[s], (step / kStages) & 1, st, 126, &abort_flag)) return;
        const PageMeta me = meta[s];
        if (me.t < 0) break;
        if (me.t != t || me.h0 != h0) {                // the next tile's queries
            t = me.t;
            h0 = me.h0;
            const int rows = tile_rows(t), req = row_req[t];
            first_pos = INT_MAX;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int m = mt * 16 + e * 8 + g;
                    const int tr = t + (p.Hkv >= M ? 0 : m / p.Hkv), h = p.Hkv >= M ? h0 + m : m % p.Hkv;
                    const bool ok = tr < t + rows && h < p.Hkv && row_req[min(tr, p.T - 1)] == req;
                    pos[mt][e] = ok ? row_pos[tr] : -1;
                    const uint32_t *src = reinterpret_cast<const uint32_t *>(q_idx + (ok ? ((long long)tr * p.Hkv + h) * DI : 0));
#pragma unroll
                    for (int ks = 0; ks < DI / 16; ++ks) {
                        a[mt][ks][e] = ok ? __ldg(src + ks * 8 + q4) : 0u;
                        a[mt][ks][2 + e] = ok ? __ldg(src + ks * 8 + q4 + 4) : 0u;
                    }
                    if (pos[mt][e] >= 0) first_pos = min(first_pos, pos[mt][e]);
                }
            first_pos = __reduce_min_sync(0xffffffffu, first_pos);
        }
        const int c = me.c;
        float mx[MT][2];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) mx[mt][0] = mx[mt][1] = -INFINITY;
        if (me.valid) {
            const uint8_t *sk = smem + s * S::STAGE;
            const bool whole = c * kPage + kPage - 1 <= first_pos;   // every row sees every token
#pragma unroll 2
            for (int nt = 0; nt < kPage / 8; ++nt) {
                float acc[MT][4];
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) acc[mt][0] = acc[mt][1] = acc[mt][2] = acc[mt][3] = 0.f;
                const int r = nt * 8 + (lane & 7);
#pragma unroll
                for (int kp = 0; kp < DI / 32; ++kp) {
                    uint32_t b[4];
                    const int ch = kp * 4 + (lane >> 3);
                    ldsm_x4(b[0], b[1], b[2], b[3], sk + (ch >> 3) * S::HALF + r * 128 + (((ch & 7) ^ (r & 7)) << 4));
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        mma16816(acc[mt], a[mt][kp * 2], b);
                        mma16816(acc[mt], a[mt][kp * 2 + 1], b + 2);
                    }
                }
                const int j = c * kPage + nt * 8 + 2 * q4;
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        if (whole || j <= pos[mt][e]) mx[mt][e] = fmaxf(mx[mt][e], acc[mt][2 * e]);
                        if (whole || j + 1 <= pos[mt][e]) mx[mt][e] = fmaxf(mx[mt][e], acc[mt][2 * e + 1]);
                    }
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[s]);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                mx[mt][e] = fmaxf(mx[mt][e], __shfl_xor_sync(0xffffffffu, mx[mt][e], 1));
                mx[mt][e] = fmaxf(mx[mt][e], __shfl_xor_sync(0xffffffffu, mx[mt][e], 2));
                const int m = mt * 16 + e * 8 + g;
                if (q4 == 0 && pos[mt][e] >= 0) {
                    const int tr = t + (p.Hkv >= M ? 0 : m / p.Hkv), h = p.Hkv >= M ? h0 + m : m % p.Hkv;
                    scores[((long long)tr * p.Hkv + h) * p.max_blocks + c] = mx[mt][e] * p.scale_idx;
                }
            }
    }
    // the blocks past each row's own, a warp to a (row, group)
    for (long long i = (long long)blockIdx.x * kConsumers + warp; i < (long long)p.T * p.Hkv; i += (long long)gridDim.x * kConsumers) {
        const int tr = (int)(i / p.Hkv), req = row_req[tr], ps = row_pos[tr];
        if (req < 0 || req >= p.R || ps < 0) continue;
        float *dst = scores + i * p.max_blocks;
        for (int c = min(ps / kPage + 1, p.max_blocks) + lane; c < p.max_blocks; c += 32) dst[c] = -INFINITY;
    }
}

}  // namespace

cudaError_t launch_paged_block_scores(const PagedProblem &p, const bf16 *q_idx, const bf16 *k_idx,
                                      const int32_t *block_table, const int32_t *q_starts, const int32_t *row_req,
                                      const int32_t *row_pos, float *scores, DeviceStatus *st, cudaStream_t s)
{
    // 16 pairs to a tile when a request brings one row (or its rows' groups fit), else 32
    const int avg = (p.T + p.R - 1) / p.R;
    const int M = (long long)avg * p.Hkv > 16 ? 32 : 16;
    const int rows_per_tile = std::max(1, M / p.Hkv);
    const int head_tiles = (p.Hkv + M - 1) / M;
    // two CTAs to an SM, fewer where that leaves under two pages of a full table each
    const long long most = 2LL * p.num_sms, rows = (long long)p.T * head_tiles;
    const long long ctas = p.T <= kPrefixRows ? std::min(most, (rows * p.max_blocks + 1) / 2) : std::min(most, rows);
    CUtensorMap tm;
    cudaError_t e = make_tmap_bf16_3d(&tm, k_idx, p.d_idx, kPage, p.n_pages, p.d_idx * 2ull, (unsigned long long)kPage * p.d_idx * 2, 64, kPage);
    if (e != cudaSuccess) return e;
    auto run = [&](auto dtag, auto mtag) {
        constexpr int DI = decltype(dtag)::value, MT = decltype(mtag)::value, smem = ScoreSmem<DI>::BYTES;
        static std::atomic<unsigned long long> allowed{0};
        if ((e = allow_smem(scores_kernel<DI, MT>, smem, allowed)) != cudaSuccess) return e;
        return launch_chained("paged_block_scores_kernel", scores_kernel<DI, MT>, dim3((unsigned)ctas), kThreads, smem, s, p, q_idx, tm, block_table,
                              q_starts, row_req, row_pos, scores, rows_per_tile, head_tiles, st);
    };
    using std::integral_constant;
    if (p.d_idx == 128)
        return M == 16 ? run(integral_constant<int, 128>{}, integral_constant<int, 1>{})
                       : run(integral_constant<int, 128>{}, integral_constant<int, 2>{});
    return M == 16 ? run(integral_constant<int, 64>{}, integral_constant<int, 1>{})
                   : run(integral_constant<int, 64>{}, integral_constant<int, 2>{});
}

}  // namespace msa
