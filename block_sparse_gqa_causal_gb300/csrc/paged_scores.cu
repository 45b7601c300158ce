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
// in registers, 16 or 32 (row, group) pairs to a CTA.  A CTA takes a share of
// consecutive blocks; the scale, a positive factor, is applied after the
// maximum.
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

template <int DI, int MT>
__global__ void __launch_bounds__(kThreads, 2)
scores_kernel(PagedProblem p, const bf16 *__restrict__ q_idx, const __grid_constant__ CUtensorMap tm_k,
              const int32_t *__restrict__ block_table, const int32_t *__restrict__ q_starts,
              const int32_t *__restrict__ row_req, const int32_t *__restrict__ row_pos, float *__restrict__ scores,
              int rows_per_tile, int head_tiles, int per, DeviceStatus *st)
{
    using S = ScoreSmem<DI>;
    constexpr int M = 16 * MT;
    extern __shared__ uint8_t raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
    __shared__ uint64_t full[kStages], empty[kStages];
    __shared__ int valid[kStages];
    __shared__ int abort_flag;

    chain_next();
    chain_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int t = blockIdx.x / head_tiles, h0 = blockIdx.x % head_tiles * M;
    const int req = row_req[t];
    if (req < 0) return;                               // a row behind the last request
    if (req >= p.R) {
        if (tid == 0) report(st, kDevCheck, 121, req);
        return;
    }
    // a tile is up to rows_per_tile rows of one request, owned by its first row
    const int first = q_starts[req], end = min(q_starts[req + 1], p.T);
    if ((t - first) % rows_per_tile != 0) return;
    const int nrows = max(1, min(rows_per_tile, end - t));
    const int pairs = min(M, nrows * min(p.Hkv, M));   // (row, group) pairs, groups fastest
    const int last_pos = row_pos[t + nrows - 1];
    const int c_lo = blockIdx.y * per, c_hi = min(c_lo + per, p.max_blocks);
    const int seen = last_pos < 0 ? 0 : min(last_pos / kPage + 1, p.max_blocks);
    const int n = max(0, min(c_hi, seen) - c_lo);      // pages of this share that some row sees
    if (last_pos / kPage >= p.max_blocks && tid == 0) report(st, kDevCheck, 122, last_pos);

    auto pair_row = [&](int m) { return t + (p.Hkv >= M ? 0 : m / p.Hkv); };
    auto pair_head = [&](int m) { return p.Hkv >= M ? h0 + m : m % p.Hkv; };
    auto pair_ok = [&](int m) { return m < pairs && pair_head(m) < p.Hkv; };

    if (tid == 0) {
        abort_flag = 0;
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        fence_mbar_init();
    }
    __syncthreads();

    if (warp == kConsumers) {
        const int32_t *row = block_table + (long long)req * p.max_blocks + c_lo;
        int mine = 0, i = 0;
        for (; i < n; ++i) {
            if (i % 32 == 0) mine = i + lane < n ? row[i + lane] : -1;
            const int page = __shfl_sync(0xffffffffu, mine, i % 32), s = i % kStages;
            if (i >= kStages && !mbar_wait_warp(&empty[s], (i / kStages - 1) & 1, st, 123, &abort_flag)) break;
            if (lane == 0) {
                const bool ok = (unsigned)page < (unsigned)p.n_pages;
                valid[s] = ok;
                if (ok) {
                    mbar_arrive_expect_tx(&full[s], S::STAGE);
                    for (int h = 0; h < DI / 64; ++h)
                        tma_load_3d(smem + s * S::STAGE + h * S::HALF, &tm_k, &full[s], h * 64, 0, page);
                } else {
                    report(st, kDevCheck, 124, page);
                    mbar_arrive(&full[s]);
                }
            }
        }
        // stay until the last copies have landed
        for (int k = max(0, i - kStages); k < i; ++k) mbar_wait_warp(&full[k % kStages], (k / kStages) & 1, st, 125, nullptr);
        return;
    }

    // this lane's pairs: accumulator rows g and g + 8 of each 16-row tile
    const int g = lane >> 2, q4 = lane & 3;
    uint32_t a[MT][DI / 16][4];
    int pos[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int m = mt * 16 + e * 8 + g;
            const bool ok = pair_ok(m);
            const int tr = ok ? pair_row(m) : t;
            pos[mt][e] = ok && row_req[tr] == req ? row_pos[tr] : -1;
            const uint32_t *src = reinterpret_cast<const uint32_t *>(q_idx + ((long long)tr * p.Hkv + (ok ? pair_head(m) : 0)) * DI);
#pragma unroll
            for (int ks = 0; ks < DI / 16; ++ks) {
                a[mt][ks][e] = ok ? __ldg(src + ks * 8 + q4) : 0u;
                a[mt][ks][2 + e] = ok ? __ldg(src + ks * 8 + q4 + 4) : 0u;
            }
        }
    auto store = [&](int c, const float (&mx)[MT][2]) {
        if (q4 != 0) return;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int m = mt * 16 + e * 8 + g;
                if (pos[mt][e] >= 0)
                    scores[((long long)pair_row(m) * p.Hkv + pair_head(m)) * p.max_blocks + c] = mx[mt][e] * p.scale_idx;
            }
    };
    const int first_pos = row_pos[t];
    for (int i = warp; i < n; i += kConsumers) {
        const int s = i % kStages, c = c_lo + i;
        if (!mbar_wait_warp(&full[s], (i / kStages) & 1, st, 126, &abort_flag)) return;
        float mx[MT][2];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) mx[mt][0] = mx[mt][1] = -INFINITY;
        if (valid[s]) {
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
            }
        store(c, mx);
    }
    // blocks of the share that no row of the tile sees
    const int from = max(c_lo, c_lo + n);
    for (int m = warp; m < pairs; m += kConsumers) {
        if (!pair_ok(m) || row_req[pair_row(m)] != req) continue;
        float *dst = scores + ((long long)pair_row(m) * p.Hkv + pair_head(m)) * p.max_blocks;
        for (int c = from + lane; c < c_hi; c += 32) dst[c] = -INFINITY;
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
    const long long tiles = (long long)p.T * head_tiles;
    // shares of blocks: about eight CTAs to an SM if every row filled its table, eight pages at least
    const long long busy = std::max<long long>(1, (p.T + rows_per_tile - 1) / rows_per_tile * (long long)head_tiles);
    const long long want = std::max<long long>(1, 8LL * p.num_sms / busy);
    const int per = (int)std::max<long long>(8, (p.max_blocks + want - 1) / want);
    const dim3 grid((unsigned)tiles, (p.max_blocks + per - 1) / per);
    CUtensorMap tm;
    cudaError_t e = make_tmap_bf16_3d(&tm, k_idx, p.d_idx, kPage, p.n_pages, p.d_idx * 2ull, (unsigned long long)kPage * p.d_idx * 2, 64, kPage);
    if (e != cudaSuccess) return e;
    auto run = [&](auto dtag, auto mtag) {
        constexpr int DI = decltype(dtag)::value, MT = decltype(mtag)::value, smem = ScoreSmem<DI>::BYTES;
        static std::atomic<unsigned long long> allowed{0};
        if ((e = allow_smem(scores_kernel<DI, MT>, smem, allowed)) != cudaSuccess) return e;
        return launch_chained("paged_block_scores_kernel", scores_kernel<DI, MT>, grid, kThreads, smem, s, p, q_idx, tm, block_table,
                              q_starts, row_req, row_pos, scores, rows_per_tile, head_tiles, per, st);
    };
    using std::integral_constant;
    if (p.d_idx == 128)
        return M == 16 ? run(integral_constant<int, 128>{}, integral_constant<int, 1>{})
                       : run(integral_constant<int, 128>{}, integral_constant<int, 2>{});
    return M == 16 ? run(integral_constant<int, 64>{}, integral_constant<int, 1>{})
                   : run(integral_constant<int, 64>{}, integral_constant<int, 2>{});
}

}  // namespace msa
