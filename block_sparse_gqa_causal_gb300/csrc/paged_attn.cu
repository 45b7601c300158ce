// paged_attn.cu -- attention of a ragged batch over a paged cache whose K and
// V are e4m3 with one scale per (page, KV head): for row t and head h of
// group r, over the tokens j <= pos(t) of the blocks selected for (t, r) (or
// of every block),
//   l_j = scale * ks * <q, k_j>,  P = softmax(l),  o = sum_j P_j vs v_j,
//   lse = log sum_j exp(l_j).
//
// Decoding reads every selected page once for the G <= 8 heads of a group, so
// the pages' bytes bound it; what has to be kept away is the conversion of
// each code to 16 bits.  The codes therefore go to the tensor cores as they
// are (e4m3 x e4m3, fp32 sums).  A 16-row MMA tile has room for twice the
// group's heads, so the other operand is split in two e4m3 terms: rows 0-7
// hold the heads' leading terms hi = rn(x), rows 8-15 lo = rn(16 (x - hi)),
// and hi + lo / 16 carries the 8 significant bits of a bf16 query exactly,
// down to 2^-23 of the row's largest feature (rows are scaled by a power of
// two to fill the range), and the probabilities with the precision that bf16
// gives them.  Sums, maxima and the outputs are fp32.
//
// With t_j = l_j log2 e + log2 vs, the weight of token j's codes is 2^t_j and
// that of the sum 2^t_j / vs, so one reference m bounds both and the products
// P V add up in the MMA's own accumulators across pages of different scales.
// m is the largest t so far, or up to 4 less: P = 16 * 2^(t - m) stays within
// 256 and the accumulators are only rescaled when t has outgrown m by more
// than that, which after a row's first pages is rare.  (Rescaling on every
// new maximum and joining each page's product in fp32 cost 830 instructions a
// warp and page instead of 300, and made them the bound: 55 us against 45 at
// 64 rows x 8 groups x 16 pages.)  P's small terms are off by at most 2^-18
// of the largest weight.
//
// Each of four warps takes 32 of a page's 128 tokens and keeps its own running
// maximum, sum and output; they are joined where a row ends.  V's operand
// needs its tokens along a register: ldmatrix with 8-bit transposition gives
// that from the row-major tile.  The tokens' order inside a 32-token step is
// chosen so that a lane's scores are the probabilities it has to feed back and
// no shared-memory phase has a bank conflict.
//
// The work is one long list of blocks, those of (row 0, group 0), then (row 0,
// group 1) and so on, cut into equal stretches for the two CTAs that each SM
// holds.  So every CTA reads the same number of pages whatever the rows'
// lengths, and a producer warp streams the stretch through one ring of stages
// (K and V tiles of a page and head, contiguous and swizzled by TMA) without a
// pause where a row ends and the next begins.  A stretch cuts at most two
// rows; those pieces' states go to the workspace, and the CTA that ends the
// last piece of a row joins them, in their order along the row.  (A second
// kernel for that took 6 us more a call.)
#include <algorithm>
#include <type_traits>

#include "paged.h"
#include "tc.cuh"

namespace msa {
namespace {

using namespace tc;

constexpr int kWarps = 4;                       // consumer warps, 32 tokens of a page each
constexpr int kThreads = 32 * (kWarps + 1);
constexpr int kStages = 3;

constexpr int kPrefixRows = 512;                // most rows whose blocks are cut evenly; above, whole rows are dealt out
constexpr int kMinBlocks = 2;                   // a stretch has at least this many blocks
constexpr int kArrivedWords = (4096 - kStatusBytes) / 4;   // the workspace's counts, one to a stretch
constexpr int kWholeBlocks = 4;                 // rows of up to so many blocks are not cut

enum { kFirst = 1, kLast = 2, kEnd = 4 };       // of a piece; of the CTA's stretch
struct Meta {
    int len;        // visible tokens of the block
    float ks;       // the page's K scale for this head
    float lv, pv;   // log2 of its V scale (-100 at least), and 16 x what that leaves of the scale (1)
    int flags;
    int t, r;       // the piece's row and group
    int part;       // the piece's place among the partial states; -1: a whole row
    int first, n;   // a cut row's first stretch and the number of its pieces
};

template <int D>
struct AttnSmem {
    static constexpr int TILE = kPage * D;      // K or V codes of a page and head
    static constexpr int STAGE = 2 * TILE;
    static constexpr int Q = 8 * D * 2;         // the group's queries, with a piece's first block
    static constexpr int OFF_Q = kStages * STAGE;
    static constexpr int BYTES = OFF_Q + kStages * Q + 1024;   // + alignment
    static constexpr int OROW = D + 8;          // a warp's output row: 8 more keeps the rows on different banks
    static_assert(kWarps * 8 * OROW * 4 <= STAGE, "the warps' outputs fit a stage");
};

// byte offset of 16-byte word w of token row r in a TMA-swizzled tile
template <int D>
__device__ __forceinline__ int at(int r, int w)
{
    return D == 128 ? r * 128 + ((w ^ (r & 7)) << 4) : r * 64 + ((w ^ ((r >> 1) & 3)) << 4);
}

// D(16x8, f32) += A(16x32, e4m3, row) * B(32x8, e4m3, col)
__device__ __forceinline__ void mma_e4m3(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two 16x16 byte matrices, transposed: lane l gives the address of row l % 16
// of matrix l / 16; it gets, for columns l/4 and l/4 + 8, rows 4(l%4)..+3 of
// the first matrix (r0, r1) and of the second (r2, r3).
__device__ __forceinline__ void ldsm_b8_t(uint32_t (&r)[4], const void *p)
{
    asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(smem_u32(p)));
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float2 from_e4m3x2(uint32_t two)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;\n" : "=r"(h) : "h"((uint16_t)two));
    return __half22float2(*reinterpret_cast<__half2 *>(&h));
}
// x = hi + lo / 16 for four values within +-448
__device__ __forceinline__ void split4(float x0, float x1, float x2, float x3, uint32_t &hi, uint32_t &lo)
{
    const uint32_t h01 = e4m3x2(x0, x1), h23 = e4m3x2(x2, x3);
    const float2 f01 = from_e4m3x2(h01), f23 = from_e4m3x2(h23);
    hi = h01 | (h23 << 16);
    lo = e4m3x2(16.f * (x0 - f01.x), 16.f * (x1 - f01.y)) | (e4m3x2(16.f * (x2 - f23.x), 16.f * (x3 - f23.y)) << 16);
}

MSA_DEV void mbar_expect_tx(uint64_t *bar, uint32_t bytes)
{
    asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;\n" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}
MSA_DEV void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

template <int D>
__global__ void __launch_bounds__(kThreads, 2)
attn_kernel(PagedProblem p, const bf16 *__restrict__ q, const __grid_constant__ CUtensorMap tm_k,
            const __grid_constant__ CUtensorMap tm_v, const float *__restrict__ k_scale,
            const float *__restrict__ v_scale, const int32_t *__restrict__ block_table,
            const int32_t *__restrict__ row_req, const int32_t *__restrict__ row_pos, const int32_t *__restrict__ sel,
            bf16 *__restrict__ o, float *__restrict__ lse, float *__restrict__ part_o, float2 *__restrict__ part_ml,
            unsigned *__restrict__ arrived, DeviceStatus *st)
{
    using S = AttnSmem<D>;
    extern __shared__ uint8_t raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
    __shared__ uint64_t full[kStages], empty[kStages];
    __shared__ Meta meta[kStages];
    __shared__ float sM[kWarps][8], sL[kWarps][8];
    __shared__ long long before[kPrefixRows + 1];   // blocks of the rows before each row, one group
    __shared__ int abort_flag, joins;

    chain_next();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, G = p.G;
    const bool even = arrived != nullptr;         // stretches of equal length; else whole rows are dealt out

    // blocks that a group of row t has to look at; 0: not a row (entries of a selection may sit in any of its slots)
    auto blocks_of = [&](int t, int &req, int &pos) {
        req = row_req[t];
        pos = row_pos[t];
        if (req < 0 || pos < 0) return 0;              // behind the last request
        if (req >= p.R || pos / kPage >= p.max_blocks) {
            report(st, kDevCheck, 141, req >= p.R ? req : pos);
            return 0;
        }
        return sel ? p.topk : pos / kPage + 1;
    };
    if (tid == 0) {
        abort_flag = 0;
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], kWarps);
        }
        fence_mbar_init();
    }
    chain_wait();
    if (even)
        for (int t = tid; t < p.T; t += kThreads) {
            int req, pos;
            before[t] = blocks_of(t, req, pos);
        }
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

    if (warp == kWarps) {
        int step = 0;
        bool live = true;
        // Waits for the next stage and starts its copies.  The arrival that completes the phase comes with the
        // block's Meta, so that the copies do not wait for the scales.
        auto start = [&](int page, int t, int r, int len, bool first) {
            const int s = step % kStages;
            if (step >= kStages && !mbar_wait_warp(&empty[s], (step / kStages - 1) & 1, st, 144, &abort_flag)) {
                live = false;
                return;
            }
            if (lane == 0) {
                const int boxes = (len + 31) / 32;             // 32-token boxes, none past the row
                const uint32_t qb = first ? G * D * 2 : 0;
                mbar_expect_tx(&full[s], boxes * 64 * D + qb);
                if (first) bulk_load(smem + S::OFF_Q + s * S::Q, q + ((long long)t * p.Hq + (long long)r * G) * D, qb, &full[s]);
                uint8_t *dst = smem + s * S::STAGE;
                for (int x = 0; x < boxes; ++x)
                    tma_load_3d(dst + x * 32 * D, &tm_k, &full[s], 0, x * 32, page * p.Hkv + r);
                for (int x = 0; x < boxes; ++x)
                    tma_load_3d(dst + S::TILE + x * 32 * D, &tm_v, &full[s], 0, x * 32, page * p.Hkv + r);
            }
        };
        auto publish = [&](const Meta &m) {
            const int s = step % kStages;
            if (lane == 0) {
                meta[s] = m;
                mbar_arrive(&full[s]);
            }
            ++step;
        };
        // blocks (a selection: slots) j0 .. j1 - 1 of group r of row t
        auto piece = [&](int t, int r, int req, int pos, int j0, int j1, int part, int first_cut, int n_cut) {
            const int c0 = pos / kPage;
            for (int base = j0; base < j1 && live; base += 32) {
                int c = -1;
                if (sel) {
                    // selected blocks ascend; an entry that does not, or lies past the row's own block, is no block
                    c = lane < p.topk ? sel[((long long)t * p.Hkv + r) * p.topk + lane] : -1;
                    int most = c;
#pragma unroll
                    for (int d = 1; d < 32; d <<= 1) {
                        const int v = __shfl_up_sync(0xffffffffu, most, d);
                        if (lane >= d) most = max(most, v);
                    }
                    most = __shfl_up_sync(0xffffffffu, most, 1);
                    if (c >= 0 && (c > c0 || (lane > 0 && c <= most))) {
                        report(st, kDevCheck, 142, c);
                        c = -1;
                    }
                    if (lane < j0 || lane >= j1) c = -1;
                } else if (base + lane < j1) {
                    c = base + lane;
                }
                int page = -1, len = 0;
                float ks = 0.f, vscale = 0.f;
                if (c >= 0) {
                    page = block_table[(long long)req * p.max_blocks + c];
                    if ((unsigned)page >= (unsigned)p.n_pages) {
                        report(st, kDevCheck, 143, page);
                    } else {
                        len = min(kPage, pos - c * kPage + 1);
                        ks = k_scale[(long long)page * p.Hkv + r];
                        vscale = v_scale[(long long)page * p.Hkv + r];
                    }
                }
                // a block without a page is an empty step, and so is a piece without any block
                unsigned todo = __ballot_sync(0xffffffffu, c >= 0);
                if (sel && !todo) todo = 1;
                bool first = base == j0;
                while (todo && live) {
                    const int l = __ffs(todo) - 1;
                    todo &= todo - 1;
                    const int blen = __shfl_sync(0xffffffffu, len, l);
                    start(__shfl_sync(0xffffffffu, page, l), t, r, blen, first);
                    if (!live) break;
                    Meta m;
                    m.len = blen;
                    m.ks = __shfl_sync(0xffffffffu, ks, l);
                    const float vs = __shfl_sync(0xffffffffu, vscale, l);
                    m.lv = fmaxf(log2f(vs), -100.f);
                    m.pv = 16.f * (vs * exp2f(-m.lv));
                    m.flags = (first ? kFirst : 0) | (!todo && (sel || base + 32 >= j1) ? kLast : 0);
                    m.t = t;
                    m.r = r;
                    m.part = part;
                    m.first = first_cut;
                    m.n = n_cut;
                    first = false;
                    publish(m);
                }
                if (sel) break;                        // at most 32 slots: one round
            }
        };
        const int me = blockIdx.x;
        if (even) {
            const long long W = before[p.T] * p.Hkv;
            const long long n = max(1LL, min((long long)gridDim.x, W / kMinBlocks));
            long long x = me < n ? W * me / n : 0;
            const long long x1 = me < n ? W * (me + 1) / n : 0;
            auto holder = [&](long long y) { return (int)(((y + 1) * n + W - 1) / W - 1); };   // the stretch that has block y
            int t = 0;
            if (x < x1) {                              // the last row that starts at or before x
                int hi = p.T;
                while (hi - t > 1) {
                    const int mid = (t + hi) >> 1;
                    if (before[mid] * p.Hkv <= x) t = mid;
                    else hi = mid;
                }
            }
            while (x < x1 && live) {
                const int nt = (int)(before[t + 1] - before[t]);
                const long long y = x - before[t] * p.Hkv;
                if (y >= (long long)nt * p.Hkv) {
                    ++t;
                    continue;
                }
                const int r = (int)(y / nt), j0 = (int)(y % nt), j1 = (int)min((long long)nt, j0 + (x1 - x));
                const bool whole = j0 == 0 && j1 == nt;
                const int f = whole ? 0 : holder(x - j0), last = whole ? 0 : holder(x - j0 + nt - 1);
                piece(t, r, row_req[t], row_pos[t], j0, j1, whole ? -1 : 2 * me + (j0 > 0 ? 0 : 1), f, last - f + 1);
                x += j1 - j0;
            }
        } else {
            const long long pairs = (long long)p.T * p.Hkv;
            for (long long i = me; i < pairs && live; i += gridDim.x) {
                int req, pos;
                const int t = (int)(i / p.Hkv), nt = blocks_of(t, req, pos);
                if (nt) piece(t, (int)(i % p.Hkv), req, pos, 0, nt, -1, 0, 0);
            }
        }
        const int copied = step;
        if (live) {
            const int s = step % kStages;
            if (step < kStages || mbar_wait_warp(&empty[s], (step / kStages - 1) & 1, st, 144, &abort_flag)) {
                if (lane == 0) {
                    meta[s].flags = kEnd;
                    meta[s].len = 0;
                    mbar_arrive(&full[s]);
                }
                ++step;
            }
        }
        // stay until the last copies have landed (the stage of the end mark has been read)
        for (int k = max(0, step - kStages); k < copied; ++k) mbar_wait_warp(&full[k % kStages], (k / kStages) & 1, st, 145, nullptr);
        return;
    }

    const int g = lane >> 2, t4 = lane & 3;
    float acc[D / 8][4];                               // head g, features 8n + 2 t4, + 1: the hi rows' sums, then the lo rows'
    float m_run = -INFINITY, l_run = 0.f, sql = 0.f;   // reference of head g; this lane's share of its sum
    uint32_t a[D / 32][4];                             // the queries' terms, features 32 ks + 4 t4 .. + 3 and + 16 ..
    const int kw = warp * 32;                          // this warp's first token of a page
    // K rows: token column j of score tile n is token 8n + (j ^ 4 (n & 1))
    const int kj = lane & 7, km = lane >> 3;
    // V rows: probability k (of 16) is lane (k / 4)'s value e = k & 1 of tile (k / 2) & 1
    const int vk = lane & 15, vn = (vk >> 1) & 1;
    const int vrow = kw + 16 * (lane >> 4) + 8 * vn + ((2 * (vk >> 2) + (vk & 1)) ^ (4 * vn));
#pragma unroll
    for (int n = 0; n < D / 8; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
#pragma unroll
    for (int ks = 0; ks < D / 32; ++ks) a[ks][0] = a[ks][1] = a[ks][2] = a[ks][3] = 0u;

    for (int step = 0;; ++step) {
        const int s = step % kStages;
        if (!mbar_wait_warp(&full[s], (step / kStages) & 1, st, 146, &abort_flag)) return;
        const Meta me = meta[s];
        if (me.flags & kEnd) return;
        if (me.flags & kFirst) {
            const bool ok = g < G;
            const uint2 *src = reinterpret_cast<const uint2 *>(smem + S::OFF_Q + s * S::Q + (ok ? g : 0) * D * 2);
            uint2 x[D / 32][2];
            uint32_t top = 0;
#pragma unroll
            for (int ks = 0; ks < D / 32; ++ks)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    x[ks][e] = ok ? src[ks * 8 + e * 4 + t4] : make_uint2(0u, 0u);
                    top = __vmaxu2(top, __vmaxu2(x[ks][e].x & 0x7FFF7FFFu, x[ks][e].y & 0x7FFF7FFFu));
                }
            top = max(top & 0xFFFFu, top >> 16);
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // not finite: NaN, and so are the scores
            const float sq = __uint_as_float(top >= 0x7F80u ? 0x7FC00000u : pow2_scale_bits(top));
            const float inv = 1.f / sq;
#pragma unroll
            for (int ks = 0; ks < D / 32; ++ks)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float2 u = unpack_bf16(x[ks][e].x), v = unpack_bf16(x[ks][e].y);
                    split4(u.x * inv, u.y * inv, v.x * inv, v.y * inv, a[ks][2 * e], a[ks][2 * e + 1]);
                }
            sql = sq * (p.scale * kLog2e);
#pragma unroll
            for (int n = 0; n < D / 8; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
            m_run = -INFINITY;
            l_run = 0.f;
        }
        if (kw < me.len) {
            uint8_t *sk = smem + s * S::STAGE, *sv = sk + S::TILE;
            if (me.len < kw + 32) {
                // rows behind the last visible token: whatever they hold must not reach 0 * V
                for (int x = lane; x < (kw + 32 - me.len) * (D / 16); x += 32)
                    reinterpret_cast<uint4 *>(sv + me.len * D)[x] = make_uint4(0u, 0u, 0u, 0u);
                fence_proxy_async();
                __syncwarp();
            }
            float sc[4][2];
            const float fac = sql * me.ks;
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                float c[4] = {0.f, 0.f, 0.f, 0.f};
                const int row = kw + 8 * n + (kj ^ (4 * (n & 1)));
#pragma unroll
                for (int kp = 0; kp < D / 64; ++kp) {
                    uint32_t b[4];
                    ldsm_x4(b[0], b[1], b[2], b[3], sk + at<D>(row, 4 * kp + km));
                    mma_e4m3(c, a[2 * kp], b[0], b[1]);
                    mma_e4m3(c, a[2 * kp + 1], b[2], b[3]);
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) sc[n][e] = fmaf(fmaf(c[2 + e], 0.0625f, c[e]), fac, me.lv);
            }
            if (me.len < kw + 32) {
#pragma unroll
                for (int n = 0; n < 4; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        if (kw + 8 * n + ((2 * t4 + e) ^ (4 * (n & 1))) >= me.len) sc[n][e] = -INFINITY;
            }
            float mx = fmaxf(fmaxf(fmaxf(sc[0][0], sc[0][1]), fmaxf(sc[1][0], sc[1][1])),
                             fmaxf(fmaxf(sc[2][0], sc[2][1]), fmaxf(sc[3][0], sc[3][1])));
            if (__any_sync(0xffffffffu, mx > m_run + 4.f)) {
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                const float m_new = fmaxf(m_run, mx);
                const float alpha = m_new == m_run ? 1.f : exp2f(m_run - m_new);
                m_run = m_new;
                l_run *= alpha;
#pragma unroll
                for (int n = 0; n < D / 8; ++n) {
                    acc[n][0] *= alpha;
                    acc[n][1] *= alpha;
                    acc[n][2] *= alpha;
                    acc[n][3] *= alpha;
                }
            }
            const float m_use = m_run == -INFINITY ? 0.f : m_run;   // no score yet but -inf (or NaN)
            float ps = 0.f;
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    sc[n][e] = exp2f(sc[n][e] - m_use);
                    ps += sc[n][e];
                    sc[n][e] *= me.pv;
                }
            l_run = fmaf(ps, exp2f(-me.lv), l_run);
            uint32_t pa[4];
            split4(sc[0][0], sc[0][1], sc[1][0], sc[1][1], pa[0], pa[1]);
            split4(sc[2][0], sc[2][1], sc[3][0], sc[3][1], pa[2], pa[3]);
#pragma unroll
            for (int w = 0; w < D / 16; ++w) {
                uint32_t b[4];
                ldsm_b8_t(b, sv + at<D>(vrow, w));
                mma_e4m3(acc[2 * w], pa, b[0], b[2]);
                mma_e4m3(acc[2 * w + 1], pa, b[1], b[3]);
            }
        }
        if (!(me.flags & kLast)) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[s]);
            continue;
        }

        // join the warps' states, in order; once all four have read it, the last block's stage takes the outputs
        l_run += __shfl_xor_sync(0xffffffffu, l_run, 1);
        l_run += __shfl_xor_sync(0xffffffffu, l_run, 2);
        if (t4 == 0) {
            sM[warp][g] = m_run;
            sL[warp][g] = l_run;
        }
        named_bar_sync(1, 32 * kWarps);
        float M = -INFINITY, L = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sM[w][g]);
#pragma unroll
        for (int w = 0; w < kWarps; ++w)               // an empty state is all zeros, one of NaN scores NaN
            L += (sM[w][g] == -INFINITY ? 1.f : exp2f(sM[w][g] - M)) * sL[w][g];
        const float f = m_run == -INFINITY ? 1.f : exp2f(m_run - M);
        const bool whole = me.part < 0;
        const float z = (whole ? (L == 0.f ? 0.f : f / L) : f) * 0.0625f;   // P carries 16
        float *sO = reinterpret_cast<float *>(smem + s * S::STAGE);
        const long long row = (long long)me.t * p.Hq + (long long)me.r * G;
        if (g < G) {
#pragma unroll
            for (int n = 0; n < D / 8; ++n)
                *reinterpret_cast<float2 *>(sO + (warp * 8 + g) * S::OROW + n * 8 + 2 * t4) =
                    make_float2(fmaf(acc[n][2], 0.0625f, acc[n][0]) * z, fmaf(acc[n][3], 0.0625f, acc[n][1]) * z);
            if (warp == 0 && t4 == 0) {
                if (whole) lse[row + g] = (M + log2f(L)) * kLn2;
                else part_ml[me.part * 8 + g] = make_float2(M, L);
            }
        }
        named_bar_sync(1, 32 * kWarps);
        for (int idx = tid * 4; idx < G * D; idx += 32 * kWarps * 4) {
            const float *src = sO + idx / D * S::OROW + idx % D;
            float4 v = *reinterpret_cast<const float4 *>(src);
#pragma unroll
            for (int w = 1; w < kWarps; ++w) {
                const float4 u = *reinterpret_cast<const float4 *>(src + w * 8 * S::OROW);
                v = make_float4(v.x + u.x, v.y + u.y, v.z + u.z, v.w + u.w);
            }
            if (whole) *reinterpret_cast<uint2 *>(o + row * D + idx) = make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
            else *reinterpret_cast<float4 *>(part_o + (long long)me.part * 8 * D + idx) = v;
        }
        if (!whole) __threadfence();                   // the state before the arrival
        fence_proxy_async();                           // the stage goes back to the copies
        named_bar_sync(1, 32 * kWarps);                // sM and sL are free again, too
        if (lane == 0) mbar_arrive(&empty[s]);
        if (whole) continue;

        // the last arrival of a cut row joins its pieces (and leaves the count at zero)
        if (tid == 0) joins = atomicInc(&arrived[me.first], me.n - 1) == (unsigned)(me.n - 1);
        named_bar_sync(1, 32 * kWarps);
        if (!joins) continue;
        __threadfence();
        for (int idx = tid * 4; idx < G * D; idx += 32 * kWarps * 4) {
            constexpr int U = 4;                       // pieces whose loads are in flight together
            const int h = idx / D;
            float Mj = -INFINITY, Lj = 0.f;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int i0 = 0; i0 < me.n; i0 += U) {
                float2 ml[U];
                float4 v[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int i = min(i0 + u, me.n - 1);
                    const long long part = 2 * (me.first + i) + (i == 0 ? 1 : 0);
                    ml[u] = __ldcg(part_ml + part * 8 + h);
                    v[u] = __ldcg(reinterpret_cast<const float4 *>(part_o + part * 8 * D + idx));
                }
                float m = Mj;
#pragma unroll
                for (int u = 0; u < U; ++u) m = fmaxf(m, ml[u].x);
                const float keep = Mj == -INFINITY ? 1.f : exp2f(Mj - m);
                Mj = m;
                Lj *= keep;
                x = make_float4(x.x * keep, x.y * keep, x.z * keep, x.w * keep);
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (i0 + u >= me.n) break;
                    const float w = ml[u].x == -INFINITY ? 1.f : exp2f(ml[u].x - Mj);
                    Lj += w * ml[u].y;
                    x = make_float4(fmaf(w, v[u].x, x.x), fmaf(w, v[u].y, x.y), fmaf(w, v[u].z, x.z), fmaf(w, v[u].w, x.w));
                }
            }
            const float inv = Lj == 0.f ? 0.f : 1.f / Lj;
            *reinterpret_cast<uint2 *>(o + row * D + idx) = make_uint2(pack_bf16(x.x * inv, x.y * inv), pack_bf16(x.z * inv, x.w * inv));
            if (idx % D == 0) lse[row + h] = (Mj + log2f(Lj)) * kLn2;
        }
    }
}

// Whether rows are cut into equal stretches.  Not with many rows (the list is
// summed up by every CTA) or short ones, where joining costs what cutting saves.
bool cuts_rows(const PagedProblem &p, bool sparse)
{
    return p.T <= kPrefixRows && (sparse ? p.topk : p.max_blocks) > kWholeBlocks;
}
// Two CTAs to an SM, fewer where that leaves stretches under kMinBlocks.
int attn_ctas(const PagedProblem &p, bool sparse)
{
    const long long rows = (long long)p.T * p.Hkv, most = std::min(2 * p.num_sms, kArrivedWords);
    return (int)std::min(most, cuts_rows(p, sparse) ? rows * (sparse ? p.topk : p.max_blocks) / kMinBlocks : rows);
}

}  // namespace

size_t paged_attn_scratch_floats(const PagedProblem &p)
{
    if (!cuts_rows(p, true) && !cuts_rows(p, false)) return 0;
    return kArrivedWords + (size_t)2 * p.num_sms * 2 * 8 * (p.d + 2);
}

cudaError_t launch_paged_attn(const PagedProblem &p, const bf16 *q, const uint8_t *k8, const uint8_t *v8,
                              const float *k_scale, const float *v_scale, const int32_t *block_table,
                              const int32_t *row_req, const int32_t *row_pos, const int32_t *sel, bf16 *o, float *lse,
                              float *scratch, DeviceStatus *st, cudaStream_t s)
{
    const int ctas = attn_ctas(p, sel != nullptr);
    // one count per stretch, zero between calls, then the partial outputs and (reference, sum) pairs
    unsigned *arrived = cuts_rows(p, sel != nullptr) ? reinterpret_cast<unsigned *>(scratch) : nullptr;
    float *part_o = scratch + kArrivedWords;
    float2 *part_ml = reinterpret_cast<float2 *>(part_o + (size_t)2 * p.num_sms * 2 * 8 * p.d);
    CUtensorMap tk, tv;
    cudaError_t e = make_tmap_u8_3d(&tk, k8, p.d, kPage, (unsigned long long)p.n_pages * p.Hkv, p.d, 32);
    if (e == cudaSuccess) e = make_tmap_u8_3d(&tv, v8, p.d, kPage, (unsigned long long)p.n_pages * p.Hkv, p.d, 32);
    if (e != cudaSuccess) return e;
    auto run = [&](auto dtag) {
        constexpr int D = decltype(dtag)::value;
        static std::atomic<unsigned long long> allowed{0};
        if ((e = allow_smem(attn_kernel<D>, AttnSmem<D>::BYTES, allowed)) != cudaSuccess) return e;
        return launch_chained("paged_attn_kernel", attn_kernel<D>, dim3(ctas), kThreads, AttnSmem<D>::BYTES, s, p, q, tk, tv,
                              k_scale, v_scale, block_table, row_req, row_pos, sel, o, lse, part_o, part_ml, arrived, st);
    };
    return p.d == 128 ? run(std::integral_constant<int, 128>{}) : run(std::integral_constant<int, 64>{});
}

}  // namespace msa
