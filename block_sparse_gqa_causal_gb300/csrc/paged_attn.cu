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
// are (tcgen05, e4m3 x e4m3, fp32 sums in TMEM), tokens or features as the 128
// rows of a product and the heads as its 16 columns:
//   S [token][16] = K [token][d] Q~ [16][d]^T,  O [feature][16] += V [token][feature]^T P~ [16][token]^T.
// Sixteen columns are twice the heads, so the other operand is split in two
// e4m3 terms: columns 0-7 hold the heads' leading terms hi = rn(x), columns
// 8-15 lo = rn(16 (x - hi)), and hi + lo / 16 carries the 8 significant bits
// of a bf16 query exactly, features below 2^-14 of the row's largest to 2^-22
// of it (queries are scaled by a power of two to fill the range).  (mma.sync
// takes e4m3 too, but at 19.6 cycles a warp and SM quarter against 7.9 for the
// 16-bit MMA of half its depth, which held the pages back.)
//
// With t_j = l_j log2 e + log2 vs, the weight of token j's codes is 2^t_j and
// that of the sum 2^t_j / vs, so one reference m per head bounds both and the
// products P V add up in TMEM across pages of different scales.  m is the
// largest t so far, or up to kLag = 3 less: P = 32 * 2^(t - m) stays within 256
// and the sums are only rescaled when t has outgrown m by more than that, which
// after a row's first page is rare.
//
// Two terms hold P = hi + lo / 32 to 8 significant bits from 256 down to 2^-7,
// 12 binades below the reference.  That is not enough: thousands of tokens under
// an attention sink weigh less than that each and more than the sink together.
// So there are three levels, 2^15 apart, each with an O of its own in TMEM; a
// probability has its terms in the level where it keeps its 8 bits and zeros in
// the others, and the levels are joined when a row's outputs are written.  8 bits
// are kept down to 2^-42 of the reference; a token below is off by 2^-50 of it.
// A lower level's product is issued for those 32 tokens only (a warp's, a step of
// the MMA) that have any there: near-uniform rows pay a vote, and under a sink
// the dense case below takes 188 us instead of 184.  A page's probabilities take
// the place of its K tile once its scores are there.
//
// The work is one long list of blocks, those of (row 0, group 0), then (row 0,
// group 1) and so on, each group's led by kPieceCost that stands for what it
// costs besides, cut into equal stretches for the two CTAs that each SM holds,
// whatever the rows' lengths.  A planner warp walks the stretch a row ahead
// (row, selection and block table are dependent loads, 2 us that would empty
// the ring at every row) and lays down each row's queries; a producer warp
// streams the pages through one ring of stages (K and V tiles of a page and
// head, contiguous and swizzled by TMA); one warp issues the MMAs, the next
// page's S before this page's P V; four warps, a token to a thread, turn scores
// into probabilities.  A stretch cuts at most two rows; those pieces' states go
// to the workspace, and the CTA that ends the last piece of a row joins them,
// in their order along the row (more than kOneGo by eights: one request of
// 65,536 tokens attending to everything, 38 pieces a row, 40 us in one go, 34
// so).
//
// At 64 rows x 8 groups x 16 blocks of d = 128 (264 MB) 54 us: it streams at
// the copy rate for 40, the first page is there after 6, and the last CTA ends
// 4 to 5 after the median one.  Every block of eight requests of up to 131,072
// tokens (1.2 GB): 183 us, 97% of the copy rate.
#include <algorithm>
#include <type_traits>

#include "paged.h"
#include "tc.cuh"

namespace msa {
namespace {

using namespace tc;

constexpr int kWarps = 4;                       // softmax warps, a token of the page to a thread
constexpr int kThreads = 32 * (kWarps + 3);     // then the producer, the MMA and the planner warp
constexpr int kStages = 3;
constexpr int kQueries = 4;                     // pieces whose queries are held
constexpr int kLevels = 3;                      // magnitudes of probabilities that are summed up apart
constexpr float kLag = 3.f;                     // log2 of what a probability may outgrow its reference by
constexpr float kOne = 32.f;                    // what the reference's probability is held as: all up to 2^kLag times that
constexpr float kLo = 32.f;                     // scale of the low term: the high one is off by 8 at most (up to 256)
constexpr float kLevelEnd = 1.f / 128;          // the least value of a level: there its two terms' 8 bits end
constexpr float kLevelStep = 1 << 15;           // from one level's end to the next one's
constexpr int kO = 32;                          // TMEM: two S buffers, then a level's O behind the other, 16 columns each
constexpr int kColumns = 128;
static_assert(kO + kLevels * 16 <= kColumns, "TMEM columns");
constexpr int kPrefixRows = 384;                // most rows whose blocks are cut evenly; above, whole rows are dealt out
constexpr int kMinBlocks = 2;                   // a stretch has at least this many blocks
// The workspace's counts, three to a stretch: of the row that it cuts off, of eight pieces from it on that another
// stretch's row has, and of the first eight of its own.
constexpr int kArrivedWords = (kHeadBytes - kStatusBytes) / 4;
constexpr int kMostCtas = kArrivedWords / 3;
constexpr int kOneGo = 16;                      // pieces of a row that are joined in one go
// What a group of a row costs next to its blocks, in blocks (its queries, its outputs): 64 rows of up to 8 blocks x 8
// groups 34 us without, 27 so.  Left out where a stretch would not get kMinBlocks without it.
constexpr int kPieceCost = 1;
constexpr int kCountShift = 48;                 // before[]: blocks below, rows that have any above
constexpr int kWholeBlocks = 4;                 // rows of up to so many blocks are not cut

enum { kFirst = 1, kLast = 2, kEnd = 4 };       // of a piece; of the CTA's stretch
struct Meta {
    int len;        // visible tokens of the block
    float ks;       // the page's K scale for this head
    float lv, il, pv;   // log2 of its V scale (-100 at least), 2^-lv, and kOne x what lv leaves of the scale (1)
    int flags;
    int t, r, q;    // the piece's row and group, and its number in the stretch
    int part;       // the piece's place among the partial states; -1: a whole row
    int first, n;   // a cut row's first stretch and the number of its pieces
};

// Up to 32 blocks of a piece, from the planner to the producer.
struct Chunk {
    int flags, t, r, q, part, first, n;
    unsigned blocks;               // which entries are blocks
    int page[32], len[32];         // len 0: no such page
};

template <int D>
struct AttnSmem {
    static constexpr int TILE = kPage * D;      // K or V codes of a page and head
    static constexpr int STAGE = 2 * TILE;
    static constexpr int Q = 16 * D;            // a row's queries: hi and lo terms of 8 heads
    static constexpr int P = 16 * kPage;        // a page's probabilities, 16 bytes (hi and lo of 8 heads) to a token
    static constexpr int OFF_Q = kStages * STAGE;
    static constexpr int BYTES = OFF_Q + kQueries * Q;
    // a page's probabilities, a level behind the other, in its K tile
    static_assert(kLevels * P <= TILE, "probabilities outgrow a K tile");
};

// byte offset of 16-byte word w of row r in a tile of D-byte rows, swizzled as TMA and the MMA descriptors do
template <int D>
__device__ __forceinline__ int at(int r, int w)
{
    return D == 128 ? r * 128 + ((w ^ (r & 7)) << 4) : r * 64 + ((w ^ ((r >> 1) & 3)) << 4);
}

// Shared-memory matrix descriptor of a tile of D-byte rows (128- or 64-byte
// swizzle).  K-major (rows are M or N): 8-row groups `group` bytes apart.
// MN-major (rows are K, D consecutive M elements each): the same, and `atom`
// bytes from one D of M to the next.
template <int D>
__device__ __forceinline__ uint64_t tile_desc(uint32_t addr, uint32_t group, uint32_t atom)
{
    uint64_t d = (uint64_t)((addr & 0x3FFFFu) >> 4);
    d |= (uint64_t)(atom >> 4) << 16;
    d |= (uint64_t)(group >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)(D == 128 ? 2 : 4) << 61;
    return d;
}
// MN-major without swizzle, 16 bytes of N to a row: eight rows of K in 128 bytes.
__device__ __forceinline__ uint64_t rows16_desc(uint32_t addr)
{
    return (uint64_t)((addr & 0x3FFFFu) >> 4) | (uint64_t)(128 >> 4) << 16 | (uint64_t)(128 >> 4) << 32 | (uint64_t)1 << 46;
}
// instruction descriptor of kind::f8f6f4: e4m3 x e4m3, fp32 sums, 128 x 16
constexpr uint32_t kIdesc = (1u << 4) | ((16u >> 3) << 17) | ((128u >> 4) << 24);

// D[tmem] (+)= A[smem] * B[smem]^T over 32 bytes of K, issued by one thread.
__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate)
{
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate));
}

__device__ __forceinline__ float lanes_max(float x)
{
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;\n" : "=f"(r) : "f"(x));   // passes NaN over
    return r;
}

// Barrier 1 over the softmax warps; whether any thread brought `x`.
__device__ __forceinline__ bool any_of(bool x)
{
    uint32_t r;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.or.pred q, 1, %2, p;\n selp.u32 %0, 1, 0, q;\n}\n"
        : "=r"(r)
        : "r"((uint32_t)x), "n"(32 * kWarps)
        : "memory");
    return r != 0;
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
// x = hi + lo / S for four values within +-448
template <int S>
__device__ __forceinline__ void split4(float x0, float x1, float x2, float x3, uint32_t &hi, uint32_t &lo)
{
    const uint32_t h01 = e4m3x2(x0, x1), h23 = e4m3x2(x2, x3);
    const float2 f01 = from_e4m3x2(h01), f23 = from_e4m3x2(h23);
    hi = h01 | (h23 << 16);
    lo = e4m3x2(S * (x0 - f01.x), S * (x1 - f01.y)) | (e4m3x2(S * (x2 - f23.x), S * (x3 - f23.y)) << 16);
}

MSA_DEV void mbar_expect_tx(uint64_t *bar, uint32_t bytes)
{
    asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;\n" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
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
    extern __shared__ __align__(1024) uint8_t raw[];
    uint8_t *smem = raw;
    __shared__ uint64_t full[kStages], empty[kStages], c_full[2], c_empty[2], q_full[kQueries], q_empty[kQueries], s_full[2], p_full[2],
        pv_done[2], drained;
    __shared__ Meta meta[kStages];
    __shared__ Chunk chunk[2];
    __shared__ float sQ[2 * kQueries][8];       // logit factor of each head's queries, times log2 e
    __shared__ float sM[kWarps][8], sL[kWarps][8];
    __shared__ uint32_t sLevels[2];             // levels below the first that a page has, a byte to a warp, a bit to a level
    static_assert(kWarps == 4, "a byte to a warp");
    __shared__ uint32_t tmem_slot;
    __shared__ long long before[kPrefixRows + 1];   // blocks, and count, of the rows before each row, one group
    __shared__ int abort_flag;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, G = p.G;
    const bool even = arrived != nullptr;         // stretches of equal length; else whole rows are dealt out

    // blocks (of a selection: slots, as many as the row can fill) that a group of row t has to look at; 0: not a row
    auto blocks_of = [&](int t, int &req, int &pos) {
        req = row_req[t];
        pos = row_pos[t];
        if (req < 0 || pos < 0) return 0;              // behind the last request
        if (req >= p.R || pos / kPage >= p.max_blocks) {
            report(st, kDevCheck, 141, req >= p.R ? req : pos);
            return 0;
        }
        return sel ? min(p.topk, pos / kPage + 1) : pos / kPage + 1;
    };
    if (smem_u32(raw) & 1023u) {                // the swizzled tiles' alignment
        if (tid == 0) report(st, kDevCheck, 157, (int)smem_u32(raw));
        return;
    }
    if (tid == 0) {
        abort_flag = 0;
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], kWarps);
            mbar_init(&pv_done[i], 1);
            mbar_init(&c_full[i], 1);
            mbar_init(&c_empty[i], 1);
        }
        for (int i = 0; i < kQueries; ++i) {
            mbar_init(&q_full[i], 1);
            mbar_init(&q_empty[i], 1);
        }
        mbar_init(&drained, 1);
        fence_mbar_init();
    }
    if (warp == kWarps + 1) {
        tmem_alloc(&tmem_slot, kColumns);
        tmem_relinquish();
    }
    // Not before: a successor that holds TMEM waits for this grid's end, and a CTA of another stream's kernel that wants
    // all of it for the successor's; this grid's must not be behind that one in the queue.
    __syncthreads();
    chain_next();
    chain_wait(q, k_scale, v_scale, block_table, row_req, row_pos, sel, part_o, part_ml, arrived);
    if (even)
        for (int t = tid; t < p.T; t += kThreads) {
            int req, pos;
            const int n = blocks_of(t, req, pos);
            before[t] = n ? n | 1LL << kCountShift : 0;
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
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tmem = tmem_slot;

    if (warp == kWarps + 2) {
        int chunks = 0, pieces = 0;
        bool live = true;
        uint4 x[D / 32];                               // a quarter of head lane / 4's query row
        auto load_q = [&](int t, int r) {
            const uint4 *src = reinterpret_cast<const uint4 *>(q + ((long long)t * p.Hq + (long long)r * G + lane / 4) * D + lane % 4 * (D / 4));
#pragma unroll
            for (int i = 0; i < D / 32; ++i) x[i] = lane / 4 < G ? __ldg(src + i) : make_uint4(0u, 0u, 0u, 0u);
        };
        // ... as hi and lo terms
        auto lay_q = [&](int qi) {
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < D / 32; ++i)
                top = __vmaxu2(__vmaxu2(top, __vmaxu2(x[i].x & 0x7FFF7FFFu, x[i].y & 0x7FFF7FFFu)),
                               __vmaxu2(x[i].z & 0x7FFF7FFFu, x[i].w & 0x7FFF7FFFu));
            top = max(top & 0xFFFFu, top >> 16);
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // not finite: NaN, and so are the scores
            const float sq = __uint_as_float(top >= 0x7F80u ? 0x7FC00000u : pow2_scale_bits(top)), inv = 1.f / sq;
            uint8_t *dst = smem + S::OFF_Q + qi % kQueries * S::Q;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                const float2 a = unpack_bf16(x[i].x), b = unpack_bf16(x[i].y), c = unpack_bf16(x[i].z), d = unpack_bf16(x[i].w);
                uint2 hi, lo;
                split4<16>(a.x * inv, a.y * inv, b.x * inv, b.y * inv, hi.x, lo.x);
                split4<16>(c.x * inv, c.y * inv, d.x * inv, d.y * inv, hi.y, lo.y);
                const int f = lane % 4 * (D / 4) + 8 * i;
                *reinterpret_cast<uint2 *>(dst + at<D>(lane / 4, f >> 4) + (f & 15)) = hi;
                *reinterpret_cast<uint2 *>(dst + at<D>(8 + lane / 4, f >> 4) + (f & 15)) = lo;
            }
            if (lane % 4 == 0) sQ[qi % (2 * kQueries)][lane / 4] = sq * (p.scale * kLog2e);
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(&q_full[qi % kQueries]);
        };
        auto slot_free = [&]() {
            return chunks < 2 || mbar_wait_warp(&c_empty[chunks & 1], ((chunks >> 1) - 1) & 1, st, 158, &abort_flag);
        };
        // blocks (a selection: slots) j0 .. j1 - 1 of group r of row t
        auto piece = [&](int t, int r, int req, int pos, int j0, int j1, int part, int first_cut, int n_cut) {
            const int c0 = pos / kPage, qi = pieces++;
            load_q(t, r);
            for (int base = j0; base < j1; base += 32) {
                int c = -1;
                if (sel) {
                    // selected blocks ascend; an entry that does not, lies past the row's own block, or behind the slots
                    // that the row's blocks can fill, is no block
                    c = lane < p.topk ? sel[((long long)t * p.Hkv + r) * p.topk + lane] : -1;
                    int most = c;
#pragma unroll
                    for (int d = 1; d < 32; d <<= 1) {
                        const int v = __shfl_up_sync(0xffffffffu, most, d);
                        if (lane >= d) most = max(most, v);
                    }
                    most = __shfl_up_sync(0xffffffffu, most, 1);
                    if (c >= 0 && (c > c0 || lane > c0 || (lane > 0 && c <= most))) {
                        report(st, kDevCheck, 142, c);
                        c = -1;
                    }
                    if (lane < j0 || lane >= j1) c = -1;
                } else if (base + lane < j1) {
                    c = base + lane;
                }
                int page = -1, len = 0;
                if (c >= 0) {
                    page = block_table[(long long)req * p.max_blocks + c];
                    if ((unsigned)page >= (unsigned)p.n_pages) {
                        report(st, kDevCheck, 143, page);
                    } else {
                        len = min(kPage, pos - c * kPage + 1);
                    }
                }
                if (!slot_free()) {
                    live = false;
                    return;
                }
                Chunk &ch = chunk[chunks & 1];
                ch.page[lane] = page;
                ch.len[lane] = len;
                // a block without a page is an empty step, and so is a piece without any block
                const unsigned blocks = __ballot_sync(0xffffffffu, c >= 0);
                const bool last = sel || base + 32 >= j1;      // at most 32 slots: one round
                if (lane == 0) {
                    ch.flags = (base == j0 ? kFirst : 0) | (last ? kLast : 0);
                    ch.t = t, ch.r = r, ch.q = qi, ch.part = part, ch.first = first_cut, ch.n = n_cut;
                    ch.blocks = sel && !blocks ? 1u : blocks;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&c_full[chunks & 1]);
                ++chunks;
                if (base == j0) {
                    if (qi >= kQueries && !mbar_wait_warp(&q_empty[qi % kQueries], (qi / kQueries - 1) & 1, st, 159, &abort_flag)) {
                        live = false;
                        return;
                    }
                    lay_q(qi);
                }
                if (last) break;
            }
        };
        const int me = blockIdx.x;
        if (even) {
            constexpr long long kBlocks = (1LL << kCountShift) - 1;
            const int cost = (before[p.T] & kBlocks) * p.Hkv / kMinBlocks > (long long)gridDim.x ? kPieceCost : 0;
            // where row t starts in the list
            auto begin = [&](int t) { return ((before[t] & kBlocks) + cost * (before[t] >> kCountShift)) * p.Hkv; };
            const long long W = begin(p.T);
            const long long n = max(1LL, min((long long)gridDim.x, W / kMinBlocks));
            long long x = me < n ? W * me / n : 0;
            const long long x1 = me < n ? W * (me + 1) / n : 0;
            auto holder = [&](long long y) { return (int)(((y + 1) * n + W - 1) / W - 1); };   // the stretch that has block y
            int t = 0;
            if (x < x1) {                              // the last row that starts at or before x
                int hi = p.T;
                while (hi - t > 1) {
                    const int mid = (t + hi) >> 1;
                    if (begin(mid) <= x) t = mid;
                    else hi = mid;
                }
            }
            while (x < x1 && live) {
                if (x >= begin(t + 1)) {
                    ++t;
                    continue;
                }
                const int nt = (int)((before[t + 1] - before[t]) & kBlocks), r = (int)((x - begin(t)) / (nt + cost));
                const long long x0 = begin(t) + (long long)r * (nt + cost) + cost;   // where the group's blocks start
                x = max(x, x0);
                if (x >= x1) break;
                const int j0 = (int)(x - x0), j1 = (int)min((long long)nt, x1 - x0);
                const bool whole = j0 == 0 && j1 == nt;
                const int f = whole ? 0 : holder(x0), last = whole ? 0 : holder(x0 + nt - 1);
                piece(t, r, row_req[t], row_pos[t], j0, j1, whole ? -1 : 2 * me + (j0 > 0 ? 0 : 1), f, last - f + 1);
                x = x0 + j1;
            }
        } else {
            const long long pairs = (long long)p.T * p.Hkv;
            for (long long i = me; i < pairs && live; i += gridDim.x) {
                int req, pos;
                const int t = (int)(i / p.Hkv), nt = blocks_of(t, req, pos);
                if (nt) piece(t, (int)(i % p.Hkv), req, pos, 0, nt, -1, 0, 0);
            }
        }
        if (live && slot_free() && lane == 0) {
            chunk[chunks & 1].flags = kEnd;
            mbar_arrive(&c_full[chunks & 1]);
        }
    } else if (warp == kWarps) {
        int step = 0;
        bool live = true, ended = false;
        auto copy = [&](const CUtensorMap *tm, uint8_t *dst, uint64_t *bar, int tile, int len) {
            for (int i = 0; i < (len + 31) / 32; ++i)          // 32-token boxes, none past the row
                tma_load_3d(dst + i * 32 * D, tm, bar, 0, i * 32, tile);
        };
        auto stage_free = [&]() {
            return step < kStages || mbar_wait_warp(&empty[step % kStages], (step / kStages - 1) & 1, st, 144, &abort_flag);
        };
        for (int i = 0; live; ++i) {
            if (!mbar_wait_warp(&c_full[i & 1], (i >> 1) & 1, st, 160, &abort_flag)) break;
            const Chunk &ch = chunk[i & 1];
            const int flags = ch.flags;
            if (flags & kEnd) {                        // a chunk of nothing else: its entries hold anything
                ended = stage_free();
                if (ended && lane == 0) {
                    meta[step % kStages].flags = kEnd;
                    meta[step % kStages].len = 0;
                    mbar_arrive(&full[step % kStages]);
                }
                break;
            }
            Meta m;
            m.t = ch.t, m.r = ch.r, m.q = ch.q, m.part = ch.part, m.first = ch.first, m.n = ch.n;
            unsigned todo = ch.blocks;
            const int page = ch.page[lane], len = ch.len[lane];
            // the scales come while the first copies are under way
            const long long ph = len ? (long long)page * p.Hkv + m.r : 0;
            const float ks = len ? k_scale[ph] : 0.f, vs = len ? v_scale[ph] : 1.f;
            __syncwarp();
            if (lane == 0) mbar_arrive(&c_empty[i & 1]);
            bool first = flags & kFirst;
            while (todo) {
                const int l = __ffs(todo) - 1, s = step % kStages;
                todo &= todo - 1;
                m.len = __shfl_sync(0xffffffffu, len, l);
                m.flags = (first ? kFirst : 0) | (!todo && (flags & kLast) ? kLast : 0);
                first = false;
                const int tile = __shfl_sync(0xffffffffu, page, l) * p.Hkv + m.r;
                if (!stage_free()) {
                    live = false;
                    break;
                }
                if (lane == 0 && m.len) {
                    mbar_expect_tx(&full[s], (m.len + 31) / 32 * 64 * D);
                    copy(&tm_k, smem + s * S::STAGE, &full[s], tile, m.len);
                    copy(&tm_v, smem + s * S::STAGE + S::TILE, &full[s], tile, m.len);
                }
                const float lane_vs = __shfl_sync(0xffffffffu, vs, l);
                m.ks = __shfl_sync(0xffffffffu, ks, l);
                m.lv = fmaxf(log2f(lane_vs), -100.f);
                m.il = exp2f(-m.lv);
                m.pv = kOne * (lane_vs * m.il);
                if (lane == 0) {
                    meta[s] = m;
                    mbar_arrive(&full[s]);
                }
                ++step;
            }
        }
        // stay until the last copies have landed (the end mark's stage has been read)
        for (int k = max(0, step - kStages + (ended ? 1 : 0)); k < step; ++k) mbar_wait_warp(&full[k % kStages], (k / kStages) & 1, st, 145, nullptr);
    } else if (warp == kWarps + 1) {
        const uint32_t base = smem_u32(smem);
        auto landed = [&](int i) { return __all_sync(0xffffffffu, mbar_test(&full[i % kStages], (i / kStages) & 1)); };
        // step i's page has landed: its scores, or the end mark passed on
        auto scores = [&](int i) {
            const int s = i % kStages;
            const Meta m = meta[s];
            if (m.flags & kEnd) {
                if (lane == 0) mbar_arrive(&s_full[i & 1]);
                return false;
            }
            if ((m.flags & kFirst) && !mbar_wait_warp(&q_full[m.q % kQueries], (m.q / kQueries) & 1, st, 161, &abort_flag)) return false;
            fence_after_sync();
            if (elect_one()) {
                const uint64_t dk = tile_desc<D>(base + s * S::STAGE, 8 * D, 16), dq = tile_desc<D>(base + S::OFF_Q + m.q % kQueries * S::Q, 8 * D, 16);
#pragma unroll
                for (int k = 0; k < D / 32; ++k) mma_f8(tmem + (i & 1) * 16, desc_adv(dk, k * 32), desc_adv(dq, k * 32), kIdesc, k > 0);
                mma_commit(&s_full[i & 1]);
                if (m.flags & kLast) mma_commit(&q_empty[m.q % kQueries]);
            }
            __syncwarp();
            return true;
        };
        bool more = mbar_wait_warp(&full[0], 0, st, 147, &abort_flag) && scores(0);
        for (int i = 0; more; ++i) {
            // the next page's scores as soon as it is there, this page's products as soon as its probabilities are
            bool ahead = false;
            uint32_t polls = 0;
            while (!__all_sync(0xffffffffu, mbar_test(&p_full[i & 1], (i >> 1) & 1))) {
                if (!ahead && landed(i + 1)) {
                    ahead = true;
                    more = scores(i + 1);
                }
                if (++polls >= kSpinLimit || ((polls & 1023u) == 1023u && *(volatile int *)&abort_flag)) break;
            }
            if (polls >= kSpinLimit || *(volatile int *)&abort_flag) {
                if (polls >= kSpinLimit) report(st, kDevTimeout, 148, i);
                abort_flag = 1;
                break;
            }
            const int s = i % kStages;
            fence_after_sync();
            const Meta m = meta[s];
            uint32_t below = sLevels[i & 1];
            if (elect_one()) {
                const uint64_t dv = tile_desc<D>(base + s * S::STAGE + S::TILE, 8 * D, D == 128 ? 16 : 8 * D);
                const uint64_t dp = rows16_desc(base + s * S::STAGE);
                for (int k = 0; k < max(1, (m.len + 31) / 32); ++k)
                    mma_f8(tmem + kO, desc_adv(dv, k * 32 * D), desc_adv(dp, k * 32 * 16), kIdesc | kAMajorMN | kBMajorMN, k > 0 || !(m.flags & kFirst));
#pragma unroll 1
                for (; below; below &= below - 1) {
                    const int bit = __ffs(below) - 1, k = bit >> 3, v = bit & 7;   // warp k's 32 tokens, level v
                    mma_f8(tmem + kO + 16 * v, desc_adv(dv, k * 32 * D), desc_adv(dp, v * S::P + k * 32 * 16), kIdesc | kAMajorMN | kBMajorMN, true);
                }
                mma_commit(&empty[s]);
                mma_commit(&pv_done[i & 1]);
            }
            __syncwarp();
            if (!ahead) more = mbar_wait_warp(&full[(i + 1) % kStages], ((i + 1) / kStages) & 1, st, 149, &abort_flag) && scores(i + 1);
        }
        if (elect_one()) mma_commit(&drained);
        __syncwarp();
        mbar_wait_warp(&drained, 0, nullptr, 0, nullptr);
    } else {
        const uint32_t lanes = (uint32_t)warp * 32u << 16;   // this warp's quarter of TMEM
        float m_ref[8], l[8], fq[8];
        bool ok = true, live = true;                   // no wait of this thread, of any has run out
        // a cut row whose piece has been handed in, and how many had been before it (thread 0)
        unsigned before_me = 0;
        int cut_n = 0, cut_first = 0;
        long long cut_row = 0;
#pragma unroll
        for (int h = 0; h < 8; ++h) m_ref[h] = -INFINITY, l[h] = fq[h] = 0.f;

        // The last CTA to hand in a piece of a row joins them; of many pieces, first the eight next to each other, and the
        // last to do that for a row the eights (each leaves its count at zero).  The first count comes back while the
        // next page is worked on.
        auto join = [&]() {
            const int n = cut_n, eights = n <= kOneGo ? 1 : (n + 7) / 8, mine = n <= kOneGo ? 0 : ((int)blockIdx.x - cut_first) / 8;
            cut_n = 0;
            int start = cut_first + 8 * mine, stride = 1, count = n <= kOneGo ? n : min(8, n - 8 * mine);
            if (tid == 0 && before_me >= (unsigned)count) report(st, kDevCheck, 164, (int)before_me);   // not zero before the call
            if (!any_of(tid == 0 && before_me == (unsigned)count - 1)) return;
            for (;;) {
                __threadfence();
                constexpr int U = 4, E = 8 * D / (32 * kWarps * 4);   // states, and float4s of a thread, in flight together
                float M[E], L[E];
                float4 y[E];
                auto part = [&](int j) { return 2LL * (start + j * stride) + (start + j * stride == cut_first ? 1 : 0); };
#pragma unroll
                for (int e = 0; e < E; ++e) M[e] = -INFINITY, L[e] = 0.f, y[e] = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int i0 = 0; i0 < count; i0 += U) {
                    float2 ml[E][U];
                    float4 x[E][U];
#pragma unroll
                    for (int e = 0; e < E; ++e)
#pragma unroll
                        for (int u = 0; u < U; ++u) {
                            const int idx = min((tid + e * 32 * kWarps) * 4, G * D - 4);
                            const long long at = part(min(i0 + u, count - 1));
                            ml[e][u] = __ldcg(part_ml + at * 8 + idx / D);
                            x[e][u] = __ldcg(reinterpret_cast<const float4 *>(part_o + at * 8 * D + idx));
                        }
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        float m = M[e];
#pragma unroll
                        for (int u = 0; u < U; ++u) m = fmaxf(m, ml[e][u].x);
                        const float keep = M[e] == -INFINITY ? 1.f : ex2(M[e] - m);   // an empty state is all zeros, one of NaN scores NaN
                        M[e] = m;
                        L[e] *= keep;
                        y[e] = make_float4(y[e].x * keep, y[e].y * keep, y[e].z * keep, y[e].w * keep);
#pragma unroll
                        for (int u = 0; u < U; ++u) {
                            if (i0 + u >= count) break;
                            const float f = ml[e][u].x == -INFINITY ? 1.f : ex2(ml[e][u].x - m);
                            L[e] = fmaf(f, ml[e][u].y, L[e]);
                            y[e] = make_float4(fmaf(f, x[e][u].x, y[e].x), fmaf(f, x[e][u].y, y[e].y), fmaf(f, x[e][u].z, y[e].z),
                                               fmaf(f, x[e][u].w, y[e].w));
                        }
                    }
                }
                const bool all = eights == 1 || stride == 8;
                const long long to = part(0);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const int idx = (tid + e * 32 * kWarps) * 4;
                    if (idx >= G * D) break;
                    if (all) {
                        const float z = L[e] == 0.f ? 0.f : 1.f / L[e];
                        *reinterpret_cast<uint2 *>(o + cut_row * D + idx) =
                            make_uint2(pack_bf16(y[e].x * z, y[e].y * z), pack_bf16(y[e].z * z, y[e].w * z));
                        if (idx % D == 0) lse[cut_row + idx / D] = (M[e] + log2f(L[e])) * kLn2;
                    } else {                           // where the first of the eight was; every thread has read what it replaces
                        *reinterpret_cast<float4 *>(part_o + to * 8 * D + idx) = y[e];
                    }
                }
                if (all) return;
                named_bar_sync(1, 32 * kWarps);        // the sums of the first have been read by all
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const int idx = (tid + e * 32 * kWarps) * 4;
                    if (idx < G * D && idx % D == 0) part_ml[to * 8 + idx / D] = make_float2(M[e], L[e]);
                }
                __threadfence();
                named_bar_sync(1, 32 * kWarps);
                if (!any_of(tid == 0 && atomicInc(&arrived[cut_first], eights - 1) == (unsigned)eights - 1)) return;
                start = cut_first;
                stride = 8;
                count = eights;
            }
        };

        for (int i = 0;; ++i) {
            const int s = i % kStages;
            ok = mbar_wait_warp(&s_full[i & 1], (i >> 1) & 1, st, 146, &abort_flag) && ok;
            fence_after_sync();
            const Meta me = meta[s];
            uint32_t c[16];
            tmem_ld16_nowait(tmem + lanes + (i & 1) * 16, c);
            tmem_wait16(c);
            const bool end = ok && (me.flags & kEnd), first = me.flags & kFirst;
            if (first) {
#pragma unroll
                for (int h = 0; h < 8; ++h) m_ref[h] = -INFINITY, l[h] = 0.f, fq[h] = sQ[me.q % (2 * kQueries)][h];
                uint32_t none[16] = {};                // only the first level's products replace what was there
#pragma unroll
                for (int v = 1; v < kLevels; ++v) tmem_st16(tmem + lanes + kO + 16 * v, none);
            }
            float x[8], over = -INFINITY;
#pragma unroll
            for (int h = 0; h < 8; ++h) {
                x[h] = fmaf(fmaf(__uint_as_float(c[8 + h]), 0.0625f, __uint_as_float(c[h])), fq[h] * me.ks, me.lv);
                if (tid >= me.len) x[h] = -INFINITY;
                over = fmaxf(over, x[h] == -INFINITY ? -INFINITY : x[h] - m_ref[h]);
            }
            // every thread passes the same barriers, also when a wait ran out
            if (any_of((over > kLag && !end) || !ok)) {
                if (any_of(!ok)) {
                    live = false;
                    break;
                }
#pragma unroll
                for (int h = 0; h < 8; ++h) {
                    const float m = lanes_max(x[h]);
                    if (lane == 0) sM[warp][h] = m;
                }
                named_bar_sync(1, 32 * kWarps);
                float alpha[8];
#pragma unroll
                for (int h = 0; h < 8; ++h) {
                    const float m = fmaxf(fmaxf(fmaxf(sM[0][h], sM[1][h]), fmaxf(sM[2][h], sM[3][h])), m_ref[h]);
                    alpha[h] = m == m_ref[h] ? 1.f : ex2(m_ref[h] - m);
                    m_ref[h] = m;
                    l[h] *= alpha[h];
                }
                if (!first) {                          // what has been added up so far
                    ok = mbar_wait_warp(&pv_done[(i - 1) & 1], ((i - 1) >> 1) & 1, st, 150, &abort_flag) && ok;
                    fence_after_sync();
#pragma unroll 1
                    for (int at = kO; at < kO + 16 * kLevels; at += 16) {
                        uint32_t v[16];
                        tmem_ld16_nowait(tmem + lanes + at, v);
                        tmem_wait16(v);
#pragma unroll
                        for (int h = 0; h < 16; ++h) v[h] = __float_as_uint(__uint_as_float(v[h]) * alpha[h & 7]);
                        tmem_st16(tmem + lanes + at, v);
                    }
                    tmem_wait_st();
                }
            }
            if (end) break;
#pragma unroll
            for (int h = 0; h < 8; ++h) {
                // no score yet but -inf (or NaN): -inf - -inf must not be
                const float e = ex2(m_ref[h] == -INFINITY ? x[h] : x[h] - m_ref[h]);
                l[h] = fmaf(e, me.il, l[h]);
                x[h] = e * me.pv;
            }
            float least = x[0];
#pragma unroll
            for (int h = 1; h < 8; ++h) least = fminf(least, x[h]);
            uint8_t *dst = smem + s * S::STAGE + tid * 16;
            // a probability has its terms in the level that fits it, zeros in the others
            const bool some = __any_sync(0xffffffffu, tid < me.len && least < kLevelEnd);
            uint32_t l1[2] = {}, l2[2] = {};           // the heads below the first, the second level, a byte each
            uint32_t below = 0;                        // the levels that the warp's tokens have
            if (some) {
                below = 2;
                if (__any_sync(0xffffffffu, tid < me.len && least < kLevelEnd / kLevelStep)) {
                    below = 6;
#pragma unroll
                    for (int h = 0; h < 8; ++h)
                        if (x[h] < kLevelEnd / kLevelStep) {
                            x[h] *= kLevelStep;
                            l2[h / 4] |= 0xFFu << (h % 4 * 8);
                        }
                }
#pragma unroll
                for (int h = 0; h < 8; ++h)
                    if (x[h] < kLevelEnd) {
                        x[h] *= kLevelStep;
                        l1[h / 4] |= 0xFFu << (h % 4 * 8);
                    }
            }
            uint32_t hi[2], lo[2];                     // e4m3 terms, four heads to a word
#pragma unroll
            for (int w = 0; w < 2; ++w) split4<(int)kLo>(x[4 * w], x[4 * w + 1], x[4 * w + 2], x[4 * w + 3], hi[w], lo[w]);
            *reinterpret_cast<uint4 *>(dst) = make_uint4(hi[0] & ~l1[0], hi[1] & ~l1[1], lo[0] & ~l1[0], lo[1] & ~l1[1]);
            if (some) {
                const uint32_t f0 = l1[0] & ~l2[0], f1 = l1[1] & ~l2[1];
                *reinterpret_cast<uint4 *>(dst + S::P) = make_uint4(hi[0] & f0, hi[1] & f1, lo[0] & f0, lo[1] & f1);
                if (below == 6) *reinterpret_cast<uint4 *>(dst + 2 * S::P) = make_uint4(hi[0] & l2[0], hi[1] & l2[1], lo[0] & l2[0], lo[1] & l2[1]);
            }
            // (every phase of pv_done is waited for: its parity tells two of them apart, not three)
            if (i >= 2) ok = mbar_wait_warp(&pv_done[i & 1], ((i >> 1) - 1) & 1, st, 151, &abort_flag) && ok;
            if (lane == 0) reinterpret_cast<uint8_t *>(&sLevels[i & 1])[warp] = (uint8_t)below;
            // rows behind the last visible token: whatever they hold must not reach 0 * V
            const int rows = max(1, (me.len + 31) / 32) * 32;
            if (tid >= me.len && tid < rows) {
                uint4 *row = reinterpret_cast<uint4 *>(smem + s * S::STAGE + S::TILE + tid * D);
#pragma unroll
                for (int w = 0; w < D / 16; ++w) row[w] = make_uint4(0u, 0u, 0u, 0u);
            }
            if (first) tmem_wait_st();
            fence_before_sync();
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[i & 1]);
            if (cut_n) join();
            if (!(me.flags & kLast)) continue;

            // the piece's outputs: this thread's feature, 8 heads
            float sum[1];
            lane_colsum<8>(l, lane, sum);
            if (lane < 8) sL[warp][lane] = sum[0];
            named_bar_sync(1, 32 * kWarps);
            const int hl = lane & 7;                   // the head whose sum and reference this lane keeps
            const float L = sL[0][hl] + sL[1][hl] + sL[2][hl] + sL[3][hl];
            float ml = m_ref[0];
#pragma unroll
            for (int h = 1; h < 8; ++h) ml = hl == h ? m_ref[h] : ml;
            const bool whole = me.part < 0;
            const float z = (!whole ? 1.f : L == 0.f ? 0.f : 1.f / L) / kOne;
            const long long row = (long long)me.t * p.Hq + (long long)me.r * G;
            if (warp == 0 && lane < G) {
                if (whole) lse[row + lane] = (ml + log2f(L)) * kLn2;
                else part_ml[me.part * 8 + lane] = make_float2(ml, L);
            }
            ok = mbar_wait_warp(&pv_done[i & 1], (i >> 1) & 1, st, 152, &abort_flag) && ok;
            fence_after_sync();
            float sum_o[8] = {};
#pragma unroll
            for (int k = kLevels - 1; k >= 0; --k) {   // the smallest first
                uint32_t v[16];
                tmem_ld16_nowait(tmem + lanes + kO + 16 * k, v);
                tmem_wait16(v);
#pragma unroll
                for (int h = 0; h < 8; ++h)
                    sum_o[h] = fmaf(sum_o[h], 1.f / kLevelStep, fmaf(__uint_as_float(v[8 + h]), 1.f / kLo, __uint_as_float(v[h])));
            }
#pragma unroll
            for (int h = 0; h < 8; ++h) {
                const float zh = __shfl_sync(0xffffffffu, z, h);
                if (h >= G || tid >= D) continue;
                const float y = sum_o[h] * zh;
                if (whole) o[(row + h) * D + tid] = __float2bfloat16_rn(y);
                else part_o[((long long)me.part * 8 + h) * D + tid] = y;
            }
            if (whole) continue;
            __threadfence();                           // the state before the count
            named_bar_sync(1, 32 * kWarps);
            if (tid == 0) {
                // the count of the piece's eight, or of the row where it has few
                const int eight = ((int)blockIdx.x - me.first) / 8;
                const int at = me.n <= kOneGo ? me.first : (eight == 0 ? 2 : 1) * kMostCtas + me.first + 8 * eight;
                before_me = atomicInc(&arrived[at], (me.n <= kOneGo ? me.n : min(8, me.n - 8 * eight)) - 1);
            }
            cut_n = me.n;
            cut_first = me.first;
            cut_row = row;
        }
        if (cut_n && live) join();
    }
    __syncthreads();
    if (warp == kWarps + 1) tmem_dealloc(tmem, kColumns);
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
    const long long rows = (long long)p.T * p.Hkv, most = std::min(2 * p.num_sms, kMostCtas);
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
    // the counts, zero between calls, then the partial outputs and (reference, sum) pairs
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
