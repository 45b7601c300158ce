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
// A producer warp streams pages (K and V tiles of one head, contiguous and
// swizzled by TMA) through a ring of stages.  Each of four warps takes 32 of a
// page's 128 tokens and keeps its own running maximum, sum and output; they
// are joined at the end.  V's operand needs its tokens along a register:
// ldmatrix with 8-bit transposition gives that from the row-major tile.  The
// tokens' order inside a 32-token step is chosen so that a lane's scores are
// the probabilities it has to feed back and no shared-memory phase has a bank
// conflict.
//
// A row's blocks are cut into shares of `per` blocks, one CTA to a share; a
// second kernel joins the shares' states where there is more than one.
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

struct Meta {
    int len;        // visible tokens of the block; -1 after the last block
    float ks, vs;   // the page's scales for this head
};

template <int D>
struct AttnSmem {
    static constexpr int TILE = kPage * D;      // K or V codes of a page and head
    static constexpr int STAGE = 2 * TILE;
    static constexpr int BYTES = kStages * STAGE + 1024;   // + alignment
};
static_assert(AttnSmem<64>::STAGE * kStages >= kWarps * 8 * 64 * 4 + 512, "the warps' states fit the stages");

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

// The share's blocks, 32 at a time: what lane `lane` holds of them.
struct Entry {
    int page, len;
    float ks, vs;
};

template <int D>
__global__ void __launch_bounds__(kThreads, 2)
attn_kernel(PagedProblem p, const bf16 *__restrict__ q, const __grid_constant__ CUtensorMap tm_k,
            const __grid_constant__ CUtensorMap tm_v, const float *__restrict__ k_scale,
            const float *__restrict__ v_scale, const int32_t *__restrict__ block_table,
            const int32_t *__restrict__ row_req, const int32_t *__restrict__ row_pos, const int32_t *__restrict__ sel,
            bf16 *__restrict__ o, float *__restrict__ lse, int per, int shares, float *__restrict__ part_o,
            float2 *__restrict__ part_ml, DeviceStatus *st)
{
    using S = AttnSmem<D>;
    extern __shared__ uint8_t raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
    __shared__ uint64_t full[kStages], empty[kStages];
    __shared__ Meta meta[kStages];
    __shared__ int abort_flag;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int sp = blockIdx.x % shares;
    const int rt = blockIdx.x / shares, r = rt % p.Hkv, t = rt / p.Hkv;
    const int req = row_req[t], pos = row_pos[t];
    if (req < 0 || pos < 0) return;                    // a row behind the last request
    const int c0 = pos / kPage;
    if (req >= p.R || c0 >= p.max_blocks) {
        if (tid == 0) report(st, kDevCheck, 141, req >= p.R ? req : pos);
        return;
    }
    // without a selection a short row has fewer shares than the longest
    const int lo = sp * per, hi = sel ? min(lo + per, p.topk) : min(lo + per, c0 + 1);
    if (!sel && lo > c0) return;
    const bool alone = shares == 1 || (!sel && c0 < per);

    if (tid == 0) {
        abort_flag = 0;
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], kWarps);
        }
        fence_mbar_init();
    }
    __syncthreads();

    if (warp == kWarps) {
        int step = 0;
        bool live = true;
        for (int base = lo; base < hi && live; base += 32) {
            int c = -1;
            if (sel) {
                // selected blocks ascend; an entry that does not, or lies past the row's own block, is no block
                c = lane < p.topk ? sel[((long long)t * p.Hkv + r) * p.topk + lane] : -1;
                int before = c;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const int v = __shfl_up_sync(0xffffffffu, before, d);
                    if (lane >= d) before = max(before, v);
                }
                before = __shfl_up_sync(0xffffffffu, before, 1);
                if (c >= 0 && (c > c0 || (lane > 0 && c <= before))) {
                    report(st, kDevCheck, 142, c);
                    c = -1;
                }
                c = __shfl_sync(0xffffffffu, c, (base + lane) & 31);
                if (base + lane >= hi) c = -1;
            } else if (base + lane < hi) {
                c = base + lane;
            }
            Entry e{-1, 0, 0.f, 0.f};
            if (c >= 0) {
                e.page = block_table[(long long)req * p.max_blocks + c];
                if ((unsigned)e.page >= (unsigned)p.n_pages) {
                    report(st, kDevCheck, 143, e.page);
                    c = -1;
                } else {
                    e.len = min(kPage, pos - c * kPage + 1);
                    e.ks = k_scale[(long long)e.page * p.Hkv + r];
                    e.vs = v_scale[(long long)e.page * p.Hkv + r];
                }
            }
            unsigned todo = __ballot_sync(0xffffffffu, c >= 0);
            while (todo) {
                const int l = __ffs(todo) - 1, s = step % kStages;
                todo &= todo - 1;
                const int page = __shfl_sync(0xffffffffu, e.page, l), len = __shfl_sync(0xffffffffu, e.len, l);
                const float ks = __shfl_sync(0xffffffffu, e.ks, l), vs = __shfl_sync(0xffffffffu, e.vs, l);
                if (step >= kStages && !mbar_wait_warp(&empty[s], (step / kStages - 1) & 1, st, 144, &abort_flag)) {
                    live = false;
                    break;
                }
                if (lane == 0) {
                    meta[s] = Meta{len, ks, vs};
                    const int boxes = (len + 31) / 32;             // 32-token boxes, none past the row
                    mbar_arrive_expect_tx(&full[s], boxes * 64 * D);
                    uint8_t *dst = smem + s * S::STAGE;
                    for (int x = 0; x < boxes; ++x)
                        tma_load_3d(dst + x * 32 * D, &tm_k, &full[s], 0, x * 32, page * p.Hkv + r);
                    for (int x = 0; x < boxes; ++x)
                        tma_load_3d(dst + S::TILE + x * 32 * D, &tm_v, &full[s], 0, x * 32, page * p.Hkv + r);
                }
                ++step;
            }
        }
        const int s = step % kStages;
        if (live && step >= kStages) live = mbar_wait_warp(&empty[s], (step / kStages - 1) & 1, st, 144, &abort_flag);
        if (live && lane == 0) {
            meta[s].len = -1;
            mbar_arrive(&full[s]);
        }
        // stay until the last copies have landed
        for (int k = max(0, step - kStages); k < step; ++k)
            if (!live || k % kStages != s) mbar_wait_warp(&full[k % kStages], (k / kStages) & 1, st, 145, nullptr);
    }

    const int g = lane >> 2, t4 = lane & 3, G = p.G;
    float acc[D / 8][2];                               // head g, features 8n + 2 t4, + 1
    float m_run = -INFINITY, l_run = 0.f;
#pragma unroll
    for (int n = 0; n < D / 8; ++n) acc[n][0] = acc[n][1] = 0.f;

    if (warp < kWarps) {
        // the queries as hi and lo terms, features 32 ks + 4 t4 .. + 3 and + 16 ..
        uint32_t a[D / 32][4];
        float sq;
        {
            const bool ok = g < G;
            const uint2 *src = reinterpret_cast<const uint2 *>(q + ((long long)t * p.Hq + (long long)r * G + (ok ? g : 0)) * D);
            uint2 x[D / 32][2];
            uint32_t top = 0;
#pragma unroll
            for (int ks = 0; ks < D / 32; ++ks)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    x[ks][e] = ok ? __ldg(src + ks * 8 + e * 4 + t4) : make_uint2(0u, 0u);
                    top = __vmaxu2(top, __vmaxu2(x[ks][e].x & 0x7FFF7FFFu, x[ks][e].y & 0x7FFF7FFFu));
                }
            top = max(top & 0xFFFFu, top >> 16);
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            sq = top >= 0x7F80u ? __uint_as_float(0x7FC00000u) : __uint_as_float(pow2_scale_bits(top));   // NaN: so are the scores
            const float inv = 1.f / sq;
#pragma unroll
            for (int ks = 0; ks < D / 32; ++ks)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float2 u = unpack_bf16(x[ks][e].x), v = unpack_bf16(x[ks][e].y);
                    split4(u.x * inv, u.y * inv, v.x * inv, v.y * inv, a[ks][2 * e], a[ks][2 * e + 1]);
                }
        }
        const float sql = sq * (p.scale * kLog2e);
        const int kw = warp * 32;                      // this warp's first token of a page
        // K rows: token column j of score tile n is token 8n + (j ^ 4 (n & 1))
        const int kj = lane & 7, km = lane >> 3;
        // V rows: probability k (of 16) is lane (k / 4)'s value e = k & 1 of tile (k / 2) & 1
        const int vk = lane & 15, vn = (vk >> 1) & 1;
        const int vrow = kw + 16 * (lane >> 4) + 8 * vn + ((2 * (vk >> 2) + (vk & 1)) ^ (4 * vn));

        for (int step = 0;; ++step) {
            const int s = step % kStages;
            if (!mbar_wait_warp(&full[s], (step / kStages) & 1, st, 146, &abort_flag)) break;
            const Meta me = meta[s];
            if (me.len < 0) break;
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
                float mx = -INFINITY;
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
                    for (int e = 0; e < 2; ++e) {
                        sc[n][e] = fmaf(c[2 + e], 0.0625f, c[e]) * fac;
                        if (kw + 8 * n + ((2 * t4 + e) ^ (4 * (n & 1))) >= me.len) sc[n][e] = -INFINITY;
                        mx = fmaxf(mx, sc[n][e]);
                    }
                }
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                const float m_new = fmaxf(m_run, mx);
                const float m_use = m_new == -INFINITY ? 0.f : m_new;
                const float alpha = exp2f(m_run - m_use);
                m_run = m_new;
                float ps = 0.f;
#pragma unroll
                for (int n = 0; n < 4; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        sc[n][e] = exp2f(sc[n][e] - m_use);
                        ps += sc[n][e];
                        sc[n][e] *= 256.f;             // the upper end of e4m3's range
                    }
                l_run = fmaf(l_run, alpha, ps);
                uint32_t pa[4];
                split4(sc[0][0], sc[0][1], sc[1][0], sc[1][1], pa[0], pa[1]);
                split4(sc[2][0], sc[2][1], sc[3][0], sc[3][1], pa[2], pa[3]);
                const float vf = me.vs * (1.f / 256.f);
#pragma unroll
                for (int w = 0; w < D / 16; ++w) {
                    uint32_t b[4];
                    ldsm_b8_t(b, sv + at<D>(vrow, w));
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float c[4] = {0.f, 0.f, 0.f, 0.f};
                        mma_e4m3(c, pa, b[e], b[2 + e]);
                        float(&x)[2] = acc[2 * w + e];
                        x[0] = fmaf(fmaf(c[2], 0.0625f, c[0]), vf, x[0] * alpha);
                        x[1] = fmaf(fmaf(c[3], 0.0625f, c[1]), vf, x[1] * alpha);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[s]);
        }
        l_run += __shfl_xor_sync(0xffffffffu, l_run, 1);
        l_run += __shfl_xor_sync(0xffffffffu, l_run, 2);
    }

    // join the four warps' states, in order
    __syncthreads();                                   // the stages are read and no copy is in flight
    float *sO = reinterpret_cast<float *>(smem), *sM = sO + kWarps * 8 * D, *sL = sM + kWarps * 8;
    if (warp < kWarps && g < G) {
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
            *reinterpret_cast<float2 *>(sO + (warp * 8 + g) * D + n * 8 + 2 * t4) = make_float2(acc[n][0], acc[n][1]);
        if (t4 == 0) {
            sM[warp * 8 + g] = m_run;
            sL[warp * 8 + g] = l_run;
        }
    }
    __syncthreads();
    for (int idx = tid; idx < G * D; idx += kThreads) {
        const int h = idx / D, col = idx % D;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sM[w * 8 + h]);
        float L = 0.f, x = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = sM[w * 8 + h] == -INFINITY ? 1.f : exp2f(sM[w * 8 + h] - M);
            L += f * sL[w * 8 + h];                    // an empty state is all zeros, one of NaN scores NaN
            x += f * sO[(w * 8 + h) * D + col];
        }
        const long long row = (long long)t * p.Hq + (long long)r * G + h;
        if (alone) {
            o[row * D + col] = __float2bfloat16_rn(L == 0.f ? 0.f : x / L);
            if (col == 0) lse[row] = (M + log2f(L)) * kLn2;
        } else {
            part_o[(row * shares + sp) * D + col] = x;
            if (col == 0) part_ml[row * shares + sp] = make_float2(M, L);
        }
    }
}

// Joins the shares of a (row, head): a warp each, shares in order.
template <int D>
__global__ void __launch_bounds__(256)
join_kernel(PagedProblem p, const int32_t *__restrict__ row_req, const int32_t *__restrict__ row_pos, int sparse, int per,
            int shares, const float *__restrict__ part_o, const float2 *__restrict__ part_ml, bf16 *__restrict__ o,
            float *__restrict__ lse)
{
    const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (row >= (long long)p.T * p.Hq) return;
    const int t = (int)(row / p.Hq), req = row_req[t], pos = row_pos[t];
    if (req < 0 || pos < 0 || req >= p.R || pos / kPage >= p.max_blocks) return;
    const int c0 = pos / kPage, ns = sparse ? shares : c0 / per + 1;
    if (ns == 1 && !sparse) return;                    // the row's only share wrote the outputs
    const float2 *ml = part_ml + row * shares;
    float M = -INFINITY;
    for (int i = lane; i < ns; i += 32) M = fmaxf(M, ml[i].x);
    M = warp_max(M);
    constexpr int PER = D / 32;
    float L = 0.f, acc[PER];
#pragma unroll
    for (int e = 0; e < PER; ++e) acc[e] = 0.f;
    for (int i = 0; i < ns; ++i) {
        const float2 x = ml[i];
        const float f = x.x == -INFINITY ? 1.f : exp2f(x.x - M);
        L += f * x.y;
        const float *src = part_o + (row * shares + i) * D + lane;
#pragma unroll
        for (int e = 0; e < PER; ++e) acc[e] += f * src[32 * e];
    }
#pragma unroll
    for (int e = 0; e < PER; ++e) o[row * D + lane + 32 * e] = __float2bfloat16_rn(L == 0.f ? 0.f : acc[e] / L);
    if (lane == 0) lse[row] = (M + log2f(L)) * kLn2;
}

// Blocks of a share: the rows' shares should fill the GPU's CTA slots (two to
// an SM) about four times, in shares of at least two blocks, at most 128 of
// them to a row.
int share_blocks(const PagedProblem &p, bool sparse)
{
    const int blocks = sparse ? p.topk : p.max_blocks;
    const long long rows = (long long)p.T * p.Hkv;
    const long long want = std::max<long long>(1, std::min<long long>(128, 8LL * p.num_sms / rows));
    return (int)std::max<long long>(std::min(2, blocks), (blocks + want - 1) / want);
}
int share_count(const PagedProblem &p, bool sparse)
{
    const int per = share_blocks(p, sparse);
    return ((sparse ? p.topk : p.max_blocks) + per - 1) / per;
}

}  // namespace

size_t paged_attn_scratch_floats(const PagedProblem &p)
{
    const size_t n = std::max(share_count(p, true), share_count(p, false));
    return n == 1 ? 0 : (size_t)p.T * p.Hq * n * (p.d + 2);
}

cudaError_t launch_paged_attn(const PagedProblem &p, const bf16 *q, const uint8_t *k8, const uint8_t *v8,
                              const float *k_scale, const float *v_scale, const int32_t *block_table,
                              const int32_t *row_req, const int32_t *row_pos, const int32_t *sel, bf16 *o, float *lse,
                              float *scratch, DeviceStatus *st, cudaStream_t s)
{
    const int per = share_blocks(p, sel != nullptr), shares = share_count(p, sel != nullptr);
    const long long rows = (long long)p.T * p.Hq;
    float *part_o = scratch;
    float2 *part_ml = reinterpret_cast<float2 *>(scratch + (shares > 1 ? rows * shares * p.d : 0));
    CUtensorMap tk, tv;
    cudaError_t e = make_tmap_u8_3d(&tk, k8, p.d, kPage, (unsigned long long)p.n_pages * p.Hkv, p.d, 32);
    if (e == cudaSuccess) e = make_tmap_u8_3d(&tv, v8, p.d, kPage, (unsigned long long)p.n_pages * p.Hkv, p.d, 32);
    if (e != cudaSuccess) return e;
    auto run = [&](auto dtag) {
        constexpr int D = decltype(dtag)::value;
        e = cudaFuncSetAttribute(attn_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, AttnSmem<D>::BYTES);
        if (e != cudaSuccess) return;
        {
            TimedLaunch timed_("paged_attn_kernel", s);
            attn_kernel<D><<<(unsigned)((long long)p.T * p.Hkv * shares), kThreads, AttnSmem<D>::BYTES, s>>>(
                p, q, tk, tv, k_scale, v_scale, block_table, row_req, row_pos, sel, o, lse, per, shares, part_o, part_ml, st);
        }
        note_launch();
        if (shares > 1) {
            TimedLaunch timed_("paged_attn_join_kernel", s);
            join_kernel<D><<<(unsigned)((rows + 7) / 8), 256, 0, s>>>(p, row_req, row_pos, sel != nullptr, per, shares,
                                                                      part_o, part_ml, o, lse);
            note_launch();
        }
    };
    if (p.d == 128) run(std::integral_constant<int, 128>{});
    else run(std::integral_constant<int, 64>{});
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace msa
