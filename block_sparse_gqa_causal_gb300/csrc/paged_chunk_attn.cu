// paged_chunk_attn.cu -- attention of chunks of new tokens over a paged 8-bit cache.
#include <algorithm>

#include <cuda_fp8.h>

#include "paged_chunk.h"
#include "tc.cuh"

namespace msa {

size_t paged_chunk_scores_scratch(const PagedProblem &p);

namespace {

constexpr int kThreads = 128;

__device__ __forceinline__ float e4m3(uint8_t c)
{
    const __half_raw h = __nv_cvt_fp8_to_halfraw(c, __NV_E4M3);
    return __half2float(__half(h));
}

// One (row, group) to a CTA, a token of the page to a thread.
template <int D>
__global__ void __launch_bounds__(kThreads)
chunk_attn_kernel(PagedProblem p, const bf16 *q, const uint8_t *k8, const uint8_t *v8, const float *k_scale, const float *v_scale,
                  const int32_t *block_table, const int32_t *q_starts, const int32_t *row_pos, const int32_t *sel, bf16 *o, float *lse,
                  DeviceStatus *st)
{
    __shared__ float sq[8][D], sp[8][kPage], red[8][4];
    chain_next();
    chain_wait(q, k8, v8, k_scale, v_scale, block_table, q_starts, row_pos, sel);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, G = p.G;
    const int t = blockIdx.x, g = blockIdx.y, pos = row_pos[t];
    int lo = 0, hi = p.R + 1;                       // the last r with q_starts[r] <= t
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (q_starts[mid] <= t) lo = mid;
        else hi = mid;
    }
    if (t == 0 && g == 0)
        for (int r = tid; r < p.R; r += kThreads)
            if (q_starts[r] < 0 || q_starts[r] > q_starts[r + 1] || q_starts[r + 1] > p.T) report(st, kDevCheck, 170, r);
    if (lo >= p.R || q_starts[lo] < 0 || t < q_starts[lo] || t >= q_starts[lo + 1] || q_starts[lo + 1] > p.T || pos < 0) return;
    if ((long long)pos >= (long long)p.max_blocks * kPage) {
        if (tid == 0) report(st, kDevCheck, 171, t);
        return;
    }
    const int req = lo, c_last = pos / kPage;
    for (int i = tid; i < G * D; i += kThreads) sq[i / D][i % D] = __bfloat162float(q[((long long)t * p.Hq + g * G + i / D) * D + i % D]);
    float m[8], z[8], acc[8];
    for (int h = 0; h < 8; ++h) m[h] = -INFINITY, z[h] = acc[h] = 0.f;
    const int entries = sel ? min(p.topk, c_last + 1) : c_last + 1;
    const int given = sel ? p.topk : entries;
    int prev = -1;
    bool any = false;
    for (int i = 0; i < given; ++i) {
        int c = sel ? sel[((long long)t * p.Hkv + g) * p.topk + i] : i;
        if (c == -1) continue;
        if (i >= entries || c <= prev || c > c_last) {
            if (tid == 0) report(st, kDevCheck, 180, t);
            continue;
        }
        prev = c;
        const int page = block_table[(long long)req * p.max_blocks + c];
        if ((unsigned)page >= (unsigned)p.n_pages) {
            if (tid == 0) report(st, kDevCheck, 173, page);
            continue;
        }
        any = true;
        const long long tile = ((long long)page * p.Hkv + g) * kPage * D;
        const float ks = k_scale[(long long)page * p.Hkv + g] * p.scale, vs = v_scale[(long long)page * p.Hkv + g];
        const bool seen = c * kPage + tid <= pos;
        __syncthreads();
        for (int h = 0; h < G; ++h) {
            float s = -INFINITY;
            if (seen) {
                s = 0.f;
                for (int e = 0; e < D; ++e) s += sq[h][e] * e4m3(k8[tile + tid * D + e]);
                s *= ks;
            }
            sp[h][tid] = s;
            const float w = warp_max(s);
            if (lane == 0) red[h][warp] = w;
        }
        __syncthreads();
        for (int h = 0; h < G; ++h) {
            const float top = fmaxf(m[h], fmaxf(fmaxf(red[h][0], red[h][1]), fmaxf(red[h][2], red[h][3])));
            const float keep = m[h] == -INFINITY ? 0.f : expf(m[h] - top);
            z[h] *= keep;
            acc[h] *= keep;
            m[h] = top;
            for (int j = 0; j < kPage && c * kPage + j <= pos; ++j) {
                const float e = expf(sp[h][j] - top);
                z[h] += e;
                if (tid < D) acc[h] += e * vs * e4m3(v8[tile + j * D + tid]);
            }
        }
    }
    for (int h = 0; h < G; ++h) {
        const long long row = (long long)t * p.Hq + g * G + h;
        if (tid < D) o[row * D + tid] = __float2bfloat16(any ? acc[h] / z[h] : 0.f);
        if (tid == 0) lse[row] = any ? m[h] + logf(z[h]) : -INFINITY;
    }
}

}  // namespace

size_t paged_chunk_scratch_bytes(const PagedProblem &p, bool attention) { return attention ? 0 : paged_chunk_scores_scratch(p); }

cudaError_t launch_paged_chunk_attn(const PagedProblem &p, const bf16 *q, const uint8_t *k8, const uint8_t *v8, const float *k_scale,
                                    const float *v_scale, const int32_t *block_table, const int32_t *q_starts, const int32_t *row_pos,
                                    const int32_t *sel, bf16 *o, float *lse, void *scratch, DeviceStatus *st, cudaStream_t s)
{
    return launch_chained("paged_chunk_attn_kernel", p.d == 128 ? chunk_attn_kernel<128> : chunk_attn_kernel<64>, dim3(p.T, p.Hkv), kThreads, 0, s,
                          p, q, k8, v8, k_scale, v_scale, block_table, q_starts, row_pos, sel, o, lse, st);
}

}  // namespace msa
