// paged_append.cu -- new tokens into a paged cache whose K and V are e4m3
// with one power-of-two scale per (page, KV head).
//
// s = 2^e, the least e for which every finite value of the page's rows is at
// most 448 s; codes are x / s rounded to nearest, ties to even.  x / s is
// exact, so a code's only error is the e4m3 rounding, and when a later token
// makes the scale grow, the codes already there move by whole binades: they
// stay exact unless they fall among the subnormals (below s 2^-6).  A scale
// that is no power of two would round every older token again.
//
// A segment is the rows of one step that go to one page.  One CTA takes a
// (segment, KV head): four warps its K rows, four its V rows.  The rows stay
// in registers between the maximum and the conversion (128 rows x 128
// features: 64 registers a lane), so the new rows are read once and the codes
// written once; that traffic bounds the call: 64 us, 99% of the copy rate, for
// 64,936 tokens of 8 KV heads (432 MB).  Three CTAs to an SM keep enough loads
// in flight across the barrier (two: 82 us, with the search for infinities in
// every row); one token a request, 64 of them, takes 4 us.
#include <cuda_fp8.h>

#include <algorithm>

#include "paged.h"

namespace msa {
namespace {

constexpr int kThreads = 256;

// two floats -> two e4m3 codes (lo in the low byte); finite values within
// +-448, NaN -> NaN code
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

template <int D>
__global__ void __launch_bounds__(kThreads, 3)
append_kernel(PagedProblem p, const uint4 *__restrict__ k_new, const uint4 *__restrict__ v_new,
              const uint4 *__restrict__ ki_new, const int32_t *__restrict__ slots, const int32_t *__restrict__ segs,
              uint8_t *__restrict__ k8, uint8_t *__restrict__ v8, float *__restrict__ k_scale,
              float *__restrict__ v_scale, uint4 *__restrict__ k_idx, DeviceStatus *st)
{
    constexpr int LPR = D / 8;                // lanes of a row, 16 bytes each
    constexpr int RPI = kThreads / 2 / LPR;   // rows of a half-CTA load
    constexpr int N = kPage / RPI;            // loads that cover a page
    __shared__ uint32_t part[2][4];

    chain_next();
    chain_wait(slots, segs);                  // every other address depends on what these say
    const int u = blockIdx.x, h = blockIdx.y, tid = threadIdx.x;
    const int t0 = segs[u], t1 = segs[u + 1], cnt = t1 - t0;
    if (cnt <= 0) return;
    if (t0 < 0 || t1 > p.T || cnt > kPage) {
        if (tid == 0) report(st, kDevCheck, 111, u);
        return;
    }
    const int slot = slots[t0];
    if (slot < 0) return;                     // a row without a page (the plan reported it)
    const int page = slot / kPage, off = slot % kPage;
    if (page >= p.n_pages || off + cnt > kPage) {
        if (tid == 0) report(st, kDevCheck, 112, slot);
        return;
    }
    if (h >= p.Hkv) {                         // the index keys: bf16 rows, copied
        const int w = p.d_idx / 8;
        const uint4 *src = ki_new + (long long)t0 * w;
        uint4 *dst = k_idx + ((long long)page * kPage + off) * w;
        for (int i = tid; i < cnt * w; i += kThreads) dst[i] = src[i];
        return;
    }
    if (!k_new) return;
    const int half = tid / (kThreads / 2), ht = tid % (kThreads / 2);
    const uint4 *src = half ? v_new : k_new;
    const long long ph = (long long)page * p.Hkv + h;
    uint8_t *codes = (half ? v8 : k8) + ph * kPage * D;
    float *scale = (half ? v_scale : k_scale) + ph;
    const float had = off > 0 ? *scale : 0.f;

    const int row0 = ht / LPR, col = ht % LPR;
    uint4 x[N];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int row = row0 + i * RPI;
        x[i] = make_uint4(0u, 0u, 0u, 0u);
        if (row < cnt) x[i] = __ldg(src + ((long long)(t0 + row) * p.Hkv + h) * LPR + col);
    }
    auto largest = [&](uint32_t v) {
        v = __reduce_max_sync(0xffffffffu, max(v & 0xFFFFu, v >> 16));
        if ((tid & 31) == 0) part[half][(tid >> 5) & 3] = v;
        named_bar_sync(1 + half, kThreads / 2);
        return max(max(part[half][0], part[half][1]), max(part[half][2], part[half][3]));
    };
#pragma unroll
    for (int i = 0; i < N; ++i)
        top = __vmaxu2(__vmaxu2(top, __vmaxu2(x[i].x & 0x7FFF7FFFu, x[i].y & 0x7FFF7FFFu)),
                       __vmaxu2(x[i].z & 0x7FFF7FFFu, x[i].w & 0x7FFF7FFFu));
    top = largest(top);
    if (top >= 0x7F80u) {                     // rare: NaN for infinities, and the largest finite value
        top = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            uint32_t *w = &x[i].x;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t a = w[e] & 0x7FFF7FFFu, bad = __vcmpgeu2(a, 0x7F807F80u);
                top = __vmaxu2(top, a & ~bad);
                w[e] |= bad & 0x7FFF7FFFu;    // e4m3 has no infinity, and 448 s would pass for a value
            }
        }
        named_bar_sync(1 + half, kThreads / 2);   // the first maxima have been read
        top = largest(top);
    }
    const float s = fmaxf(had, __uint_as_float(pow2_scale_bits(top)));
    const float inv = 1.f / s;
    if (off > 0 && s > had) {                 // the page's older codes, to the larger scale
        const float f = had * inv;
        uint4 *old = reinterpret_cast<uint4 *>(codes);
        for (int i = ht; i < off * D / 16; i += kThreads / 2) {
            uint4 c = old[i];
            uint32_t *w = &c.x;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 a = from_e4m3x2(w[e] & 0xFFFFu), b = from_e4m3x2(w[e] >> 16);
                w[e] = e4m3x2(a.x * f, a.y * f) | (e4m3x2(b.x * f, b.y * f) << 16);
            }
            old[i] = c;
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int row = row0 + i * RPI;
        if (row >= cnt) break;
        const uint32_t *w = &x[i].x;
        uint32_t c[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 f = unpack_bf16(w[e]);
            c[e] = e4m3x2(f.x * inv, f.y * inv);
        }
        *reinterpret_cast<uint2 *>(codes + (off + row) * D + col * 8) = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
    }
    if (ht == 0) *scale = s;                  // every thread of the half has read it before the barrier
}

}  // namespace

cudaError_t launch_paged_append(const PagedProblem &p, const bf16 *k_new, const bf16 *v_new, const bf16 *ki_new,
                                const int32_t *slots, const int32_t *segs, uint8_t *k8, uint8_t *v8, float *k_scale,
                                float *v_scale, bf16 *k_idx, DeviceStatus *st, cudaStream_t s)
{
    const dim3 grid(paged_segments(p), p.Hkv + (ki_new ? 1 : 0));
    return launch_chained("paged_append_kernel", p.d == 128 ? append_kernel<128> : append_kernel<64>, grid, kThreads, 0, s, p,
                          reinterpret_cast<const uint4 *>(k_new), reinterpret_cast<const uint4 *>(v_new),
                          reinterpret_cast<const uint4 *>(ki_new), slots, segs, k8, v8, k_scale, v_scale,
                          reinterpret_cast<uint4 *>(k_idx), st);
}

}  // namespace msa
