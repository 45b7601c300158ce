// rotary.cu -- rotary positions of queries and keys, forward and backward.
//
// Token t at position p turns the pair (x_i, x_j) of a head by p f_i:
//   y_i = g (x_i cos - x_j sin),  y_j = g (x_i sin + x_j cos);
// the backward pass is the transposed map, the same with sin negated.
//
// The angle: f_i / 2 pi comes as a 64-bit fraction of a turn, so p times it, in
// 64-bit integers, is the turn's fraction exactly (the whole turns fall off at the
// top), whatever p; its upper 32 bits go to sincospif.  In fp32, p f_i alone is
// off by 2^-4 radians at a position of a million.
//
// Each feature is read and written once; the bytes bound it.  A CTA takes a few
// tokens, makes their cosines and sines once (a thread to a pair) for all
// heads of q and k, and then streams the heads: a thread takes 16 features, the
// two 16-byte words that hold eight pairs.  32,768 tokens of 64 + 8 heads of 128
// features: 179 us, the copy rate; 64 tokens: 5 us, the launch and one chain of
// loads.
#include <algorithm>

#include "paged.h"

namespace msa {
namespace {

constexpr int kThreads = 256;
constexpr int kMostPairs = 128;

template <int TOK, bool INTER>
__global__ void __launch_bounds__(kThreads)
rotary_kernel(RotaryProblem p, const bf16 *q, const bf16 *k, const int32_t *positions, const unsigned long long *freqs, bf16 *q_out,
              bf16 *k_out)
{
    __shared__ __align__(16) float2 cs[TOK][kMostPairs];
    __shared__ int skip[TOK];
    chain_next();
    chain_wait(q, k, positions, freqs);
    const int tid = threadIdx.x, t0 = blockIdx.x * TOK, pairs = p.d_rot / 2;
    const int toks = min(TOK, p.T - t0);
    for (int i = tid; i < toks * pairs; i += kThreads) {
        const int tk = i / pairs, j = i - tk * pairs, t = t0 + tk;
        const int pos = positions ? positions[t] : p.offset + t % p.period;
        const int turn = (int)((unsigned long long)(unsigned)pos * freqs[j] >> 32);
        float s, c;
        sincospif((float)turn * 0x1p-31f, &s, &c);
        cs[tk][j] = make_float2(p.scale * c, p.backward ? -p.scale * s : p.scale * s);
        if (j == 0) skip[tk] = pos < 0;
    }
    __syncthreads();
    const int per_head = p.d / 16, turned = p.d_rot / 16;       // 16 features each
    const int heads = p.Hq + p.Hkv, units = heads * per_head;
    for (int i = tid; i < toks * units; i += kThreads) {
        const int tk = i / units, r = i - tk * units, h = r / per_head, j = r - h * per_head;
        const bool is_q = h < p.Hq;
        const long long t = t0 + tk;
        const bf16 *x = is_q ? q + t * p.q_stride + (long long)h * p.d : k + t * p.k_stride + (long long)(h - p.Hq) * p.d;
        bf16 *y = is_q ? q_out + t * p.q_out_stride + (long long)h * p.d : k_out + t * p.k_out_stride + (long long)(h - p.Hq) * p.d;
        const int w0 = INTER || j >= turned ? 2 * j : j, w1 = INTER || j >= turned ? 2 * j + 1 : j + turned;
        if (skip[tk]) {
            if (p.zeros & (is_q ? 1 : 2)) reinterpret_cast<uint4 *>(y)[w0] = reinterpret_cast<uint4 *>(y)[w1] = make_uint4(0, 0, 0, 0);
            continue;
        }
        uint4 a = reinterpret_cast<const uint4 *>(x)[w0], b = reinterpret_cast<const uint4 *>(x)[w1];
        if (j < turned) {
            const float4 *f = reinterpret_cast<const float4 *>(&cs[tk][8 * j]);
            uint32_t u[4] = {a.x, a.y, a.z, a.w}, v[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float4 c = f[e];                          // {cos, sin} of pairs 2e and 2e + 1
                if constexpr (INTER) {
                    uint32_t *w = e < 2 ? u : v;                // pair m in word m of the 32 bytes
                    const float2 m = unpack_bf16(w[2 * (e & 1)]), n = unpack_bf16(w[2 * (e & 1) + 1]);
                    w[2 * (e & 1)] = pack_bf16(m.x * c.x - m.y * c.y, m.x * c.y + m.y * c.x);
                    w[2 * (e & 1) + 1] = pack_bf16(n.x * c.z - n.y * c.w, n.x * c.w + n.y * c.z);
                } else {
                    const float2 m = unpack_bf16(u[e]), n = unpack_bf16(v[e]);
                    u[e] = pack_bf16(m.x * c.x - n.x * c.y, m.y * c.z - n.y * c.w);
                    v[e] = pack_bf16(m.x * c.y + n.x * c.x, m.y * c.w + n.y * c.z);
                }
            }
            a = make_uint4(u[0], u[1], u[2], u[3]);
            b = make_uint4(v[0], v[1], v[2], v[3]);
        }
        reinterpret_cast<uint4 *>(y)[w0] = a;
        reinterpret_cast<uint4 *>(y)[w1] = b;
    }
}

}  // namespace

cudaError_t launch_rotary(const RotaryProblem &p, const bf16 *q, const bf16 *k, const int32_t *positions,
                          const unsigned long long *freqs, bf16 *q_out, bf16 *k_out, cudaStream_t s)
{
    auto run = [&](auto kernel, int tok) {
        return launch_chained("rotary_kernel", kernel, dim3((unsigned)((p.T + (long long)tok - 1) / tok)), kThreads, 0, s, p, q, k, positions, freqs,
                              q_out, k_out);
    };
    // four tokens share a CTA's set-up where that leaves a CTA to every place on the GPU
    if (p.T >= 4 * 8 * p.num_sms) return p.interleaved ? run(rotary_kernel<4, true>, 4) : run(rotary_kernel<4, false>, 4);
    return p.interleaved ? run(rotary_kernel<1, true>, 1) : run(rotary_kernel<1, false>, 1);
}

}  // namespace msa
