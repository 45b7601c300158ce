// paged.h -- problem description and launchers of the paged-cache operators
// (plan, append, block scores, block selection, attention), shared by their
// C-ABI layer (paged_api.cu) and kernels.
#pragma once

#include <atomic>
#include <utility>

#include "msa_internal.h"

namespace msa {

constexpr int kPage = 128;   // tokens of a page: one MSA block

// The workspace's head: the status word, then the attention's arrival counts, zero between its calls.  No other call writes
// there, so that the calls may share a workspace.
constexpr size_t kHeadBytes = 4096;

struct PagedProblem {
    int R, T, max_blocks, n_pages, Hq, Hkv, G, d, d_idx, topk;
    float scale, scale_idx;
    int num_sms;
};

// Entries of a plan's segment list: a request of n new tokens touches at most
// 2 + n/128 pages and at most n of them.
inline int paged_segments(const PagedProblem &p)
{
    const long long s = 2LL * p.R + p.T / kPage;
    return s < p.T ? (int)s : p.T;
}

// The least power of two s with amax <= 448 s (448: the largest e4m3 value),
// at least 2^-112, as fp32 bits, from the bits of |amax| in bf16: with
// amax = m 2^x, m in [1, 2), s = 2^(x-8) when m <= 1.75 and 2^(x-7) above.
__host__ __device__ __forceinline__ uint32_t pow2_scale_bits(uint32_t abs_bf16)
{
    int e = (int)(abs_bf16 >> 7) - 127 - 8 + ((abs_bf16 & 0x7Fu) > 0x60u ? 1 : 0);
    if (abs_bf16 == 0 || e < -112) e = -112;
    return (uint32_t)(e + 127) << 23;
}

// 3-D byte TMA tensor map (dims innermost first), box {box0, box1, 1}, with a
// 128-byte (box0 = 128) or 64-byte (box0 = 64) swizzle, zero fill out of bounds.
cudaError_t make_tmap_u8_3d(CUtensorMap *map, const void *base, unsigned long long d0, unsigned long long d1,
                            unsigned long long d2, unsigned box0, unsigned box1);

// The paged kernels follow one another in a step, each a few microseconds to a
// few tens, so each may be set up while its predecessor still runs: it is
// launched with programmatic stream serialisation, lets its own successor be
// set up in turn (chain_next) and waits for the predecessor's end, its writes
// visible, before it touches global memory (chain_wait).  After any other
// kernel this is an ordinary launch.
// The pointers given take on new values, as far as the compiler can tell, so that no load through them
// (loads of const __restrict__ data may pass a memory clobber) is moved above the wait.
template <class... P>
MSA_DEV void chain_wait(P &...ptrs)
{
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    auto renew = [](auto &p) { asm volatile("" : "+l"(p)::"memory"); };
    (renew(ptrs), ...);
}
MSA_DEV void chain_next() { asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory"); }

template <class... P, class... A>
cudaError_t launch_chained(const char *name, void (*kernel)(P...), dim3 grid, int threads, int smem, cudaStream_t s, A &&...args)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    TimedLaunch timed_(name, s);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
    if (e == cudaSuccess) note_launch();
    else cudaGetLastError();                 // reported by this call: not left for the next one to find
    return e;
}

// Allows `bytes` of dynamic shared memory for a kernel, once per device (`done`: the kernel's own).
template <class K>
cudaError_t allow_smem(K *kernel, int bytes, std::atomic<unsigned long long> &done)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = dev >= 0 && dev < 64 ? 1ull << dev : 0;
    if (bit & done.load(std::memory_order_acquire)) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && bit) done.fetch_or(bit, std::memory_order_release);
    if (e != cudaSuccess) cudaGetLastError();
    return e;
}

struct PlanArgs {
    const int32_t *new_lens, *lens_in, *ended, *free_in;
    int32_t *held, *block_table, *free_pages, *lens_out, *free_out, *q_starts, *row_req, *row_pos, *slots, *segs;
};
size_t paged_plan_scratch_ints(const PagedProblem &p);
cudaError_t launch_paged_plan(const PagedProblem &p, const PlanArgs &a, int32_t *scratch, DeviceStatus *st, cudaStream_t s);

cudaError_t launch_paged_append(const PagedProblem &p, const bf16 *k_new, const bf16 *v_new, const bf16 *ki_new,
                                const int32_t *slots, const int32_t *segs, uint8_t *k8, uint8_t *v8, float *k_scale,
                                float *v_scale, bf16 *k_idx, DeviceStatus *st, cudaStream_t s);

cudaError_t launch_paged_block_scores(const PagedProblem &p, const bf16 *q_idx, const bf16 *k_idx,
                                      const int32_t *block_table, const int32_t *q_starts, const int32_t *row_req,
                                      const int32_t *row_pos, float *scores, DeviceStatus *st, cudaStream_t s);

cudaError_t launch_paged_block_topk(const PagedProblem &p, const float *scores, const int32_t *row_pos, int32_t *sel,
                                    DeviceStatus *st, cudaStream_t s);

// Floats of partial outputs and (max, sum) pairs, for either form (with a
// selection and without).
size_t paged_attn_scratch_floats(const PagedProblem &p);
cudaError_t launch_paged_attn(const PagedProblem &p, const bf16 *q, const uint8_t *k8, const uint8_t *v8,
                              const float *k_scale, const float *v_scale, const int32_t *block_table,
                              const int32_t *row_req, const int32_t *row_pos, const int32_t *sel, bf16 *o, float *lse,
                              float *scratch, DeviceStatus *st, cudaStream_t s);

struct ForkArgs {
    const int32_t *src, *fork_lens;
    int32_t *lens, *held, *block_table, *free_pages, *free_state, *shares, *moves;
};
size_t paged_fork_scratch_bytes(const PagedProblem &p);
cudaError_t launch_paged_fork(const PagedProblem &p, const ForkArgs &a, void *scratch, DeviceStatus *st, cudaStream_t s);

struct CompactArgs {
    const int32_t *lens, *held, *block_table, *shares;
    int32_t *block_table_out, *free_pages, *free_state, *shares_out, *moves;
};
size_t paged_compact_scratch_bytes(const PagedProblem &p);
cudaError_t launch_paged_compact(const PagedProblem &p, const CompactArgs &a, void *scratch, DeviceStatus *st, cudaStream_t s);

cudaError_t launch_paged_copy(const PagedProblem &p, const int32_t *moves, int n_moves, uint8_t *k8, uint8_t *v8, float *k_scale,
                              float *v_scale, bf16 *k_idx, DeviceStatus *st, cudaStream_t s);

// Chunks of new tokens (paged_chunk.cu): scratch bytes of the tiles' plan, and for attention of the cut tiles' states.
size_t paged_chunk_scratch_bytes(const PagedProblem &p, bool attention);
cudaError_t launch_paged_chunk_scores(const PagedProblem &p, const bf16 *q_idx, const bf16 *k_idx, const int32_t *block_table,
                                      const int32_t *q_starts, const int32_t *row_pos, float *scores, void *scratch, DeviceStatus *st,
                                      cudaStream_t s);
cudaError_t launch_paged_chunk_attn(const PagedProblem &p, const bf16 *q, const uint8_t *k8, const uint8_t *v8, const float *k_scale,
                                    const float *v_scale, const int32_t *block_table, const int32_t *q_starts, const int32_t *row_pos,
                                    const int32_t *sel, bf16 *o, float *lse, void *scratch, DeviceStatus *st, cudaStream_t s);

// Rotary positions (rotary.cu).
struct RotaryProblem {
    int T, Hq, Hkv, d, d_rot, period, offset, num_sms, zeros;
    bool interleaved, backward;
    float scale;
    long long q_stride, k_stride, q_out_stride, k_out_stride;
};
cudaError_t launch_rotary(const RotaryProblem &p, const bf16 *q, const bf16 *k, const int32_t *positions,
                          const unsigned long long *freqs, bf16 *q_out, bf16 *k_out, cudaStream_t s);

}  // namespace msa
