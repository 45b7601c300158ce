// paged_api.cu -- the C-ABI of the paged-cache operators (declared in
// include/msa.h): argument validation, workspace carve-up, launches.
#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include <algorithm>
#include <atomic>

#include "msa.h"
#include "paged.h"

namespace msa {
msa_status set_error(msa_status st, const char *msg);
}

using namespace msa;

namespace {

msa_status refuse(msa_status st, const char *fmt, ...)
{
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    return set_error(st, buf);
}

// SMs of the current device (asked for once per device).
int current_sms()
{
    static std::atomic<int> known[64];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 148;
    const bool keep = dev >= 0 && dev < 64;
    if (keep && (n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return 148;
    if (keep) known[dev].store(n, std::memory_order_relaxed);
    return n;
}

msa_status make_paged(const msa_paged_shape *s, PagedProblem &p)
{
    if (!s) return refuse(MSA_ERR_INVALID_ARGUMENT, "shape is NULL");
    if (s->R < 1 || s->T < 1 || s->max_blocks < 1 || s->n_pages < 1 || s->Hq < 1 || s->Hkv < 1 || s->d < 1 ||
        s->d_idx < 1 || s->topk < 1)
        return refuse(MSA_ERR_INVALID_ARGUMENT, "paged shape has a non-positive size (R=%d T=%d max_blocks=%d n_pages=%d "
                      "Hq=%d Hkv=%d d=%d d_idx=%d topk=%d)", s->R, s->T, s->max_blocks, s->n_pages, s->Hq, s->Hkv, s->d,
                      s->d_idx, s->topk);
    if (s->Hq % s->Hkv != 0) return refuse(MSA_ERR_INVALID_ARGUMENT, "Hq (%d) is not a multiple of Hkv (%d)", s->Hq, s->Hkv);
    const int G = s->Hq / s->Hkv;
    if (G != 1 && G != 2 && G != 4 && G != 8) return refuse(MSA_ERR_UNSUPPORTED, "Hq/Hkv must be 1, 2, 4 or 8 (got %d)", G);
    if (s->d != 64 && s->d != 128) return refuse(MSA_ERR_UNSUPPORTED, "d must be 64 or 128 (got %d)", s->d);
    if (s->d_idx != 64 && s->d_idx != 128) return refuse(MSA_ERR_UNSUPPORTED, "d_idx must be 64 or 128 (got %d)", s->d_idx);
    if (s->topk > 32) return refuse(MSA_ERR_UNSUPPORTED, "topk must be <= 32 (got %d)", s->topk);
    if (!(s->scale >= 0.f) || !(s->scale_idx >= 0.f) || isinf(s->scale) || isinf(s->scale_idx))
        return refuse(MSA_ERR_INVALID_ARGUMENT, "scales must be finite and >= 0 (0 selects the default)");
    // positions, slots and (page, head) tiles are 32-bit integers; grids hold (row, head, share)
    if (s->max_blocks > (1 << 23) || s->n_pages > (1 << 23) || s->R > (1 << 24) || s->Hkv > 32768 ||
        (long long)s->n_pages * s->Hkv >= (1LL << 31) || (long long)s->T * s->Hq >= (1LL << 24))
        return refuse(MSA_ERR_UNSUPPORTED, "problem too large (max_blocks, n_pages <= 2^23, R <= 2^24, Hkv <= 32768, "
                      "n_pages * Hkv < 2^31, T * Hq < 2^24)");
    p.R = s->R; p.T = s->T; p.max_blocks = s->max_blocks; p.n_pages = s->n_pages;
    p.Hq = s->Hq; p.Hkv = s->Hkv; p.G = G; p.d = s->d; p.d_idx = s->d_idx; p.topk = s->topk;
    p.scale = s->scale > 0.f ? s->scale : 1.0f / sqrtf((float)s->d);
    p.scale_idx = s->scale_idx > 0.f ? s->scale_idx : 1.0f / sqrtf((float)s->d_idx);
    p.num_sms = current_sms();
    return MSA_OK;
}

size_t scratch_bytes(const PagedProblem &p, int op)
{
    switch (op) {
    case MSA_OP_PAGED_PLAN: return kHeadBytes - kStatusBytes + paged_plan_scratch_ints(p) * 4;
    case MSA_OP_PAGED_ATTN: return paged_attn_scratch_floats(p) * 4;
    case MSA_OP_PAGED_FORK: return kHeadBytes - kStatusBytes + paged_fork_scratch_bytes(p);
    case MSA_OP_PAGED_COMPACT: return kHeadBytes - kStatusBytes + paged_compact_scratch_bytes(p);
    case MSA_OP_PAGED_CHUNK_SCORES: return kHeadBytes - kStatusBytes + paged_chunk_scratch_bytes(p, false);
    case MSA_OP_PAGED_CHUNK_ATTN: return kHeadBytes - kStatusBytes + paged_chunk_scratch_bytes(p, true);
    default: return 0;
    }
}

// Shape, workspace and its size, common to the calls.
msa_status begin(const msa_paged_shape *shape, int op, void *ws, size_t ws_bytes, PagedProblem &p)
{
    const msa_status st = make_paged(shape, p);
    if (st != MSA_OK) return st;
    if (!ws) return refuse(MSA_ERR_INVALID_ARGUMENT, "workspace is NULL");
    if (((uintptr_t)ws & 255u) != 0) return refuse(MSA_ERR_INVALID_ARGUMENT, "workspace is not 256-byte aligned");
    const size_t need = kStatusBytes + scratch_bytes(p, op);
    if (ws_bytes < need) return refuse(MSA_ERR_WORKSPACE, "workspace too small: %zu < %zu bytes", ws_bytes, need);
    return MSA_OK;
}

struct Arg {
    const void *ptr;
    const char *name;
    unsigned align;
};
template <size_t N>
msa_status check(const Arg (&args)[N])
{
    for (const Arg &a : args) {
        if (!a.ptr) return refuse(MSA_ERR_INVALID_ARGUMENT, "%s is NULL", a.name);
        if ((uintptr_t)a.ptr % a.align) return refuse(MSA_ERR_INVALID_ARGUMENT, "%s is not %u-byte aligned", a.name, a.align);
    }
    return MSA_OK;
}

msa_status done(cudaError_t e, const char *what)
{
    return e == cudaSuccess ? MSA_OK : refuse(MSA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

msa_status optional4(const void *ptr, const char *name)
{
    return (uintptr_t)ptr % 4 ? refuse(MSA_ERR_INVALID_ARGUMENT, "%s is not 4-byte aligned", name) : MSA_OK;
}

void *behind_head(void *ws) { return static_cast<char *>(ws) + kHeadBytes; }

DeviceStatus *status(void *ws) { return static_cast<DeviceStatus *>(ws); }
const bf16 *b16(const void *x) { return static_cast<const bf16 *>(x); }

}  // namespace

extern "C" {

size_t msa_paged_workspace_size(const msa_paged_shape *shape, int op)
{
    PagedProblem p;
    if (make_paged(shape, p) != MSA_OK) return 0;
    if (op < MSA_OP_PAGED_PLAN || (op > MSA_OP_PAGED_ATTN && op < MSA_OP_PAGED_FORK) || op > MSA_OP_PAGED_CHUNK_ATTN) {
        refuse(MSA_ERR_INVALID_ARGUMENT, "unknown paged op %d", op);
        return 0;
    }
    return kStatusBytes + (scratch_bytes(p, op) + 255) / 256 * 256;
}

msa_status msa_paged_plan(const msa_paged_shape *shape, const int32_t *new_lens, const int32_t *lens_in,
                          const int32_t *ended, int32_t *block_table, int32_t *free_pages, const int32_t *free_in,
                          int32_t *lens_out, int32_t *free_out, int32_t *q_starts, int32_t *row_req, int32_t *row_pos,
                          int32_t *slots, int32_t *segs, void *workspace, size_t workspace_bytes, void *stream)
{
    return msa_paged_plan_held(shape, new_lens, lens_in, ended, nullptr, block_table, free_pages, free_in, lens_out, free_out,
                               q_starts, row_req, row_pos, slots, segs, workspace, workspace_bytes, stream);
}

msa_status msa_paged_plan_held(const msa_paged_shape *shape, const int32_t *new_lens, const int32_t *lens_in,
                               const int32_t *ended, int32_t *held, int32_t *block_table, int32_t *free_pages,
                               const int32_t *free_in, int32_t *lens_out, int32_t *free_out, int32_t *q_starts,
                               int32_t *row_req, int32_t *row_pos, int32_t *slots, int32_t *segs, void *workspace,
                               size_t workspace_bytes, void *stream)
{
    PagedProblem p;
    msa_status st = begin(shape, MSA_OP_PAGED_PLAN, workspace, workspace_bytes, p);
    if (st != MSA_OK) return st;
    st = check({{new_lens, "new_lens", 4}, {lens_in, "lens_in", 4}, {block_table, "block_table", 4},
                {free_pages, "free_pages", 4}, {free_in, "free_in", 4}, {lens_out, "lens_out", 4},
                {free_out, "free_out", 4}, {q_starts, "q_starts", 4}, {row_req, "row_req", 4}, {row_pos, "row_pos", 4},
                {slots, "slots", 4}, {segs, "segs", 4}});
    if (st != MSA_OK) return st;
    if ((uintptr_t)ended % 4) return refuse(MSA_ERR_INVALID_ARGUMENT, "ended is not 4-byte aligned");
    if ((uintptr_t)held % 4) return refuse(MSA_ERR_INVALID_ARGUMENT, "held is not 4-byte aligned");
    const PlanArgs a{new_lens, lens_in, ended, free_in, held, block_table, free_pages, lens_out, free_out, q_starts, row_req,
                     row_pos, slots, segs};
    int32_t *scratch = reinterpret_cast<int32_t *>(static_cast<char *>(workspace) + kHeadBytes);
    return done(launch_paged_plan(p, a, scratch, status(workspace), static_cast<cudaStream_t>(stream)),
                "paged_plan launch");
}

msa_status msa_paged_append(const msa_paged_shape *shape, const void *k_new, const void *v_new, const void *k_idx_new,
                            const int32_t *slots, const int32_t *segs, void *k8, void *v8, float *k_scale, float *v_scale,
                            void *k_idx, void *workspace, size_t workspace_bytes, void *stream)
{
    PagedProblem p;
    msa_status st = begin(shape, MSA_OP_PAGED_APPEND, workspace, workspace_bytes, p);
    if (st != MSA_OK) return st;
    st = check({{slots, "slots", 4}, {segs, "segs", 4}});
    if (st != MSA_OK) return st;
    const bool kv = k_new || v_new || k8 || v8 || k_scale || v_scale, ki = k_idx_new || k_idx;
    if (!kv && !ki) return refuse(MSA_ERR_INVALID_ARGUMENT, "nothing to append: every pair is NULL");
    if (kv) {
        st = check({{k_new, "k_new", 16}, {v_new, "v_new", 16}, {k8, "k8", 16}, {v8, "v8", 16}, {k_scale, "k_scale", 4},
                    {v_scale, "v_scale", 4}});
        if (st != MSA_OK) return st;
    }
    if (ki) {
        st = check({{k_idx_new, "k_idx_new", 16}, {k_idx, "k_idx", 16}});
        if (st != MSA_OK) return st;
    }
    return done(launch_paged_append(p, b16(k_new), b16(v_new), b16(k_idx_new), slots, segs, static_cast<uint8_t *>(k8),
                                    static_cast<uint8_t *>(v8), k_scale, v_scale, static_cast<bf16 *>(k_idx),
                                    status(workspace), static_cast<cudaStream_t>(stream)),
                "paged_append launch");
}

msa_status msa_paged_block_scores(const msa_paged_shape *shape, const void *q_idx, const void *k_idx,
                                  const int32_t *block_table, const int32_t *q_starts, const int32_t *row_req,
                                  const int32_t *row_pos, float *block_scores, void *workspace, size_t workspace_bytes,
                                  void *stream)
{
    PagedProblem p;
    msa_status st = begin(shape, MSA_OP_PAGED_BLOCK_SCORES, workspace, workspace_bytes, p);
    if (st != MSA_OK) return st;
    st = check({{q_idx, "q_idx", 16}, {k_idx, "k_idx", 16}, {block_table, "block_table", 4}, {q_starts, "q_starts", 4},
                {row_req, "row_req", 4}, {row_pos, "row_pos", 4}, {block_scores, "block_scores", 4}});
    if (st != MSA_OK) return st;
    return done(launch_paged_block_scores(p, b16(q_idx), b16(k_idx), block_table, q_starts, row_req, row_pos, block_scores,
                                          status(workspace), static_cast<cudaStream_t>(stream)),
                "paged_block_scores launch");
}

msa_status msa_paged_block_topk(const msa_paged_shape *shape, const float *block_scores, const int32_t *row_pos,
                                int32_t *sel_idx, void *workspace, size_t workspace_bytes, void *stream)
{
    PagedProblem p;
    msa_status st = begin(shape, MSA_OP_PAGED_BLOCK_TOPK, workspace, workspace_bytes, p);
    if (st != MSA_OK) return st;
    st = check({{block_scores, "block_scores", 4}, {row_pos, "row_pos", 4}, {sel_idx, "sel_idx", 4}});
    if (st != MSA_OK) return st;
    return done(launch_paged_block_topk(p, block_scores, row_pos, sel_idx, status(workspace), static_cast<cudaStream_t>(stream)),
                "paged_block_topk launch");
}

msa_status msa_paged_attn(const msa_paged_shape *shape, const void *q, const void *k8, const void *v8, const float *k_scale,
                          const float *v_scale, const int32_t *block_table, const int32_t *row_req, const int32_t *row_pos,
                          const int32_t *sel_idx, void *o, float *lse, void *workspace, size_t workspace_bytes,
                          void *stream)
{
    PagedProblem p;
    msa_status st = begin(shape, MSA_OP_PAGED_ATTN, workspace, workspace_bytes, p);
    if (st != MSA_OK) return st;
    st = check({{q, "q", 16}, {k8, "k8", 16}, {v8, "v8", 16}, {k_scale, "k_scale", 4}, {v_scale, "v_scale", 4},
                {block_table, "block_table", 4}, {row_req, "row_req", 4}, {row_pos, "row_pos", 4}, {o, "o", 16},
                {lse, "lse", 4}});
    if (st != MSA_OK) return st;
    if ((uintptr_t)sel_idx % 4) return refuse(MSA_ERR_INVALID_ARGUMENT, "sel_idx is not 4-byte aligned");
    return done(launch_paged_attn(p, b16(q), static_cast<const uint8_t *>(k8), static_cast<const uint8_t *>(v8), k_scale,
                                  v_scale, block_table, row_req, row_pos, sel_idx, static_cast<bf16 *>(o), lse,
                                  reinterpret_cast<float *>(static_cast<char *>(workspace) + kStatusBytes), status(workspace),
                                  static_cast<cudaStream_t>(stream)),
                "paged_attn launch");
}

msa_status msa_paged_fork(const msa_paged_shape *shape, const int32_t *src, const int32_t *fork_lens, int32_t *lens,
                          int32_t *held, int32_t *block_table, int32_t *free_pages, int32_t *free_state, int32_t *shares,
                          int32_t *moves, void *workspace, size_t workspace_bytes, void *stream)
{
    PagedProblem p;
    msa_status st = begin(shape, MSA_OP_PAGED_FORK, workspace, workspace_bytes, p);
    if (st != MSA_OK) return st;
    st = check({{src, "src", 4}, {lens, "lens", 4}, {block_table, "block_table", 4}, {free_pages, "free_pages", 4},
                {free_state, "free_state", 4}, {shares, "shares", 4}, {moves, "moves", 4}});
    if (st != MSA_OK || (st = optional4(fork_lens, "fork_lens")) != MSA_OK || (st = optional4(held, "held")) != MSA_OK) return st;
    const ForkArgs a{src, fork_lens, lens, held, block_table, free_pages, free_state, shares, moves};
    return done(launch_paged_fork(p, a, behind_head(workspace), status(workspace), static_cast<cudaStream_t>(stream)),
                "paged_fork launch");
}

msa_status msa_paged_compact(const msa_paged_shape *shape, const int32_t *lens, const int32_t *held, const int32_t *block_table,
                             const int32_t *shares, int32_t *block_table_out, int32_t *free_pages, int32_t *free_state,
                             int32_t *shares_out, int32_t *moves, void *workspace, size_t workspace_bytes, void *stream)
{
    PagedProblem p;
    msa_status st = begin(shape, MSA_OP_PAGED_COMPACT, workspace, workspace_bytes, p);
    if (st != MSA_OK) return st;
    st = check({{lens, "lens", 4}, {block_table, "block_table", 4}, {block_table_out, "block_table_out", 4},
                {free_pages, "free_pages", 4}, {free_state, "free_state", 4}, {moves, "moves", 4}});
    if (st != MSA_OK || (st = optional4(held, "held")) != MSA_OK || (st = optional4(shares, "shares")) != MSA_OK ||
        (st = optional4(shares_out, "shares_out")) != MSA_OK)
        return st;
    if (!shares != !shares_out) return refuse(MSA_ERR_INVALID_ARGUMENT, "one of shares and shares_out is NULL");
    const CompactArgs a{lens, held, block_table, shares, block_table_out, free_pages, free_state, shares_out, moves};
    return done(launch_paged_compact(p, a, behind_head(workspace), status(workspace), static_cast<cudaStream_t>(stream)),
                "paged_compact launch");
}

msa_status msa_paged_copy(const msa_paged_shape *shape, const int32_t *moves, int n_moves, void *k8, void *v8, float *k_scale,
                          float *v_scale, void *k_idx, void *workspace, size_t workspace_bytes, void *stream)
{
    PagedProblem p;
    msa_status st = begin(shape, MSA_OP_PAGED_COPY, workspace, workspace_bytes, p);
    if (st != MSA_OK) return st;
    st = check({{moves, "moves", 4}});
    if (st != MSA_OK) return st;
    if (n_moves < 1 || n_moves > (1 << 24)) return refuse(MSA_ERR_INVALID_ARGUMENT, "n_moves must be 1..2^24 (got %d)", n_moves);
    const bool kv = k8 || v8 || k_scale || v_scale;
    if (!kv && !k_idx) return refuse(MSA_ERR_INVALID_ARGUMENT, "nothing to copy: every cache is NULL");
    if (kv) {
        st = check({{k8, "k8", 16}, {v8, "v8", 16}, {k_scale, "k_scale", 4}, {v_scale, "v_scale", 4}});
        if (st != MSA_OK) return st;
    }
    if ((uintptr_t)k_idx % 16) return refuse(MSA_ERR_INVALID_ARGUMENT, "k_idx is not 16-byte aligned");
    return done(launch_paged_copy(p, moves, n_moves, static_cast<uint8_t *>(k8), static_cast<uint8_t *>(v8), k_scale, v_scale,
                                  static_cast<bf16 *>(k_idx), status(workspace), static_cast<cudaStream_t>(stream)),
                "paged_copy launch");
}

msa_status msa_paged_chunk_scores(const msa_paged_shape *shape, const void *q_idx, const void *k_idx, const int32_t *block_table,
                                  const int32_t *q_starts, const int32_t *row_pos, float *block_scores, void *workspace,
                                  size_t workspace_bytes, void *stream)
{
    PagedProblem p;
    msa_status st = begin(shape, MSA_OP_PAGED_CHUNK_SCORES, workspace, workspace_bytes, p);
    if (st != MSA_OK) return st;
    st = check({{q_idx, "q_idx", 16}, {k_idx, "k_idx", 16}, {block_table, "block_table", 4}, {q_starts, "q_starts", 4},
                {row_pos, "row_pos", 4}, {block_scores, "block_scores", 4}});
    if (st != MSA_OK) return st;
    return done(launch_paged_chunk_scores(p, b16(q_idx), b16(k_idx), block_table, q_starts, row_pos, block_scores,
                                          behind_head(workspace), status(workspace), static_cast<cudaStream_t>(stream)),
                "paged_chunk_scores launch");
}

msa_status msa_paged_chunk_attn(const msa_paged_shape *shape, const void *q, const void *k8, const void *v8, const float *k_scale,
                                const float *v_scale, const int32_t *block_table, const int32_t *q_starts, const int32_t *row_pos,
                                const int32_t *sel_idx, void *o, float *lse, void *workspace, size_t workspace_bytes,
                                void *stream)
{
    PagedProblem p;
    msa_status st = begin(shape, MSA_OP_PAGED_CHUNK_ATTN, workspace, workspace_bytes, p);
    if (st != MSA_OK) return st;
    st = check({{q, "q", 16}, {k8, "k8", 16}, {v8, "v8", 16}, {k_scale, "k_scale", 4}, {v_scale, "v_scale", 4},
                {block_table, "block_table", 4}, {q_starts, "q_starts", 4}, {row_pos, "row_pos", 4}, {o, "o", 16}, {lse, "lse", 4}});
    if (st != MSA_OK || (st = optional4(sel_idx, "sel_idx")) != MSA_OK) return st;
    return done(launch_paged_chunk_attn(p, b16(q), static_cast<const uint8_t *>(k8), static_cast<const uint8_t *>(v8), k_scale, v_scale,
                                        block_table, q_starts, row_pos, sel_idx, static_cast<bf16 *>(o), lse, behind_head(workspace),
                                        status(workspace), static_cast<cudaStream_t>(stream)),
                "paged_chunk_attn launch");
}

namespace {

msa_status rotary(const msa_rotary_shape *s, bool backward, const void *q, const void *k, const int32_t *positions,
                  const unsigned long long *freqs, void *q_out, void *k_out, void *stream)
{
    if (!s) return refuse(MSA_ERR_INVALID_ARGUMENT, "shape is NULL");
    if (s->T < 1 || s->Hq < 1 || s->Hkv < 1 || s->d < 1 || s->d_rot < 1 || s->period < 0 || s->offset < 0 || s->q_stride < 0 ||
        s->k_stride < 0 || s->q_out_stride < 0 || s->k_out_stride < 0)
        return refuse(MSA_ERR_INVALID_ARGUMENT, "rotary shape has a size out of range (T=%d Hq=%d Hkv=%d d=%d d_rot=%d period=%d "
                      "offset=%d)", s->T, s->Hq, s->Hkv, s->d, s->d_rot, s->period, s->offset);
    if (s->d_rot > s->d) return refuse(MSA_ERR_INVALID_ARGUMENT, "d_rot (%d) is larger than d (%d)", s->d_rot, s->d);
    if (!(s->scale >= 0.f) || isinf(s->scale)) return refuse(MSA_ERR_INVALID_ARGUMENT, "scale must be finite and >= 0 (0 selects 1)");
    if (s->zeros < 0 || s->zeros > 3) return refuse(MSA_ERR_INVALID_ARGUMENT, "zeros must be 0..3 (got %d)", s->zeros);
    if (s->d % 16 || s->d > 256) return refuse(MSA_ERR_UNSUPPORTED, "d must be a multiple of 16 up to 256 (got %d)", s->d);
    if (s->d_rot % 16) return refuse(MSA_ERR_UNSUPPORTED, "d_rot must be a multiple of 16 (got %d)", s->d_rot);
    if (s->Hq > 32768 || s->Hkv > 32768) return refuse(MSA_ERR_UNSUPPORTED, "Hq and Hkv must be <= 32768 (got %d, %d)", s->Hq, s->Hkv);
    RotaryProblem p;
    p.T = s->T; p.Hq = q ? s->Hq : 0; p.Hkv = k ? s->Hkv : 0; p.d = s->d; p.d_rot = s->d_rot;
    p.period = s->period ? s->period : s->T; p.offset = s->offset; p.num_sms = current_sms();
    p.interleaved = s->interleaved != 0; p.backward = backward; p.zeros = s->zeros;
    p.scale = s->scale > 0.f ? s->scale : 1.f;
    if (!positions && (long long)p.offset + p.period > (1LL << 31)) return refuse(MSA_ERR_INVALID_ARGUMENT, "positions pass 2^31 - 1");
    auto stride = [&](long long given, int heads) { return given ? given : (long long)heads * s->d; };
    p.q_stride = stride(s->q_stride, s->Hq); p.k_stride = stride(s->k_stride, s->Hkv);
    p.q_out_stride = stride(s->q_out_stride, s->Hq); p.k_out_stride = stride(s->k_out_stride, s->Hkv);
    auto bad = [&](long long st, int heads) { return st % 8 || st < (long long)heads * s->d || st > (1LL << 31); };
    if (bad(p.q_stride, s->Hq) || bad(p.q_out_stride, s->Hq) || bad(p.k_stride, s->Hkv) || bad(p.k_out_stride, s->Hkv))
        return refuse(MSA_ERR_INVALID_ARGUMENT, "strides must be multiples of 8, no less than a token's heads, at most 2^31");
    if (!q && !k && !q_out && !k_out) return refuse(MSA_ERR_INVALID_ARGUMENT, "nothing to turn: both pairs are NULL");
    msa_status st = check({{freqs, "freqs", 8}});
    if (st == MSA_OK && (q || q_out)) st = check({{q, "q", 16}, {q_out, "q_out", 16}});
    if (st == MSA_OK && (k || k_out)) st = check({{k, "k", 16}, {k_out, "k_out", 16}});
    if (st != MSA_OK || (st = optional4(positions, "positions")) != MSA_OK) return st;
    if ((q && q == q_out && p.q_stride != p.q_out_stride) || (k && k == k_out && p.k_stride != p.k_out_stride))
        return refuse(MSA_ERR_INVALID_ARGUMENT, "an output in its input's place has another stride");
    if ((q && q == q_out && (s->zeros & 1)) || (k && k == k_out && (s->zeros & 2)))
        return refuse(MSA_ERR_INVALID_ARGUMENT, "zeros for an output in its input's place");
    return done(launch_rotary(p, b16(q), b16(k), positions, freqs, static_cast<bf16 *>(q_out), static_cast<bf16 *>(k_out),
                              static_cast<cudaStream_t>(stream)),
                "rotary launch");
}

}  // namespace

msa_status msa_rotary_fwd(const msa_rotary_shape *shape, const void *q, const void *k, const int32_t *positions,
                          const unsigned long long *freqs, void *q_out, void *k_out, void *stream)
{
    return rotary(shape, false, q, k, positions, freqs, q_out, k_out, stream);
}

msa_status msa_rotary_bwd(const msa_rotary_shape *shape, const void *dq_out, const void *dk_out, const int32_t *positions,
                          const unsigned long long *freqs, void *dq, void *dk, void *stream)
{
    return rotary(shape, true, dq_out, dk_out, positions, freqs, dq, dk, stream);
}

}  // extern "C"
