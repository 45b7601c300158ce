// paged_chunk.h -- the tiles that chunks of new tokens are cut into, shared by
// the chunk calls' kernels (paged_chunk.cu, paged_chunk_attn.cu).
#pragma once

#include "paged.h"

namespace msa {

// Up to `tokens` consecutive rows of one request.
struct ChunkTile {
    int row, rows, req, pages;      // first row, rows, request; pages that its furthest row sees
};

constexpr int kTileRows = 256;      // (row, head) pairs of a tile: two products of 128 rows

// Products that a page costs a tile of `pairs` pairs.
__host__ __device__ __forceinline__ int tile_halves(int pairs) { return pairs > kTileRows / 2 ? 2 : 1; }

// The plan: the number of tiles and whether any request was left out, the tiles in the order of rows, and the work of those before each (one more than
// tiles), in products: pages x halves.
struct ChunkPlan {
    int *n_tiles;
    ChunkTile *tiles;
    long long *before;
    __host__ __device__ ChunkPlan(void *at, long long most)
    {
        n_tiles = static_cast<int *>(at);
        tiles = reinterpret_cast<ChunkTile *>(n_tiles + 4);
        before = reinterpret_cast<long long *>(tiles + most);
    }
    static size_t bytes(long long most) { return (size_t)(16 + most * sizeof(ChunkTile) + (most + 1) * 8 + 255) / 256 * 256; }
};

// Tiles of `tokens` rows that T rows of R requests make at most.
inline long long chunk_tiles(const PagedProblem &p, int tokens)
{
    const long long whole = p.T / tokens, any = p.T;
    return whole + p.R < any ? whole + p.R : any;
}

// pairs: those of a token.
cudaError_t launch_chunk_plan(const PagedProblem &p, const int32_t *q_starts, const int32_t *row_pos, int tokens, int pairs, void *plan,
                              DeviceStatus *st, cudaStream_t s);

// The stretch of CTA `cta`: work units [from, to) of `total`.
struct ChunkShare {
    long long share, from, to;
    __host__ __device__ ChunkShare(long long total, int ctas, int least, int cta)
    {
        share = (total + ctas - 1) / ctas;
        if (share < least) share = least;
        from = share * cta < total ? share * cta : total;
        to = from + share < total ? from + share : total;
    }
};

// The last i < n with before[i] * scale <= w, by a whole warp (before[0] = 0 <= w).
MSA_DEV int chunk_find(const long long *before, int n, long long scale, long long w, int lane)
{
    int lo = 0;
    while (n - lo > 1) {
        const int step = (n - lo + 31) / 32;
        const int i = lo + lane * step;
        const unsigned in = __ballot_sync(0xffffffffu, i < n && before[i] * scale <= w);
        const int last = 31 - __clz(in);                 // lane 0's is always in
        lo += last * step;
        n = min(n, lo + step);
    }
    return lo;
}

}  // namespace msa
