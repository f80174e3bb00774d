// Low-rank adapters beside a shared projection: arguments of the kernels in
// sam_kernels_adapter.hip and sam_kernels_adapter_ring.hip, and their
// launchers.
//
//   Y[m] = X[m] W + scale[a] (X[m] A[a]^T) B[a],   a = ids[m]
//
// The rank-r intermediate of a row, T[m] = scale[a] X[m] A[a]^T, is made
// first (shrink). Where the product's tiles fill the machine, the tile's own
// kernel starts its accumulators at T[m] B[a] and runs the K loop on top, so
// Y is written once and never read; where they do not, K is split over
// workgroups and the pass that sums the partials adds T[m] B[a] (finish).
#pragma once

#include "sam_internal.h"

namespace sam {

constexpr int kMaxRank = 128;

// One shrink: rows of T from rows of X (stride ldx) and the adapters' r rows
// of K values. The backward pass runs two (X with A, dY with B).
struct ShrinkSide {
    const void* X;
    long long ldx;
    const void* A;       // [n][r] rows, row stride lda
    long long lda;
    int K;
    float* t32;          // [ksplit][M][rp]: partial sums over K of the scaled T
    // What a second kernel makes of them (with `round`):
    int keep;            // their sum goes to the first of them
    void* t16;           // [M][np][rp]: T / factor as np values of the operands' type that add up to it, or null
    float* factor;       // [M]: the power of two that t16 was divided by, or null
};

struct ShrinkArgs {
    ShrinkSide side[2];
    int sides;
    int M, n, r, rp;     // rp = r rounded up to 16, 32, 64 or 128
    const int* ids;
    const float* scale;  // [n] or null (1)
    int np;              // 2, or 3 (bfloat16: then the values are exactly T)
    int wide;            // 64 rows a workgroup, else 16 rows x 16 ranks
    int round;
    int ksplit;          // K ranges, a workgroup each
    int slots;           // workgroups sharing the distinct adapters of a row block
    // Grouping of rows by adapter, done by n further workgroups (backward):
    int* order;          // [M] rows sorted by adapter, in row order inside one; null: no grouping
    int* seg;            // [n + 1] where each adapter's rows start in it
    // ... and chunks of its rows, listed by the second kernel:
    int chunk;           // rows per chunk
    int max_chunks;      // ceil(M / chunk) + n
    int* chunk_first;    // [n + 1] each adapter's first chunk
    int* part_first;     // [n] ... and its first place among the partials, which adapters with several chunks have
    int4* chunks;        // [max_chunks] adapter (-1: no such chunk), place in `order`, rows, first row of a run or -1
};

// Whether the shrink rounds T itself: there is nothing left to add up.
__host__ __device__ inline bool shrink_rounds(const ShrinkArgs& a) { return a.wide && a.ksplit == 1; }

// Sum of the split partials of X W plus T B.
struct FinishArgs {
    const float* part;   // [split][M] rows of N floats, row stride ldp (a multiple of 4)
    long long ldp;
    int split;
    const float* t32;    // [tsplit][M][rp]
    int tsplit;
    const void* B;       // [n][r] rows of N values, row stride ldb
    long long ldb;
    const int* ids;
    int M, N, n, r, rp;
    void* Y;
    long long ldy;
    int out16;           // 1: Y in the operands' type, 0: FP32
};

// The adapters' term inside a ring kernel's tile.
struct AdapterRing {
    const void* B;       // [n][r] rows of at least nb values, row stride ldb
    long long ldb;
    int nb;              // columns of B that may be read, a multiple of 8
    int n, r, rp, M, N;
    const int* ids;
    const void* t16;
    int np;              // values that a T is made of (ShrinkArgs)
    const float* factor;
    void* Y;
    long long ldy;
    int out16;
};

struct AdapterRingArgs {
    GemmArgs g;
    AdapterRing x;
};

// Gradients of the adapters: out[a][i][c] = sum over the rows m of adapter a
// of T[m][i] X[m][c].
struct OuterSide {
    const float* t32;    // [M][rp], scaled
    const void* X;
    long long ldx;
    int cols;
    float* out;          // [n][r][cols]
    float* part;         // [][r][cols]: the chunks of adapters that have more than one, in adapter order
};

struct OuterArgs {
    OuterSide side[2];
    int M, n, r, rp;
    const int* order;
    int chunk, max_chunks;   // as in ShrinkArgs
    const int* chunk_first;
    const int* part_first;
    const int4* chunks;
};

constexpr int kMaxPads = 5;
// Up to kMaxPads copies of 16-bit operands in one launch.
hipError_t launch_adapter_pad(const PadCopy* c, int n, hipStream_t s);
hipError_t launch_adapter_shrink(int dtype, const ShrinkArgs& a, hipStream_t s);
// The second kernel: sums over K ranges, their rounding, the list of chunks.
hipError_t launch_adapter_round(int dtype, const ShrinkArgs& a, hipStream_t s);
hipError_t launch_adapter_finish(int dtype, const FinishArgs& a, hipStream_t s);
// `f`: the sum of the split product's partials in the same launch, or null.
hipError_t launch_adapter_outer(int dtype, const OuterArgs& a, const FinishArgs* f, hipStream_t s);
// Tiles of the ring kernels used here. `tile` 0: 256 x 256, 1: 192 x 256, 2:
// 128 x 128 (with the adapters' term, or split-K partials with `x` null), 3:
// 64 x 128, 4: 32 x 128, 5: 16 x 128 (partials only). bt: W given as n rows of
// K; g.N is n, the product's columns, rounded up to 8. `shrink`, with tiles 3
// to 5: workgroups of the same launch that make T's partial sums and group the
// rows (not null; no rows: none).
struct AdapterTile {
    int bm, bn;
};
AdapterTile adapter_tile(int tile);
hipError_t launch_adapter_ring(int tile, int dtype, int bt, const GemmArgs& g, int n, const AdapterRing* x,
                               const ShrinkArgs* shrink, hipStream_t s);

}  // namespace sam
