// T = X A[a]^T of few rows, as a part of a workgroup grid: used by a kernel
// of its own and beside the tiles of a split projection, which do not need T.
#pragma once

#include "sam_adapter.h"
#include "sam_ring16.h"

namespace sam {

// Workgroups that shrink_part takes for a call's sides together.
__host__ __device__ inline int shrink_wgs(const ShrinkArgs& a)
{
    return (a.M + 15) / 16 * a.slots * a.ksplit * (a.rp / 16) * a.sides;
}

// 16 rows x 16 ranks over one range of K, for the distinct adapters among the
// rows (a slot each) on 16x16x32 blocks: the workgroup's waves take pieces of
// 64 values of K in turn and add up through LDS in wave order. Both operands
// are K-contiguous, so fragments come straight from memory: a lane holds 16
// consecutive values of K of one row (32 bytes), the first eight for one MFMA
// and the others for the next, the same for both operands. Rows of other
// adapters read zeros and are not written.
// Bound by latency: NW x 4 pieces' loads are under way at once, and the K
// ranges are cut such that they are all there are.
constexpr int kShrinkBatch = 4;

template <int DT, int NW>
__device__ __forceinline__ void shrink_part(const ShrinkArgs& a, int wg)
{
    using namespace dma;
    __shared__ float part[NW][16][20];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int rbs = a.rp / 16, per_side = (a.M + 15) / 16 * a.slots * a.ksplit * rbs;
    const ShrinkSide& sd = a.side[wg >= per_side];
    if (wg >= per_side) wg -= per_side;
    const int rb = wg % rbs;
    wg /= rbs;
    const int slot = wg % a.slots;
    wg /= a.slots;
    const int split = wg % a.ksplit, m0 = wg / a.ksplit * 16;
    const int K = sd.K;
    const int pieces = (K + 63) / 64;
    const int p0 = (int)((long long)pieces * split / a.ksplit), p1 = (int)((long long)pieces * (split + 1) / a.ksplit);

    const int row = lane & 15, grp = lane >> 4;
    int id = m0 + row < a.M ? a.ids[m0 + row] : -1;
    if ((unsigned)id >= (unsigned)a.n) id = -1;
    unsigned left = (unsigned)(__ballot(id >= 0) & 0xFFFFull);
    const __amdgpu_buffer_rsrc_t rX =
        make_rsrc(static_cast<const char*>(sd.X) + (long long)m0 * sd.ldx * 2, (long long)(a.M - m0) * sd.ldx * 2);

    for (int d = 0; left; ++d) {
        const int ad = __builtin_amdgcn_readlane(id, __ffs((int)left) - 1);
        const unsigned same = (unsigned)(__ballot(id == ad) & 0xFFFFull);
        left &= ~same;
        if (d % a.slots != slot) continue;
        const __amdgpu_buffer_rsrc_t rA = make_rsrc(static_cast<const char*>(sd.A) + (long long)ad * a.r * sd.lda * 2,
                                                    (long long)a.r * sd.lda * 2);
        const int xrow = (same >> row) & 1 ? (int)(row * sd.ldx * 2) : kOOB;
        const int arow = 16 * rb + row < a.r ? (int)((16 * rb + row) * sd.lda * 2) : kOOB;
        v4f acc = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int p = p0 + wave; p < p1; p += NW * kShrinkBatch) {
            u4 fx[kShrinkBatch][2], fa[kShrinkBatch][2];
#pragma unroll
            for (int b = 0; b < kShrinkBatch; ++b) {
                const int k = (p + b * NW) * 64 + 16 * grp;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const bool ok = p + b * NW < p1 && k + 8 * h < K;
                    const int off = (k + 8 * h) * 2;
                    fx[b][h] = __builtin_amdgcn_raw_buffer_load_b128(rX, ok && xrow != kOOB ? xrow + off : kOOB, 0, 0);
                    fa[b][h] = __builtin_amdgcn_raw_buffer_load_b128(rA, ok && arow != kOOB ? arow + off : kOOB, 0, 0);
                }
            }
#pragma unroll
            for (int b = 0; b < kShrinkBatch; ++b)
#pragma unroll
                for (int h = 0; h < 2; ++h) Mf<DT, 16>::mfma(acc, fx[b][h], fa[b][h]);
        }
        __syncthreads();   // the last slot's sums are read
#pragma unroll
        for (int v = 0; v < 4; ++v) part[wave][4 * grp + v][row] = acc[v];
        __syncthreads();
        const float f = a.scale ? a.scale[ad] : 1.0f;
#pragma unroll
        for (int i = tid; i < 256; i += NW * 64) {
            const int orow = i >> 4, c = i & 15;
            float v = 0.0f;
#pragma unroll
            for (int w = 0; w < NW; ++w) v += part[w][orow][c];
            // Ranks past r: zeros also where X holds Inf.
            if ((same >> orow) & 1)
                sd.t32[((long long)split * a.M + m0 + orow) * a.rp + 16 * rb + c] = 16 * rb + c < a.r ? v * f : 0.0f;
        }
    }
}

// Rows sorted by adapter, one workgroup per adapter: it counts the valid ids
// below its own (where its rows start) and writes its rows in row order. Each
// wave has a range of the rows. Bound by the loads' latency: 32 are under way
// at once, the last ones of a range in eights (65536 rows, one adapter, beside
// the shrink of 256 columns on both sides: 33 us; eight all along 41).
template <int NW>
__device__ __forceinline__ void group_rows(const ShrinkArgs& a, int ad, int (&sums)[2 * NW])
{
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int per = ((a.M + NW * 64 - 1) / (NW * 64)) * 64;
    const int m0 = min(wave * per, a.M), m1 = min(m0 + per, a.M);
    // use(row, id) of the wave's rows, 64 a step; ids past the range are -1.
    auto batch = [&](int m, auto count, auto use) {
        constexpr int U = decltype(count)::value;
        int id[U];
#pragma unroll
        for (int u = 0; u < U; ++u) id[u] = a.ids[min(m + 64 * u + lane, a.M - 1)];
#pragma unroll
        for (int u = 0; u < U; ++u) use(m + 64 * u + lane, m + 64 * u + lane < m1 ? id[u] : -1);
    };
    auto scan = [&](auto use) {
        int m = m0;
        for (; m + 64 * 32 <= m1; m += 64 * 32) batch(m, std::integral_constant<int, 32>{}, use);
        for (; m < m1; m += 64 * 8) batch(m, std::integral_constant<int, 8>{}, use);
    };
    int below = 0, mine = 0;
    scan([&](int, int id) {
        below += (unsigned)id < (unsigned)ad;
        mine += id == ad;
    });
#pragma unroll
    for (int d = 32; d; d >>= 1) {
        below += __shfl_xor(below, d);
        mine += __shfl_xor(mine, d);
    }
    if (lane == 0) {
        sums[wave] = below;
        sums[NW + wave] = mine;
    }
    __syncthreads();
    int at = 0, all = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        at += sums[w] + (w < wave ? sums[NW + w] : 0);
        all += sums[w] + sums[NW + w];
    }
    if (tid == 0) {
        a.seg[ad] = at;
        if (ad == a.n - 1) a.seg[a.n] = all;
    }
    scan([&](int row, int id) {
        const unsigned long long b = __ballot(id == ad);
        if (id == ad) a.order[at + __popcll(b & ((1ull << lane) - 1))] = row;
        at += __popcll(b);
    });
}

// The workgroups of a grid that make T of up to 128 rows, and the grouping.
__host__ __device__ inline int shrink_all_wgs(const ShrinkArgs& a) { return shrink_wgs(a) + (a.order ? a.n : 0); }

template <int DT, int NW>
__device__ __forceinline__ void shrink_or_group(const ShrinkArgs& a, int wg)
{
    __shared__ int sums[2 * NW];
    const int wgs = shrink_wgs(a);
    if (wg >= wgs)
        group_rows<NW>(a, wg - wgs, sums);
    else
        shrink_part<DT, NW>(a, wg);
}

}  // namespace sam
