// The shared projection of rows that carry adapters: the 16-bit ring kernel
// (sam_ring16.h) with the adapters' term added inside the tile, and its
// narrow tiles for few rows, which leave split-K partials.
//
// The term costs one or two MFMA k-steps per 16 ranks and tile: T B[a] is
// made in the accumulators before the K loop, from T of the tile's rows
// (rounded to the operands' type, with what the rounding left as 16 further
// values of the same k-step: 16x16x32 blocks hold 16 ranks and their
// remainders, so T counts with 2^-17 (bf16) or 2^-22 (f16) relative to its
// row's largest value, not with 2^-9 or 2^-12; an FP32 result of bf16 takes
// a third, T exactly) and B[a]'s rows in LDS. Measured at 4096 x 11008 x 4096,
// rank 64: 12 us of 290; 256 x 4096 x 11008, rank 32: 5 of 46. Each row was
// divided by a power of two before it was rounded, so that binary16 neither
// overflows nor loses small rows; the accumulators are multiplied by it before
// the K loop starts. An Inf in a row's own B meets T's values one by one (one
// of them may be 0, or of the other sign) and may come out as NaN.
#include "sam_adapter.h"
#include "sam_adapter_shrink.h"
#include "sam_ring16.h"

namespace sam {

namespace {

template <int DT> struct Out16;
template <> struct Out16<DT_BF16> { typedef __bf16 T; };
template <> struct Out16<DT_F16> { typedef _Float16 T; };

// Every LDS write of this wave done, then the workgroup's barrier. The asm
// keeps the compiler from moving LDS accesses across.
__device__ __forceinline__ void lds_sync()
{
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

struct AdapterHook {
    static constexpr bool ON = true, B_ONCE = false;
    typedef AdapterRing Args;
    static __device__ __forceinline__ int b_rows(const GemmArgs&, const AdapterRing* x) { return x->N; }
    static constexpr int RC = 32;   // ranks of one adapter in LDS at a time

    // The tile's ids, straight into LDS ahead of the ring's loads, so that
    // the list below is made while those are under way.
    template <int BM>
    static __device__ __forceinline__ int* tile_ids()
    {
        __shared__ __attribute__((aligned(16))) int ids[(BM + 63) / 64 * 64];
        return ids;
    }

    template <int BM>
    static __device__ __forceinline__ void before(const AdapterRing& x, int m0, int wave, int lane)
    {
        if (wave * 64 < BM)
            dma::lds_load4(dma::rsrc_words(x.ids + m0, x.n ? (long long)(x.M - m0) * 4 : 0),   // no adapters: no ids
                           dma::lds_addr(tile_ids<BM>() + wave * 64), (wave * 64 + lane) * 4);
    }

    // FILL: ring loads of this wave issued after `before`.
    template <int DT, int BM, int BN, int NW, int TM, int TN, int FILL>
    static __device__ __forceinline__ void start(const AdapterRing& x, v4f (&acc)[TM][TN], int m0, int n0, int wm0,
                                                 int wn0, int wave, int lane)
    {
        using namespace dma;
        static_assert(FILL < 64 && BM <= NW * 64, "ids are the oldest loads; one row per thread");
        __shared__ __attribute__((aligned(1024))) unsigned char bl[RC * BN * 2];
        __shared__ int list[BM];
        __shared__ int count;
        int* ids = tile_ids<BM>();
        const int tid = wave * 64 + lane;
        const int lrow = lane & 15, lgrp = lane >> 4, s16 = lane & 15;
        if (tid == 0) count = 0;
        wait_cnt<FILL, 0>();
        lds_sync();
        // Rows past M read zeros above; they, and ids that name no adapter,
        // become -1. A row whose id differs from the row's before it heads a
        // run; the runs' adapters, each once, are the tile's list (its order
        // does not matter: a row takes the term of its own adapter alone).
        int id = -1, prev = -1;
        if (tid < BM) {
            id = ids[tid];
            prev = tid ? ids[tid - 1] : -1;
            if (m0 + tid >= x.M || (unsigned)id >= (unsigned)x.n) id = -1;
        }
        lds_sync();
        if (tid < BM) {
            ids[tid] = id;
            if (id >= 0 && (tid == 0 || prev != id)) list[atomicAdd(&count, 1)] = id;
        }
        lds_sync();
        const int heads = __builtin_amdgcn_readfirstlane(count);
        if (heads == 0) return;
        bool dup = false;
        if (tid < heads)
            for (int e = 0; e < tid; ++e) dup |= list[e] == list[tid];
        lds_sync();
        if (dup) list[tid] = -1;
        lds_sync();

        constexpr int CPR = BN / 8, RPI = 64 / CPR;   // 16-byte chunks per row of B, rows per 1 KB load
        constexpr int INS = RC * BN * 2 / 1024;       // loads per chunk of ranks
        static_assert(INS % NW == 0, "loads must split evenly over waves");
        const __amdgpu_buffer_rsrc_t rT = make_rsrc(static_cast<const char*>(x.t16) + (long long)m0 * x.rp * x.np * 2,
                                                    (long long)(x.M - m0) * x.rp * x.np * 2);
        __builtin_amdgcn_sched_barrier(0);
        bool first = true;
#pragma clang loop unroll(disable)
        for (int e = 0; e < heads; ++e) {
            const int ad = __builtin_amdgcn_readfirstlane(list[e]);
            if (ad < 0) continue;
#pragma clang loop unroll(disable)
            for (int r0 = 0; r0 < x.rp; r0 += RC) {
                // Ranks r0 .. r0 + RC - 1 of B[ad], columns n0 .. n0 + BN - 1,
                // placed and swizzled as the ring's B; ranks past r and
                // columns past N read zeros.
                if (!first) lds_sync();   // the last chunk's reads are done
                first = false;
                const long long base = (((long long)ad * x.r + r0) * x.ldb + n0) * 2;
                const i4 rB = rsrc_words(static_cast<const char*>(x.B) + base,
                                         ((long long)(x.r - r0) * x.ldb - n0) * 2);
#pragma unroll
                for (int q = 0; q < INS / NW; ++q) {
                    const int I = wave + q * NW;
                    const int row = I * RPI + lane / CPR;
                    const int c = (lane % CPR) ^ nsw(row);
                    const bool ok = r0 + row < x.r && n0 + c * 8 < x.nb;
                    lds_load16(rB, lds_addr(bl + I * 1024), ok ? (int)((row * x.ldb + c * 8) * 2) : kOOB);
                }
                asm volatile("s_waitcnt vmcnt(0)\n\ts_barrier" ::: "memory");
                const int steps = min(RC, x.rp - r0) / 16 * (x.np - 1);
#pragma clang loop unroll(disable)
                for (int st = 0; st < steps; ++st) {
                    // T of the wave's rows: lane groups 0 and 1 hold 8 ranks
                    // each, groups 2 and 3 the same ranks' remainders. Third
                    // values take a step of their own, groups 0 and 1 alone.
                    const int t = x.np == 3 ? st >> 1 : st, piece = x.np == 3 && (st & 1) ? 2 : 0;
                    u4 ft[TM], fb[TN];
#pragma unroll
                    for (int i = 0; i < TM; ++i) {
                        const int row = wm0 + 16 * i + lrow;
                        const int off = ((row * x.np + piece + (lgrp >> 1)) * x.rp + r0 + 16 * t + 8 * (lgrp & 1)) * 2;
                        ft[i] = __builtin_amdgcn_raw_buffer_load_b128(rT, piece && lgrp > 1 ? kOOB : off, 0, 0);
                    }
#pragma unroll
                    for (int j = 0; j < TN; ++j) {
                        u2 h[2];
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            const int col = wn0 + 16 * j + 4 * (s16 & 3);
                            const int row = 16 * t + 8 * (lgrp & 1) + 4 * half + (s16 >> 2);
                            const int c = (col >> 3) ^ nsw(row);
                            const v4s v = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                SAM_LDS4S(bl + row * BN * 2 + c * 16 + (col & 7) * 2));
                            h[half] = __builtin_bit_cast(u2, v);
                        }
                        fb[j] = u4{h[0][0], h[0][1], h[1][0], h[1][1]};
                    }
                    // A row takes the sum only if the adapter is its own, by
                    // selection: another request's Inf or NaN cannot reach it.
#pragma unroll
                    for (int i = 0; i < TM; ++i) {
                        const bool mine = ids[wm0 + 16 * i + lrow] == ad;
#pragma unroll
                        for (int j = 0; j < TN; ++j) {
                            v4f v = acc[i][j];
                            Mf<DT, 16>::mfma(v, fb[j], ft[i]);
#pragma unroll
                            for (int q = 0; q < 4; ++q) acc[i][j][q] = mine ? v[q] : acc[i][j][q];
                        }
                    }
                }
            }
        }
        __builtin_amdgcn_sched_barrier(0);
        const __amdgpu_buffer_rsrc_t rF = make_rsrc(x.factor + m0, (long long)(x.M - m0) * 4);
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            const int row = wm0 + 16 * i + lrow;
            const float v = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rF, row * 4, 0, 0));
            const float f = ids[row] >= 0 ? v : 1.0f;
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q) acc[i][j][q] *= f;
        }
        __builtin_amdgcn_sched_barrier(0);
    }

    // Lane l holds row l % 16 of a block, columns 4 (l / 16) .. + 3.
    template <int DT, int TM, int TN>
    static __device__ __forceinline__ void store(const AdapterRing& x, const v4f (&acc)[TM][TN], int m0, int n0, int wm0,
                                                 int wn0, int lane)
    {
        using namespace dma;
        typedef typename Out16<DT>::T H;
        const int es = x.out16 ? 2 : 4;
        const int rows = x.M - m0, cols = x.N - n0;
        const int ldy = (int)x.ldy;
        const __amdgpu_buffer_rsrc_t rY =
            make_rsrc(static_cast<char*>(x.Y) + ((long long)m0 * x.ldy + n0) * es,
                      ((long long)(rows - 1) * x.ldy + cols) * es);
        const bool vec = x.N % 4 == 0 && x.ldy % 4 == 0;   // four columns: all inside Y, aligned to 4 values
        auto each = [&](auto put) {
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j) put(acc[i][j], wm0 + 16 * i + (lane & 15), wn0 + 16 * j + 4 * (lane >> 4));
        };
        auto half4 = [](const v4f& v) {
            typedef H h4 __attribute__((ext_vector_type(4)));
            const h4 h = {(H)v[0], (H)v[1], (H)v[2], (H)v[3]};
            return __builtin_bit_cast(u2, h);
        };
        if (vec && x.out16) {
            each([&](const v4f& v, int row, int col) {
                const bool ok = row < rows && col < cols;
                __builtin_amdgcn_raw_buffer_store_b64(half4(v), rY, ok ? (row * ldy + col) * 2 : kOOB, 0, 0);
            });
        } else if (vec) {
            each([&](const v4f& v, int row, int col) {
                const bool ok = row < rows && col < cols;
                __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u4, v), rY, ok ? (row * ldy + col) * 4 : kOOB, 0, 0);
            });
        } else if (x.out16) {
            // Rows that do not start on 8 bytes. Where they do not start on 4
            // either, a lane stores the four values that do, one to the left
            // of its own: the first is the last one of the lane (or block)
            // beside it. Words that do not start on 4 bytes cost more: 2049 x
            // 4097 over 1025 39 us, this way 36.
            const int hi = min(cols, wn0 + 16 * TN);
#pragma unroll
            for (int i = 0; i < TM; ++i) {
                const int row = wm0 + 16 * i + (lane & 15);
                unsigned short* y = static_cast<unsigned short*>(x.Y) + (long long)(m0 + row) * x.ldy + n0;
                const int odd = (int)(((long long)(m0 + row) * x.ldy + n0 + wn0) & 1);
                unsigned beside = 0;
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    const u2 h = half4(acc[i][j]);
                    const unsigned last = h[1] >> 16;
                    const unsigned left = __builtin_amdgcn_ds_bpermute(((lane + 48) & 63) * 4, lane >= 48 ? beside : last);
                    beside = last;
                    const u2 v = odd ? u2{left | h[0] << 16, h[0] >> 16 | h[1] << 16} : h;
                    const int col = wn0 + 16 * j + 4 * (lane >> 4) - odd;
                    if (row >= rows) continue;
                    if (col >= wn0 && col + 4 <= hi)
                        __builtin_memcpy(y + col, &v, 8);
                    else
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            if (col + q >= wn0 && col + q < hi) y[col + q] = (unsigned short)(v[q >> 1] >> (16 * (q & 1)));
                    if (odd && j == TN - 1 && lane >= 48 && col + 4 < hi) y[col + 4] = (unsigned short)last;
                }
            }
        } else {
            // The hardware's unaligned stores, single values at the end of a row.
            float* Y = static_cast<float*>(x.Y) + (long long)m0 * x.ldy + n0;
            each([&](const v4f& v, int row, int col) {
                if (row >= rows || col >= cols) return;
                float* o = Y + (long long)row * ldy + col;
                if (col + 4 <= cols)
                    __builtin_memcpy(o, &v, 16);
                else
#pragma unroll
                    for (int q = 0; q < 3; ++q)
                        if (col + q < cols) o[q] = v[q];
            });
        }
    }
};

// One workgroup per tile, whole K, the adapters' term inside.
template <int DT, int BM, int BN, int WM, int WN, int NBUF, int MODE>
__global__ void __launch_bounds__(WM * WN * 64)
__attribute__((amdgpu_waves_per_eu(1, ring16_waves_per_eu<BM, BN, WM, WN, 64, NBUF>())))
adapter_ring_kernel(AdapterRingArgs a)
{
    int tm, tn, s;
    dma::tile_coords(blockIdx.x, a.g, tm, tn, s);
    ring16_segment<DT, BM, BN, WM, WN, 64, NBUF, MODE, 16, 1, false, AdapterHook>(a.g, tm, tn, 0, a.g.K, nullptr, 0, 0,
                                                                                 0, true, &a.x);
}

// One workgroup per (tile, K range): partials with rows of N rounded up to 8
// floats, of which the columns past n are not meant to be read.
template <bool ONCE>
struct PartHook {
    static constexpr bool ON = false, B_ONCE = ONCE;
    typedef int Args;
    static __device__ __forceinline__ int b_rows(const GemmArgs&, const int* n) { return *n; }
};

template <int DT, int BM, int BN, int WM, int WN, int NBUF, int MODE>
__global__ void __launch_bounds__(WM * WN * 64)
__attribute__((amdgpu_waves_per_eu(1, ring16_waves_per_eu<BM, BN, WM, WN, 64, NBUF>())))
adapter_part_kernel(GemmArgs g, int n)
{
    int tm, tn, s;
    dma::tile_coords(blockIdx.x, g, tm, tn, s);
    const int kbeg = s * g.k_chunk;
    const int kend = min(g.K, kbeg + g.k_chunk);
    ring16_segment<DT, BM, BN, WM, WN, 64, NBUF, MODE, 16, 1, false, PartHook<false>>(g, tm, tn, kbeg, kend, nullptr, s, 0, 0,
                                                                              true, &n);
}

// The same for few rows, with `more` workgroups in front (a multiple of 8, so
// that the tiles keep their XCDs) for T's partial sums, which nothing here
// needs: a launch less, and their loads are under way beside the tiles'.
template <int DT, int BM, int BN, int WM, int WN, int NBUF, int MODE>
__global__ void __launch_bounds__(WM * WN * 64)
__attribute__((amdgpu_waves_per_eu(1, ring16_waves_per_eu<BM, BN, WM, WN, 64, NBUF>())))
adapter_part_shrink_kernel(GemmArgs g, int n, ShrinkArgs a, int more)
{
    if ((int)blockIdx.x < more) {
        if ((int)blockIdx.x < shrink_all_wgs(a)) shrink_or_group<DT, WM * WN>(a, blockIdx.x);
        return;
    }
    int tm, tn, s;
    dma::tile_coords(blockIdx.x - more, g, tm, tn, s);
    const int kbeg = s * g.k_chunk;
    const int kend = min(g.K, kbeg + g.k_chunk);
    ring16_segment<DT, BM, BN, WM, WN, 64, NBUF, MODE, 16, 1, false, PartHook<true>>(g, tm, tn, kbeg, kend, nullptr, s, 0, 0,
                                                                              true, &n);
}

typedef void (*AdapterKernelFn)(AdapterRingArgs);
typedef void (*AdapterPartFn)(GemmArgs, int);
typedef void (*AdapterPartShrinkFn)(GemmArgs, int, ShrinkArgs, int);

struct TileKernels {
    int bm, bn, threads;
    AdapterKernelFn fused[2][2];   // [dtype - 1][bt]
    AdapterPartFn part[2][2];
    AdapterPartShrinkFn shrink[2][2];
};

#define SAM_AD_FUSED(BM, BN, WM, WN, NBUF)                                                         \
    {{adapter_ring_kernel<DT_BF16, BM, BN, WM, WN, NBUF, 0>, adapter_ring_kernel<DT_BF16, BM, BN, WM, WN, NBUF, 3>}, \
     {adapter_ring_kernel<DT_F16, BM, BN, WM, WN, NBUF, 0>, adapter_ring_kernel<DT_F16, BM, BN, WM, WN, NBUF, 3>}}
#define SAM_AD_PART(BM, BN, WM, WN, NBUF)                                                          \
    {{adapter_part_kernel<DT_BF16, BM, BN, WM, WN, NBUF, 0>, adapter_part_kernel<DT_BF16, BM, BN, WM, WN, NBUF, 3>}, \
     {adapter_part_kernel<DT_F16, BM, BN, WM, WN, NBUF, 0>, adapter_part_kernel<DT_F16, BM, BN, WM, WN, NBUF, 3>}}
#define SAM_AD_SHRINK(BM, BN, WM, WN, NBUF)                                                        \
    {{adapter_part_shrink_kernel<DT_BF16, BM, BN, WM, WN, NBUF, 0>,                                 \
      adapter_part_shrink_kernel<DT_BF16, BM, BN, WM, WN, NBUF, 3>},                                \
     {adapter_part_shrink_kernel<DT_F16, BM, BN, WM, WN, NBUF, 0>,                                  \
      adapter_part_shrink_kernel<DT_F16, BM, BN, WM, WN, NBUF, 3>}}
#define SAM_AD_NONE {{nullptr, nullptr}, {nullptr, nullptr}}

const TileKernels kTiles[] = {
    {256, 256, 512, SAM_AD_FUSED(256, 256, 2, 4, 2), SAM_AD_NONE, SAM_AD_NONE},
    {192, 256, 512, SAM_AD_FUSED(192, 256, 2, 4, 2), SAM_AD_NONE, SAM_AD_NONE},
    {128, 128, 512, SAM_AD_FUSED(128, 128, 2, 4, 4), SAM_AD_PART(128, 128, 2, 4, 4), SAM_AD_NONE},
    {64, 128, 256, SAM_AD_NONE, SAM_AD_NONE, SAM_AD_SHRINK(64, 128, 1, 4, 3)},
    {32, 128, 256, SAM_AD_NONE, SAM_AD_NONE, SAM_AD_SHRINK(32, 128, 1, 4, 3)},
    {16, 128, 128, SAM_AD_NONE, SAM_AD_NONE, SAM_AD_SHRINK(16, 128, 1, 2, 4)},
};

}  // namespace

AdapterTile adapter_tile(int tile) { return {kTiles[tile].bm, kTiles[tile].bn}; }

hipError_t launch_adapter_ring(int tile, int dtype, int bt, const GemmArgs& g, int n, const AdapterRing* x,
                               const ShrinkArgs* shrink, hipStream_t s)
{
    const TileKernels& k = kTiles[tile];
    const dim3 grid((unsigned)((long long)g.tiles_m * g.tiles_n * g.split));
    if (x) {
        const AdapterKernelFn fn = k.fused[dtype - 1][bt];
        if (!fn) return hipErrorInvalidDeviceFunction;
        hipLaunchKernelGGL(fn, grid, dim3(k.threads), 0, s, AdapterRingArgs{g, *x});
    } else if (const AdapterPartShrinkFn beside = k.shrink[dtype - 1][bt]) {
        const int more = (shrink_all_wgs(*shrink) + 7) / 8 * 8;
        hipLaunchKernelGGL(beside, dim3(grid.x + more), dim3(k.threads), 0, s, g, n, *shrink, more);
    } else {
        const AdapterPartFn fn = k.part[dtype - 1][bt];
        if (!fn) return hipErrorInvalidDeviceFunction;
        hipLaunchKernelGGL(fn, grid, dim3(k.threads), 0, s, g, n);
    }
    return hipGetLastError();
}

}  // namespace sam
