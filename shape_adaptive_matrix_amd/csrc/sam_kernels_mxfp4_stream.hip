// The 4-bit projection for few rows: every weight is read once and used by up
// to 64 rows, so what bounds it is the weight's memory rate (and, for small
// weights, the latency of a launch and of one trip to memory).
//
//  * The scaled 16x16x128 MFMA takes 16 rows of W as its first operand and 16
//    rows of X as its second. Lane group g of four holds one block of 32 of a
//    step's four. The order of the blocks within the sum is free: a lane takes
//    two neighbouring blocks of a 128-byte line of its row, 32 bytes in a
//    piece with their two scales, for two steps.
//  * A workgroup has 16 NB rows of W at a time and all of K, its waves every
//    NW-th line. W goes straight to registers, U lines a wave ahead of their
//    use (of a workgroup 16 KB each with NB = 1); nothing is shared, so there
//    is no LDS trip and no barrier in the loop. A workgroup that has a next
//    tile loads it behind the last one's lines.
//  * Waves' sums meet in LDS and are added in their order: the same bits
//    every time.
//  * X's codes lie in LDS where they fit, for all of a workgroup's tiles. With
//    few values of X (stream4_rounds) every workgroup rounds X itself, while
//    its first weights are on their way; otherwise a launch before it does.
//    More codes than LDS holds are read from memory (from the L2: all
//    workgroups read the same), a line ahead.
#include "sam_dma.h"
#include "sam_mxfp4.h"
#include "sam_quant4.h"

namespace sam {

namespace {

using namespace quant4;
using dma::kOOB;
using dma::make_rsrc;

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));

constexpr int NW = 8, NT = NW * 64;
// Where X comes from: its codes in LDS, made or copied by the workgroup, or
// in memory. LDS for them such that four, three, two or one workgroup run on a
// CU.
enum Source : int { kRound, kCopy, kDirect };
constexpr int kHoldRound = 32 * 1024, kHoldThree = 36 * 1024, kHoldTwo = 72 * 1024, kHoldOne = 144 * 1024;

// Bytes of M rows' codes and scales in LDS: rows of whole lines; a block more
// and four bytes more put rows on banks of their own.
__host__ __device__ __forceinline__ int code_stride(int lines) { return (lines * 8 + 1) * 16; }
__host__ __device__ __forceinline__ int scale_stride(int lines) { return lines * 8 + 4; }
__host__ __device__ __forceinline__ long long held_bytes(long long M, int lines)
{
    return M * (code_stride(lines) + scale_stride(lines));
}
// Values of X that a workgroup rounds itself: 4 rows of 4096 (11008 rows of W:
// 10.1 us); with 8, 13.1 us here and 11.5 with a launch of their own.
constexpr long long kRoundHere = 16384;
// Lines a wave has on the way. Two are a whole tile of 4096 values; with four,
// half of what a wave issues there lies behind the tile's last line (16 rows,
// 131072 x 4096: 74 us, so 65).
constexpr int kAhead = 2;

// An LDS barrier that leaves global loads under way.
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// What a lane loads of a line (256 values) of a row: two blocks, two scales.
struct Pair {
    u4 c[2];
    unsigned s, t;   // both scales in s, or the second in t
};

template <int NB> struct Line {
    Pair w[NB];
};

__device__ __forceinline__ void store_value(const Stream4Args& a, long long at, float v)
{
    if (a.out == DT_F32) static_cast<float*>(a.y)[at] = v;
    else if (a.out == DT_BF16) static_cast<__bf16*>(a.y)[at] = (__bf16)v;
    else static_cast<_Float16*>(a.y)[at] = (_Float16)v;
}

// WB, XB: which bytes of ws and xs hold the scales.
template <int WB, int XB>
__device__ __forceinline__ v4f product(const u4& w, const u4& x, v4f acc, int ws, int xs)
{
    // E2M1 operands are four registers; what would follow them is not read.
    const v8i a = __builtin_bit_cast(v8i, __builtin_shufflevector(w, w, 0, 1, 2, 3, -1, -1, -1, -1));
    const v8i b = __builtin_bit_cast(v8i, __builtin_shufflevector(x, x, 0, 1, 2, 3, -1, -1, -1, -1));
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, acc, 4, 4, WB, ws, XB, xs);
}

// Up to 16 rows of codes and scales that start at `codes` and `scales`; none:
// all reads give zeros.
struct Rows4 {
    __amdgpu_buffer_rsrc_t c, s;
    __device__ __forceinline__ Rows4(const unsigned char* codes, const unsigned char* scales, int kb, int rows)
        : c(__builtin_amdgcn_make_buffer_rsrc(const_cast<unsigned char*>(codes), (short)0, rows * kb * 16, 0x00020000)),
          s(__builtin_amdgcn_make_buffer_rsrc(const_cast<unsigned char*>(scales), (short)0, rows * kb, 0x00020000)) {}
};

// The lane's pair of line `line` (wave-uniform): `off` is its row and pair in
// blocks, `block` the pair's place in a line. Blocks past the row's end read
// as zeros (codes and scale); rows of whole lines (WHOLE) need no look at each.
template <bool WHOLE>
__device__ __forceinline__ void load_pair(Pair& p, const Rows4& r, int off, int block, int line, int kb)
{
    if constexpr (WHOLE) {
        p.c[0] = __builtin_amdgcn_raw_buffer_load_b128(r.c, off * 16, line * 128, 0);
        p.c[1] = __builtin_amdgcn_raw_buffer_load_b128(r.c, off * 16 + 16, line * 128, 0);
        p.s = __builtin_amdgcn_raw_buffer_load_b16(r.s, off, line * 8, 0);
    } else {
        const int left = kb - line * 8 - block, at = off + line * 8;
        p.c[0] = __builtin_amdgcn_raw_buffer_load_b128(r.c, left > 0 ? at * 16 : kOOB, 0, 0);
        p.c[1] = __builtin_amdgcn_raw_buffer_load_b128(r.c, left > 1 ? at * 16 + 16 : kOOB, 0, 0);
        p.s = __builtin_amdgcn_raw_buffer_load_b8(r.s, left > 0 ? at : kOOB, 0, 0);
        p.t = __builtin_amdgcn_raw_buffer_load_b8(r.s, left > 1 ? at + 1 : kOOB, 0, 0);
    }
}

// Workgroups that run on a CU at once, by LDS; registers are kept to that (two
// waves a SIMD each).
constexpr int stream_groups(int hold, int nb)
{
    const int fit = 160 * 1024 / (hold + NW * nb * 1024);
    return hold < 1024 ? 2 : (fit > 4 ? 4 : fit);   // a few KB: what the registers take
}

// DT: X's type where it is rounded here. MB, NB: blocks of 16 rows of X and of
// W. U: lines on the way. HOLD: LDS for X.
template <int SRC, int DT, bool ALIGNED, bool WHOLE, int MB, int NB, int U, int HOLD>
__global__ void __launch_bounds__(NT) stream4_kernel(Stream4Args a)
{
    static_assert(SRC != kRound || MB == 1, "rounded here: up to 16 rows");
    __shared__ __attribute__((aligned(16))) unsigned char held[HOLD];
    __shared__ __attribute__((aligned(16))) float sums[NW][NB * 256];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r16 = lane & 15, g = lane >> 4;
    const int kb = a.kb, lines = (kb + 7) / 8;
    const int tiles = (a.N + 16 * NB - 1) / (16 * NB);
    const int stride = code_stride(lines), sstride = scale_stride(lines);
    unsigned char* hs = held + a.M * stride;

    const int off = r16 * kb + 2 * g;
    // The wave's lines of its tiles, one after the other; of a tile a multiple
    // of U (past the last line: zeros, and no traffic).
    const int turns = ((lines + NW - 1) / NW + U - 1) / U * U, grid = gridDim.x;
    Line<NB> w[U];
    int t_load = blockIdx.x, l_load = 0;   // next to load
    auto load_next = [&](Line<NB>& l) {
        const int line = l_load * NW + wave;
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            const long long n = ((long long)t_load * NB + j) * 16;
            const int rows = line < lines && n < a.N ? min(a.N - (int)n, 16) : 0;
            load_pair<WHOLE>(l.w[j], Rows4(a.codes + n * kb * 16, a.scales + n * kb, kb, rows), off, 2 * g, line, kb);
        }
        const bool last = l_load + 1 == turns;
        l_load = last ? 0 : l_load + 1;
        t_load += last ? grid : 0;
    };
#pragma unroll
    for (int u = 0; u < U; ++u) load_next(w[u]);

    if constexpr (SRC == kRound) {
        typedef typename Ty<DT>::T T;
        constexpr int W = DT == DT_F32 ? 8 : 4;
        const int per_row = lines * 32;   // quarters of blocks
        for (int i = tid; i < a.M * per_row; i += NT) {
            const int row = i / per_row, q = i - row * per_row;
            unsigned x[W], m = 0;
            const int n = a.K - q * 8;
            load_words<DT, ALIGNED>(static_cast<const T*>(a.x) + (n > 0 ? row * a.ldx + q * 8 : 0), n, x);
#pragma unroll
            for (int j = 0; j < W; ++j) m = max_bits<DT>(m, x[j]);
            if (DT != DT_F32) m = max(m & 0xFFFFu, m >> 16);
            m = max(m, quad<0xB1>(m));
            m = max(m, quad<0x4E>(m));
            const unsigned code = scale_code<DT>(m);
            *reinterpret_cast<unsigned*>(held + row * stride + q * 4) = to_codes<DT>(x, code);
            if ((q & 3) == 0) hs[row * sstride + q / 4] = (unsigned char)code;
        }
    } else if constexpr (SRC == kCopy) {
        const __amdgpu_buffer_rsrc_t rc = make_rsrc(a.xc, (long long)a.M * kb * 16), rs = make_rsrc(a.xs, (long long)a.M * kb);
        const int per_row = lines * 8, total = a.M * per_row;
        for (int i0 = 0; i0 < total; i0 += 4 * NT) {
            u4 c[4];
            unsigned s[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int i = i0 + q * NT + tid, row = i / per_row, block = i - row * per_row;
                const bool in = i < total && block < kb;
                c[q] = __builtin_amdgcn_raw_buffer_load_b128(rc, in ? (row * kb + block) * 16 : kOOB, 0, 0);
                s[q] = __builtin_amdgcn_raw_buffer_load_b8(rs, in ? row * kb + block : kOOB, 0, 0);
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int i = i0 + q * NT + tid, row = i / per_row, block = i - row * per_row;
                if (i >= total) continue;
                *reinterpret_cast<u4*>(held + row * stride + block * 16) = c[q];
                hs[row * sstride + block] = (unsigned char)s[q];
            }
        }
    }
    if (SRC != kDirect) lds_barrier();

    // Rows of X past the last: any of its rows, their results are dropped.
    auto load_x = [&](Pair (&x)[MB], int line) {
#pragma unroll
        for (int i = 0; i < MB; ++i) {
            const int row = min(16 * i + r16, a.M - 1);
            if constexpr (SRC == kDirect) {
                load_pair<WHOLE>(x[i], Rows4(a.xc, a.xs, kb, line < lines ? a.M : 0), row * kb + 2 * g, 2 * g, line, kb);
            } else {
                const int block = min(line, lines - 1) * 8 + 2 * g;
                x[i].c[0] = *reinterpret_cast<const u4*>(held + row * stride + block * 16);
                x[i].c[1] = *reinterpret_cast<const u4*>(held + row * stride + block * 16 + 16);
                x[i].s = *reinterpret_cast<const unsigned short*>(hs + row * sstride + block);
            }
        }
    };

    for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        v4f acc[NB][MB];
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
            for (int i = 0; i < MB; ++i) acc[j][i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
        Pair x[2][MB];
        if (SRC == kDirect) load_x(x[0], wave);
        for (int t0 = 0; t0 < turns; t0 += U) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int line = (t0 + u) * NW + wave;
                static_assert(U % 2 == 0, "two sets of X by turns");
                if (SRC == kDirect) load_x(x[(u + 1) % 2], line + NW);
                else load_x(x[u % 2], line);
#pragma unroll
                for (int j = 0; j < NB; ++j)
#pragma unroll
                    for (int i = 0; i < MB; ++i) {
                        const Pair& p = w[u].w[j];
                        const Pair& q = x[u % 2][i];
                        constexpr bool XT = SRC == kDirect && !WHOLE;
                        acc[j][i] = product<0, 0>(p.c[0], q.c[0], acc[j][i], (int)p.s, (int)q.s);
                        acc[j][i] = product<WHOLE ? 1 : 0, XT ? 0 : 1>(p.c[1], q.c[1], acc[j][i], (int)(WHOLE ? p.s : p.t), (int)(XT ? q.t : q.s));
                    }
                __builtin_amdgcn_sched_barrier(0);
                load_next(w[u]);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        const int n0 = tile * 16 * NB;
#pragma unroll
        for (int i = 0; i < MB; ++i) {
            if (i && 16 * i >= a.M) continue;
            lds_barrier();   // the last sums are read
#pragma unroll
            for (int j = 0; j < NB; ++j) *reinterpret_cast<v4f*>(&sums[wave][j * 256 + lane * 4]) = acc[j][i];
            lds_barrier();
            for (int o = tid; o < 16 * NB * min(a.M - 16 * i, 16); o += NT) {
                const int m = o / (16 * NB), n = o % (16 * NB);
                const int at = n / 16 * 256 + (n % 16 / 4 * 16 + m) * 4 + n % 4;
                float v = sums[0][at];
#pragma unroll
                for (int k = 1; k < NW; ++k) v += sums[k][at];
                if (n0 + n < a.N) store_value(a, (16 * i + m) * a.ldy + n0 + n, v);
            }
        }
    }
}

template <int SRC, int DT, bool ALIGNED, int MB, int NB, int U, int HOLD>
hipError_t run(const Stream4Args& a, hipStream_t s)
{
    const long long tiles = ((long long)a.N + 16 * NB - 1) / (16 * NB);
    constexpr int at_once = 256 * stream_groups(HOLD, NB);
    void (*fn)(Stream4Args) = a.kb % 8 == 0 ? stream4_kernel<SRC, DT, ALIGNED, true, MB, NB, U, HOLD>
                                            : stream4_kernel<SRC, DT, ALIGNED, false, MB, NB, U, HOLD>;
    hipLaunchKernelGGL(fn, dim3((unsigned)(tiles < at_once ? tiles : at_once)), dim3(NT), 0, s, a);
    return hipGetLastError();
}

template <int DT, bool ALIGNED>
hipError_t round_here(const Stream4Args& a, hipStream_t s) { return run<kRound, DT, ALIGNED, 1, 1, kAhead, kHoldRound>(a, s); }

template <int MB>
hipError_t from_codes(const Stream4Args& a, hipStream_t s)
{
    const long long bytes = held_bytes(a.M, (a.kb + 7) / 8);
    if (bytes <= kHoldThree) return run<kCopy, DT_F32, true, MB, 1, kAhead, kHoldThree>(a, s);
    if (bytes <= kHoldTwo) return run<kCopy, DT_F32, true, MB, 1, kAhead, kHoldTwo>(a, s);
    if (bytes <= kHoldOne) return run<kCopy, DT_F32, true, MB, 1, kAhead, kHoldOne>(a, s);
    // From memory two blocks of W share X's loads, where that leaves every CU a
    // workgroup (32 rows of 11008: N = 4096 18.4 us by two blocks, 15.0 by one;
    // N = 8192 22.4 and 26.6).
    if constexpr (MB <= 2)
        return a.N <= 16 * 256 ? run<kDirect, DT_F32, true, MB, 1, kAhead, 16>(a, s) : run<kDirect, DT_F32, true, MB, 2, kAhead, 16>(a, s);
    return hipErrorInvalidValue;
}

}  // namespace

bool stream4_takes(long long M, long long kb)
{
    return M <= 32 || (M <= 64 && held_bytes(M, (int)((kb + 7) / 8)) <= kHoldOne);
}

bool stream4_rounds(long long M, long long kb)
{
    return M <= 16 && M * kb * 32 <= kRoundHere && held_bytes(M, (int)((kb + 7) / 8)) <= kHoldRound;
}

hipError_t launch_stream4(int dtype, const Stream4Args& a, hipStream_t s)
{
    if (!a.xc) {
        const int es = dtype == DT_F32 ? 4 : 2;
        const bool al = ((unsigned long long)a.x & 15) == 0 && a.ldx * es % 16 == 0;
        typedef hipError_t (*Fn)(const Stream4Args&, hipStream_t);
        static const Fn fn[3][2] = {{round_here<DT_F32, false>, round_here<DT_F32, true>}, {round_here<DT_BF16, false>, round_here<DT_BF16, true>},
                                    {round_here<DT_F16, false>, round_here<DT_F16, true>}};
        return fn[dtype][al](a, s);
    }
    if (a.M <= 16) return from_codes<1>(a, s);
    if (a.M <= 32) return from_codes<2>(a, s);
    return from_codes<4>(a, s);
}

}  // namespace sam
