// Kernels around the shared projection of rows that carry low-rank adapters:
// the rank-r intermediate T (shrink), the sum of a split projection's
// partials with the adapters' term (finish), and the gradients of the
// adapters (outer). sam_adapter.h has the formulas.
#include "sam_adapter.h"
#include "sam_adapter_shrink.h"
#include "sam_ring16.h"

namespace sam {

namespace {

template <int DT> struct Half;
template <> struct Half<DT_BF16> { typedef __bf16 T; };
template <> struct Half<DT_F16> { typedef _Float16 T; };

template <int DT>
__device__ __forceinline__ unsigned short to_bits(float v)
{
    return __builtin_bit_cast(unsigned short, (typename Half<DT>::T)v);
}

template <int DT>
__device__ __forceinline__ float from_bits(unsigned short b)
{
    return (float)__builtin_bit_cast(typename Half<DT>::T, b);
}

// v as a value of the type and what that leaves, again as such a value: hi +
// lo has 16 (bf16) or 22 (f16) of v's 24 bits. Inf and NaN leave nothing.
template <int DT>
__device__ __forceinline__ void split_bits(float v, unsigned short& hi, unsigned short& lo)
{
    hi = to_bits<DT>(v);
    const float rest = v - from_bits<DT>(hi);
    lo = fabsf(v) < INFINITY ? to_bits<DT>(rest) : (unsigned short)0;
}

// v as three bfloat16 values that add up to it exactly: 8 of its 24 bits each
// (those under 2^-133 vanish). Inf and NaN leave nothing.
__device__ __forceinline__ void split3_bits(float v, unsigned short (&o)[3])
{
    const bool fine = fabsf(v) < INFINITY;
    const unsigned h = __float_as_uint(v) & 0xFFFF0000u;
    const float r1 = v - __uint_as_float(h);
    const unsigned m = __float_as_uint(r1) & 0xFFFF0000u;
    const float r2 = r1 - __uint_as_float(m);
    o[0] = fine ? (unsigned short)(h >> 16) : to_bits<DT_BF16>(v);
    o[1] = fine ? (unsigned short)(m >> 16) : (unsigned short)0;
    o[2] = fine ? (unsigned short)(__float_as_uint(r2) >> 16) : (unsigned short)0;
}

constexpr int kShrinkWaves = 4, kWideRows = 64;

// Rounds a row of T, held by LANES threads (column c0 + LANES q): divides by
// the power of two below the row's largest value. One with Inf or NaN gets 1:
// nothing finite comes of it.
template <int DT, int NQ, int LANES>
__device__ __forceinline__ void round_row(const ShrinkArgs& a, const ShrinkSide& sd, const float (&t)[NQ], long long m,
                                          int c0, bool mine)
{
    float big = 0.0f;
    bool odd = false;
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
        big = fmaxf(big, fabsf(t[q]));
        odd |= !(fabsf(t[q]) < INFINITY);
    }
#pragma unroll
    for (int s = LANES / 2; s; s >>= 1) {
        big = fmaxf(big, __shfl_xor(big, s));
        odd |= __shfl_xor((int)odd, s) != 0;
    }
    int e = big > 0.0f ? ilogbf(big) : -126;
    e = odd ? 0 : (e < -126 ? -126 : e);
    if (mine && c0 == 0) sd.factor[m] = ldexpf(1.0f, e);
    if (!mine || !sd.t16) return;
    unsigned short* o = static_cast<unsigned short*>(sd.t16) + m * a.np * a.rp;
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
        const int c = c0 + LANES * q;
        if (c >= a.rp) continue;
        const float v = ldexpf(t[q], -e);
        if (DT == DT_BF16 && a.np == 3) {
            unsigned short p[3];
            split3_bits(v, p);
#pragma unroll
            for (int i = 0; i < 3; ++i) o[i * a.rp + c] = p[i];
        } else {
            unsigned short hi, lo;
            split_bits<DT>(v, hi, lo);
            o[c] = hi;
            o[a.rp + c] = lo;
        }
    }
}

// T of up to 128 rows.
template <int DT>
__global__ void __launch_bounds__(kShrinkWaves * 64) adapter_shrink_kernel(ShrinkArgs a)
{
    shrink_or_group<DT, kShrinkWaves>(a, blockIdx.x);
}

// T of 64 rows over one range of K, for calls with many rows: for each
// distinct adapter among them a product of 64 rows and RP ranks. Both operands
// go straight into LDS, rows of 128 bytes or 256 a wave instruction (loads
// into fragments would touch 64 lines per KB: measured at 4096 x 11008, rank
// 64, 54 us, this 36), through a ring of NBUF stages; wave w has rows
// 16 w .. + 15. The partial sums of the K ranges are added, and rounded, by
// adapter_round_kernel; one range alone is rounded here.
// Bound by reading X once: A's traffic from L2 is r / 64 of X's.
template <int DT, int NR>
__global__ void __launch_bounds__(kShrinkWaves * 64) adapter_shrink_wide_kernel(ShrinkArgs a)
{
    using namespace dma;
    constexpr int NW = kShrinkWaves;
    constexpr int RP = 16 * NR;
    constexpr int BK = NR == 1 ? 128 : 64;                 // the waves' loads of A must come out even
    constexpr int ROW = BK * 2, CP = ROW / 16, RPL = 64 / CP, RSW = 16 / CP;   // as in the ring kernels
    constexpr int XB = kWideRows * ROW, STAGE = XB + RP * ROW;
    constexpr int X_PW = XB / 1024 / NW, A_PW = RP * ROW / 1024 / NW, LPS = X_PW + A_PW;
    constexpr int NBUF = 80 * 1024 / STAGE;                // two workgroups a CU
    static_assert(A_PW * 1024 * NW == RP * ROW && NBUF >= 3 && (NBUF - 1) * LPS < 64, "ring");
    __shared__ __attribute__((aligned(1024))) unsigned char lds[NBUF * STAGE];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int blocks = (a.M + kWideRows - 1) / kWideRows;
    int wg = blockIdx.x;
    if (a.order) {   // first, for they take longest
        if (wg < a.n) {
            group_rows<NW>(a, wg, *reinterpret_cast<int(*)[2 * NW]>(lds));
            return;
        }
        wg -= a.n;
    }
    // A block's further adapters first, too: behind all others they would
    // start when those end.
    const int per_slot = blocks * a.ksplit * a.sides;
    const int slot = a.slots - 1 - wg / per_slot;
    wg %= per_slot;
    const int second = wg >= blocks * a.ksplit;
    const ShrinkSide& sd = a.side[second];
    if (second) wg -= blocks * a.ksplit;
    const int split = wg / blocks;
    const int m0 = (wg - split * blocks) * kWideRows;
    // The K ranges take stages in turn, so that a row's neighbouring pieces
    // are read at the same time.
    const int stages = (sd.K + BK - 1) / BK;
    const int nk = (stages - split + a.ksplit - 1) / a.ksplit;

    int id = m0 + lane < a.M ? a.ids[m0 + lane] : -1;
    if ((unsigned)id >= (unsigned)a.n) id = -1;
    unsigned long long left = __ballot(id >= 0);
    const char* Xb = static_cast<const char*>(sd.X) + (long long)m0 * sd.ldx * 2;
    const int lrow = lane & 15, grp = lane >> 4;

    for (int d = 0; left; ++d) {
        const int ad = __builtin_amdgcn_readlane(id, __ffsll((long long)left) - 1);
        const unsigned long long same = __ballot(id == ad);
        left &= ~same;
        if (d % a.slots != slot) continue;
        const char* Ab = static_cast<const char*>(sd.A) + (long long)ad * a.r * sd.lda * 2;
        // A lane's places in the rows, kept; a stage moves the base. Stages
        // past the last one read zeros: the waits count on every load.
        int off[LPS];
        const int tail = sd.K % BK;   // values of K in a last stage that is not whole
#pragma unroll
        for (int q = 0; q < LPS; ++q) {
            const int row = (wave + (q < X_PW ? q : q - X_PW) * NW) * RPL + lane / CP;
            const bool ok = q < X_PW ? (same >> row) & 1 : row < a.r;
            off[q] = ok ? (int)((row * (q < X_PW ? sd.ldx : sd.lda) + (lane % CP ^ row / RSW % CP) * 8) * 2) : kOOB;
        }
        const long long step = (long long)a.ksplit * BK * 2;
        const char *xk = Xb + (long long)split * BK * 2, *ak = Ab + (long long)split * BK * 2;   // of the next stage to load
        int next = 0;
        const int x_lds = __builtin_amdgcn_readfirstlane(lds_addr(lds)) + wave * 1024;
        auto load = [&](int b) {   // into stage b of the ring
            const bool in = next < nk;
            const i4 sX = rsrc_words(xk, in ? kOOB : 0), sA = rsrc_words(ak, in ? kOOB : 0);
            auto one = [&](int q, int o) {
                lds_load16(q < X_PW ? sX : sA, x_lds + b * STAGE + (q < X_PW ? q * NW * 1024 : XB + (q - X_PW) * NW * 1024), o);
            };
            if (tail && next * a.ksplit + split == stages - 1) {
#pragma unroll
                for (int q = 0; q < LPS; ++q) {
                    const int row = (wave + (q < X_PW ? q : q - X_PW) * NW) * RPL + lane / CP;
                    one(q, (lane % CP ^ row / RSW % CP) * 8 >= tail ? kOOB : off[q]);
                }
            } else {
#pragma unroll
                for (int q = 0; q < LPS; ++q) one(q, off[q]);
            }
            ++next;
            xk += step;
            ak += step;
        };
        v4f acc[NR];
#pragma unroll
        for (int q = 0; q < NR; ++q) acc[q] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
        wait_cnt<0, 15>();   // the counts below are of the ring's loads alone
#pragma unroll
        for (int b = 0; b < NBUF - 1; ++b) load(b);
        // The ring's stages unrolled: their places are constants.
        for (int st = 0; st < nk; st += NBUF)
#pragma unroll
            for (int b = 0; b < NBUF; ++b) {
                if (st + b >= nk) break;
                wait_cnt<(NBUF - 2) * LPS, 0>();   // this wave's part of the stage is there; its reads of the last one are done
                barrier();
                load((b + NBUF - 1) % NBUF);       // into the stage that all waves have left
                // All fragments of the stage, then its MFMAs: one LDS latency a stage, not one each.
                auto piece = [&](int place, int t, int row) {
                    return *reinterpret_cast<const u4*>(lds + b * STAGE + place + row * ROW + ((4 * t + grp) ^ (row / RSW % CP)) * 16);
                };
                u4 fx[BK / 32], fa[BK / 32][NR];
#pragma unroll
                for (int t = 0; t < BK / 32; ++t) {
                    fx[t] = piece(0, t, 16 * wave + lrow);
#pragma unroll
                    for (int q = 0; q < NR; ++q) fa[t][q] = piece(XB, t, 16 * q + lrow);
                }
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int t = 0; t < BK / 32; ++t)
#pragma unroll
                    for (int q = 0; q < NR; ++q) Mf<DT, 16>::mfma(acc[q], fx[t], fa[t][q]);
            }
        // Nothing in flight, nothing unread, before the ring is filled again.
        wait_cnt<0, 0>();
        barrier();
        const float f = a.scale ? a.scale[ad] : 1.0f;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const int row = 16 * wave + 4 * grp + v;
            const bool mine = (same >> row) & 1;
            float t[NR];
#pragma unroll
            for (int q = 0; q < NR; ++q) t[q] = 16 * q + lrow < a.r ? acc[q][v] * f : 0.0f;   // ranks past r: zeros also where X holds Inf
            if (mine && (sd.keep || !shrink_rounds(a))) {
                float* o = sd.t32 + ((long long)split * a.M + m0 + row) * RP + lrow;
#pragma unroll
                for (int q = 0; q < NR; ++q) o[16 * q] = t[q];
            }
            if (shrink_rounds(a) && sd.factor) round_row<DT, NR, 16>(a, sd, t, m0 + row, lrow, mine);
        }
    }
}

// The adapters' rows cut into chunks of a.chunk, numbered in adapter order:
// where each adapter's chunks start, and each chunk's place; of adapters with
// several chunks also where their partials start. One workgroup,
// 256 adapters at a time; a thread has every 256th of their chunks (65536 rows
// of one adapter, 512 chunks: 4.6 us; with an adapter's chunks on one thread
// 170).
__device__ __forceinline__ void list_chunks(const ShrinkArgs& a)
{
    __shared__ int sums[2][4], firsts[256], begins[257];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int base = 0, parts = 0;
    for (int a0 = 0; a0 < a.n; a0 += 256) {
        const int ad = a0 + tid;
        const int begin = a.seg[min(ad, a.n)], rows = a.seg[min(ad + 1, a.n)] - begin;
        const int count = ad < a.n ? max((rows + a.chunk - 1) / a.chunk, 1) : 0;   // without rows: one that gives zeros
        const int several = count > 1 ? count : 0;
        int sum = count, psum = several;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(sum, d), p = __shfl_up(psum, d);
            if (lane >= d) {
                sum += o;
                psum += p;
            }
        }
        __syncthreads();   // the last step's values are read
        if (lane == 63) {
            sums[0][wave] = sum;
            sums[1][wave] = psum;
        }
        begins[tid] = begin;
        if (tid == 255) begins[256] = begin + rows;
        __syncthreads();
        const int from = base;
        int first = base + sum - count, part = parts + psum - several;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            first += w < wave ? sums[0][w] : 0;
            part += w < wave ? sums[1][w] : 0;
            base += sums[0][w];
            parts += sums[1][w];
        }
        firsts[tid] = first;   // past the last adapter: `base`, as it is now
        if (ad < a.n) {
            a.chunk_first[ad] = first;
            a.part_first[ad] = part;
        }
        __syncthreads();
        for (int c = from + tid; c < base; c += 256) {
            int of = 0;   // the last adapter whose chunks start at c or before
#pragma unroll
            for (int d = 128; d; d >>= 1)
                if (firsts[of + d] <= c) of += d;
            const int skip = (c - firsts[of]) * a.chunk;
            const int at = begins[of] + skip, n = min(a.chunk, begins[of + 1] - at);
            const int row0 = n ? a.order[at] : 0;
            // Rows of one run need no look-up.
            a.chunks[c] = make_int4(a0 + of, at, n, n == 0 || a.order[at + n - 1] - row0 == n - 1 ? row0 : -1);
        }
    }
    if (tid == 0) a.chunk_first[a.n] = base;
    for (int c = base + tid; c < a.max_chunks; c += 256) a.chunks[c] = make_int4(-1, 0, 0, -1);
}

// The sum of a row's partials in K order, into the first of them, and its
// rounded form. 32 threads per row, rows without an adapter left out.
template <int DT, int NQ>
__global__ void __launch_bounds__(256) adapter_round_kernel(ShrinkArgs a)
{
    if (shrink_rounds(a) || (int)blockIdx.x >= (a.M + 7) / 8) {
        if (blockIdx.y == 0) list_chunks(a);
        return;
    }
    const int c0 = threadIdx.x & 31;
    const int m = blockIdx.x * 8 + (threadIdx.x >> 5);
    const ShrinkSide& sd = a.side[blockIdx.y];
    const int id = m < a.M ? a.ids[m] : -1;
    const bool mine = (unsigned)id < (unsigned)a.n;
    float t[NQ];
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
        const int c = c0 + 32 * q;
        float v = 0.0f;
        const float* p = sd.t32 + (long long)m * a.rp + c;
        const long long step = (long long)a.M * a.rp;
        for (int s0 = 0; s0 < a.ksplit; s0 += 8) {
            float w[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) w[u] = mine && c < a.rp && s0 + u < a.ksplit ? p[(s0 + u) * step] : 0.0f;
#pragma unroll
            for (int u = 0; u < 8; ++u) v += w[u];
        }
        t[q] = v;
        if (sd.keep && a.ksplit > 1 && mine && c < a.rp) sd.t32[(long long)m * a.rp + c] = v;
    }
    if (sd.factor) round_row<DT, NQ, 32>(a, sd, t, m, c0, mine);
}

// 4 values of B as floats.
template <int DT>
__device__ __forceinline__ void floats_of(const uint2& w, float (&o)[4])
{
    o[0] = from_bits<DT>((unsigned short)w.x);
    o[1] = from_bits<DT>((unsigned short)(w.x >> 16));
    o[2] = from_bits<DT>((unsigned short)w.y);
    o[3] = from_bits<DT>((unsigned short)(w.y >> 16));
}

// Y[m][c] = sum over splits of part, in split order, + sum_i T[m][i] B[a][i][c].
// A wave has 256 columns of a row. WS 4: the four waves of a workgroup share
// one row's sums, a quarter of the partials and of the ranks each, and add up
// in wave order; WS 1: a row each, four rows a workgroup (B of one adapter
// then comes from L1 for three of them).
// Bound by latency: nothing that is loaded depends on anything but the row's
// id, so all first loads go out before the first is used. Measured at 64 rows
// x 11008, rank 16, 2 partials: 6.8 us (one load at a time, 5 partials: 39).
template <int DT, int WS>
__device__ __forceinline__ void finish_rows(const FinishArgs& a, int wg)
{
    constexpr int UP = WS == 4 ? 4 : 8, UB = 8;   // partials, rows of B under way at once; what is more than there are comes from L1
    __shared__ float4 red[3][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int strips = (a.N + 255) / 256;
    const int m = WS == 4 ? wg / strips : wg / strips * 4 + wave;
    if (WS == 1 && m >= a.M) return;
    const int c = (wg % strips) * 256 + 4 * lane;
    const int left = a.N - c, cc = left > 0 ? c : 0;   // lanes past N read the first columns
    const int p = WS == 4 ? wave : 0;
    const int s0 = a.split * p / WS, s1 = a.split * (p + 1) / WS;
    const int i0 = a.r * p / WS, i1 = a.r * (p + 1) / WS;
    int id = a.n ? a.ids[m] : -1;
    if ((unsigned)id >= (unsigned)a.n || i0 == i1) id = -1;

    float4 w[UP];
    auto load_parts = [&](int s) {
#pragma unroll
        for (int u = 0; u < UP; ++u)
            w[u] = *reinterpret_cast<const float4*>(a.part + ((long long)min(s + u, a.split - 1) * a.M + m) * a.ldp + cc);
    };
    // T of the wave's ranks, a lane each (two with more than 64), summed over its own partials.
    float t[2] = {0.0f, 0.0f};
    uint2 wb[UB];
    const unsigned short* B = static_cast<const unsigned short*>(a.B) + (long long)max(id, 0) * a.r * a.ldb + cc;
    auto load_b = [&](int i) {
#pragma unroll
        for (int u = 0; u < UB; ++u) wb[u] = *reinterpret_cast<const uint2*>(B + min(i + u, i1 - 1) * a.ldb);
    };
    load_parts(s0);
    if (id >= 0) {
        load_b(i0);
#pragma unroll
        for (int q = 0; q < (WS == 4 ? 1 : 2); ++q) {
            const int i = i0 + 64 * q + lane;
            const float* tp = a.t32 + (long long)m * a.rp + min(i, i1 - 1);
            const long long step = (long long)a.M * a.rp;
            t[q] = *tp;
            for (int s = 1; s < a.tsplit; s += 8) {
                float x[8];
#pragma unroll
                for (int u = 0; u < 8; ++u) x[u] = tp[min(s + u, a.tsplit - 1) * step];
#pragma unroll
                for (int u = 0; u < 8; ++u) t[q] += s + u < a.tsplit ? x[u] : 0.0f;
            }
        }
    }
    float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int s = s0; s < s1;) {
#pragma unroll
        for (int u = 0; u < UP; ++u)
            if (s + u < s1) {
                y.x += w[u].x; y.y += w[u].y; y.z += w[u].z; y.w += w[u].w;
            }
        s += UP;
        if (s < s1) load_parts(s);
    }
    if (id >= 0)
        for (int i = i0; i < i1;) {
#pragma unroll
            for (int u = 0; u < UB; ++u)
                if (i + u < i1) {
                    const int j = i + u - i0;
                    const float f = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(t[WS == 4 ? 0 : j >> 6]), j & 63));
                    y.x = fmaf(f, from_bits<DT>((unsigned short)wb[u].x), y.x);
                    y.y = fmaf(f, from_bits<DT>((unsigned short)(wb[u].x >> 16)), y.y);
                    y.z = fmaf(f, from_bits<DT>((unsigned short)wb[u].y), y.z);
                    y.w = fmaf(f, from_bits<DT>((unsigned short)(wb[u].y >> 16)), y.w);
                }
            i += UB;
            if (i < i1) load_b(i);
        }
    if constexpr (WS == 4) {
        if (wave) red[wave - 1][lane] = y;
        __syncthreads();
        if (wave) return;
#pragma unroll
        for (int q = 0; q < 3; ++q) {
            const float4 x = red[q][lane];
            y.x += x.x; y.y += x.y; y.z += x.z; y.w += x.w;
        }
    }
    if (left <= 0) return;
    // Four values at a time also where the row does not start on 8 or 16
    // bytes: the hardware's unaligned stores.
    const float v[4] = {y.x, y.y, y.z, y.w};
    const long long off = (long long)m * a.ldy + c;
    if (a.out16) {
        unsigned short h[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) h[q] = to_bits<DT>(v[q]);
        unsigned short* o = static_cast<unsigned short*>(a.Y) + off;
        if (left >= 4)
            __builtin_memcpy(o, h, 8);
        else
#pragma unroll
            for (int q = 0; q < 3; ++q)
                if (q < left) o[q] = h[q];
    } else {
        float* o = static_cast<float*>(a.Y) + off;
        if (left >= 4)
            __builtin_memcpy(o, v, 16);
        else
#pragma unroll
            for (int q = 0; q < 3; ++q)
                if (q < left) o[q] = v[q];
    }
}

constexpr int kOuterCols = 256;

// out[ad][i][c] = sum over a chunk's rows m of T[m][i] X[m][c], for 256
// columns c: MFMA with the rows as its K, 32 a step. X rows come through
// registers into LDS (their order is the grouping's, so each lane has its own
// address) and are read with the transposing LDS read; T is split into 16-bit
// values, an MFMA each, and read the same way. bfloat16: three values, exactly
// T. binary16: each rank's T divided by a power of two of its own, the largest
// finite T of the rank in the chunk (read once ahead for that), a value and its
// remainder: right to 2^-22 of that largest, whatever the other ranks hold.
// Bound by reading X once. Measured at X, dY 4096 x 4096, rank 16, 8
// adapters in runs, both gradients: 18 us with loads two steps ahead, 22.6 one
// step ahead, 14 with all of it but the loads.
// Chunks of adapters with one chunk go to `out`, others to `part`, which
// outer_sum adds in order.
template <int DT, int NR>
__device__ __forceinline__ void outer_tile(const OuterArgs& a, int block)
{
    using namespace dma;
    constexpr int RP = 16 * NR;
    constexpr int NP = DT == DT_BF16 ? 3 : 2;
    // Values per T row in LDS; not a multiple of 128 bytes, so that the four
    // rows of a transposing read fall on different banks.
    constexpr int TROW = NP * RP + (NP * RP % 64 == 0 ? 8 : 0);
    constexpr int XB = 32 * kOuterCols * 2, TB = 32 * TROW * 2;
    __shared__ __attribute__((aligned(1024))) unsigned char lds[2][XB + TB];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int strips0 = (a.side[0].cols + kOuterCols - 1) / kOuterCols;
    const int wgs0 = strips0 * a.max_chunks;
    const bool second = block >= wgs0;
    const OuterSide& sd = a.side[second];
    const int wg = second ? block - wgs0 : block;
    const int ch = wg % a.max_chunks, c0 = (wg / a.max_chunks) * kOuterCols;
    const int4 w = a.chunks[ch];
    const int ad = w.x, rows = w.z, row0 = w.w;
    if (ad < 0) return;
    const int* order = a.order + w.y;
    const bool run = row0 >= 0;

    // Loads of step s into one of two register sets: X 32 rows x 512 bytes,
    // four 16-byte pieces a thread; T 32 rows x RP floats, RP / 8 a thread.
    // None sits behind a condition (the compiler could not count how many
    // follow it, and would wait for all): rows past the chunk's end and
    // columns past X's read its last ones, and become zeros in `put`. A step's
    // row numbers come a step ahead of it.
    constexpr int TP = RP / 8;
    struct Set {
        u4 x[4];
        float t[TP];
    };
    __shared__ float largest[4][DT == DT_F16 ? RP : 1];
    __shared__ int exponent[DT == DT_F16 ? RP : 1];   // of each rank's scale
    Set set[2];
    int next_row = 0;   // of the next step to load, row lane % 32
    const int trow = tid >> 3, tc = (tid & 7) * TP;
    const int col = c0 + (tid & 31) * 8;
    const unsigned short* xc = static_cast<const unsigned short*>(sd.X) + min(col, (sd.cols - 1) & ~7);
    auto load = [&](int s, Set& r) {
        const int rows_here = next_row;
        next_row = order[min((s + 1) * 32 + (lane & 31), rows - 1)];
        auto row_of = [&](int i) -> long long {
            return run ? row0 + min(s * 32 + i, rows - 1) : __shfl(rows_here, i);
        };
#pragma unroll
        for (int q = 0; q < 4; ++q) r.x[q] = *reinterpret_cast<const u4*>(xc + row_of(q * 8 + (tid >> 5)) * sd.ldx);
        const float* p = sd.t32 + row_of(trow) * RP + tc;
#pragma unroll
        for (int q = 0; q < TP; q += 2) {
            const float2 v = *reinterpret_cast<const float2*>(p + q);
            r.t[q] = v.x;
            r.t[q + 1] = v.y;
        }
    };
    auto put = [&](int s, const Set& r) {
        unsigned char* xb = lds[s & 1];
        unsigned char* tb = xb + XB;
        const int left = rows - s * 32;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int row = q * 8 + (tid >> 5), c = (tid & 31) ^ nsw(row);
            *reinterpret_cast<u4*>(xb + row * kOuterCols * 2 + c * 16) = row < left && col < sd.cols ? r.x[q] : u4{0u, 0u, 0u, 0u};
        }
#pragma unroll
        for (int q = 0; q < TP; q += 2) {
            unsigned short h[2][NP];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float t = trow < left ? r.t[q + k] : 0.0f;
                if constexpr (NP == 3)
                    split3_bits(t, h[k]);
                else
                    split_bits<DT>(ldexpf(t, -exponent[tc + q + k]), h[k][0], h[k][1]);
            }
#pragma unroll
            for (int k = 0; k < NP; ++k)
                *reinterpret_cast<unsigned*>(tb + (trow * TROW + k * RP + tc + q) * 2) = h[0][k] | (unsigned)h[1][k] << 16;
        }
    };
    const int grp = lane >> 4, s16 = lane & 15;
    v4f acc[NR][4];
#pragma unroll
    for (int i = 0; i < NR; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    auto multiply = [&](int s) {
        const unsigned char* xb = lds[s & 1];
        const unsigned char* tb = xb + XB;
        u4 fx[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            u2 h[2];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int col = wave * 64 + 16 * j + 4 * (s16 & 3);
                const int row = 8 * grp + 4 * half + (s16 >> 2);
                const int c = (col >> 3) ^ nsw(row);
                h[half] = __builtin_bit_cast(u2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    SAM_LDS4S(xb + row * kOuterCols * 2 + c * 16 + (col & 7) * 2)));
            }
            fx[j] = u4{h[0][0], h[0][1], h[1][0], h[1][1]};
        }
#pragma unroll
        for (int i = 0; i < NP * NR; ++i) {
            u2 h[2];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int col = 16 * i + 4 * (s16 & 3);
                const int row = 8 * grp + 4 * half + (s16 >> 2);
                h[half] = __builtin_bit_cast(u2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    SAM_LDS4S(tb + (row * TROW + col) * 2)));
            }
            const u4 ft = u4{h[0][0], h[0][1], h[1][0], h[1][1]};
#pragma unroll
            for (int j = 0; j < 4; ++j) Mf<DT, 16>::mfma(acc[i % NR][j], ft, fx[j]);
        }
    };
    // A step's values are in LDS from its `put` to the barrier after the next
    // one's: two buffers, one barrier a step.
    const int steps = (rows + 31) / 32;
    auto fill = [&] {
        if (!steps) return;
        next_row = order[min(lane & 31, rows - 1)];
        load(0, set[0]);
        load(1, set[1]);
    };
    if constexpr (DT == DT_F16) {
        // The ranks' exponents: a thread has four ranks of every R-th row, U of
        // them under way at once, the first ones ahead of the steps' loads.
        // Chunks of 64 rows: not seen (1025 rows, 768 x 2049, rank 24, both
        // gradients 32.4 us with and without); of 256 rows of 4096 x 4096 0 us
        // at rank 16, 2.3 of 54 at 32, 4.6 of 79 at 64.
        constexpr int LR = RP / 4, R = 256 / LR, U = RP == 16 ? 4 : (RP == 32 ? 2 : 16);
        const int rank = tid % LR * 4;
        float4 v[U] = {};
        float big[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        auto peek = [&](int m) {   // rows past the end: the last one again; no load waits for another
            const float* p = sd.t32 + rank;
            if (run) {
#pragma unroll
                for (int u = 0; u < U; ++u)
                    v[u] = *reinterpret_cast<const float4*>(p + (long long)(row0 + min(m + u * R + tid / LR, rows - 1)) * RP);
            } else {
                int o[U];
#pragma unroll
                for (int u = 0; u < U; ++u) o[u] = order[min(m + u * R + tid / LR, rows - 1)];
#pragma unroll
                for (int u = 0; u < U; ++u) v[u] = *reinterpret_cast<const float4*>(p + (long long)o[u] * RP);
            }
        };
        if (rows) peek(0);
        fill();
        for (int m = 0; m < rows; m += U * R) {
            if (m) peek(m);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const float t[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
                for (int q = 0; q < 4; ++q) big[q] = fabsf(t[q]) < INFINITY ? fmaxf(big[q], fabsf(t[q])) : big[q];
            }
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
#pragma unroll
            for (int d = LR; d < 64; d <<= 1) big[q] = fmaxf(big[q], __shfl_xor(big[q], d));
            if (lane < LR) largest[wave][rank + q] = big[q];
        }
        __syncthreads();
        if (tid < RP) {
            const float t = fmaxf(fmaxf(largest[0][tid], largest[1][tid]), fmaxf(largest[2][tid], largest[3][tid]));
            exponent[tid] = t > 0.0f ? max(ilogbf(t), -126) : -126;
        }
        __syncthreads();
    } else {
        fill();
    }
    int s = 0;
    for (; s + 2 < steps; s += 2)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            put(s + h, set[h]);
            load(s + h + 2, set[h]);   // past the last step: its last row, not used
            __syncthreads();
            multiply(s + h);
        }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (s + h >= steps) break;
        put(s + h, set[h]);
        __syncthreads();
        multiply(s + h);
    }
    const int first_ch = a.chunk_first[ad], part = a.part_first[ad] + ch - first_ch;
    const bool direct = a.chunk_first[ad + 1] - first_ch == 1;
    float* o = (direct ? sd.out : sd.part) + (long long)(direct ? ad : part) * a.r * sd.cols;
#pragma unroll
    for (int i = 0; i < NR; ++i)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const int row = 16 * i + 4 * grp + v;
            if (row >= a.r) continue;
            float back = 1.0f;
            if constexpr (DT == DT_F16) back = ldexpf(1.0f, exponent[row]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int c = c0 + wave * 64 + 16 * j + s16;
                if (c < sd.cols) o[(long long)row * sd.cols + c] = acc[i][j][v] * back;
            }
        }
}

template <int DT, int WS>
__global__ void __launch_bounds__(256) adapter_finish_kernel(FinishArgs a)
{
    finish_rows<DT, WS>(a, blockIdx.x);
}

// Waves a SIMD that the outer product's registers have to leave room for.
constexpr int outer_waves(int nr) { return nr <= 2 ? 3 : (nr == 4 ? 2 : 1); }

template <int DT, int NR>
__global__ void __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(outer_waves(NR)))) adapter_outer_kernel(OuterArgs a)
{
    outer_tile<DT, NR>(a, blockIdx.x);
}

// Both in one launch, where the backward pass has both: neither needs the other.
template <int DT, int NR, int WS>
__global__ void __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(outer_waves(NR))))
adapter_outer_finish_kernel(OuterArgs o, FinishArgs f, int outer_wgs)
{
    if ((int)blockIdx.x < outer_wgs)
        outer_tile<DT, NR>(o, blockIdx.x);
    else
        finish_rows<DT, WS>(f, blockIdx.x - outer_wgs);
}

// Adapters with several chunks get the sum of their partials. A wave has 256
// values; WS 4: the four waves of a workgroup have the same ones and a quarter
// of the chunks each, in chunk order, and their sums are added in wave order.
// Latency bounds it, so all of a batch's loads go out together.
template <int WS>
__global__ void __launch_bounds__(256) adapter_outer_sum_kernel(OuterArgs a)
{
    __shared__ float sums[3][256];
    constexpr int V = 1024 / WS;   // values of a workgroup
    const long long v0 = (long long)a.r * a.side[0].cols, v1 = (long long)a.r * a.side[1].cols;
    const int b0 = (int)((v0 + V - 1) / V), b1 = (int)((v1 + V - 1) / V);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int ad = (int)(blockIdx.x / (unsigned)(b0 + b1)), b = (int)(blockIdx.x % (unsigned)(b0 + b1));
    const int count = a.chunk_first[ad + 1] - a.chunk_first[ad];
    if (count == 1) return;
    const bool second = b >= b0;
    const OuterSide& sd = a.side[second];
    const long long vals = second ? v1 : v0;
    const long long at = (long long)(second ? b - b0 : b) * V + (WS == 4 ? 0 : wave * 256) + lane;
    const float* part = sd.part + (long long)a.part_first[ad] * vals;
    const int begin = WS == 4 ? (int)((long long)count * wave / 4) : 0;
    const int end = WS == 4 ? (int)((long long)count * (wave + 1) / 4) : count;
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int c = begin; c < end; c += 8) {
        float x[8][4];
#pragma unroll
        for (int u = 0; u < 8; ++u)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const long long i = at + 64 * q;
                x[u][q] = c + u < end && i < vals ? part[(long long)(c + u) * vals + i] : 0.0f;
            }
#pragma unroll
        for (int u = 0; u < 8; ++u)
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] += x[u][q];
    }
    if (WS == 4) {
        if (wave) {
#pragma unroll
            for (int q = 0; q < 4; ++q) sums[wave - 1][lane + 64 * q] = v[q];
        }
        __syncthreads();
        if (wave) return;
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int w = 0; w < 3; ++w) v[q] += sums[w][lane + 64 * q];
    }
    float* out = sd.out + (long long)ad * vals;
#pragma unroll
    for (int q = 0; q < 4; ++q)
        if (at + 64 * q < vals) out[at + 64 * q] = v[q];
}

// Copies of operands whose rows are no whole 16-byte pieces, into rows that
// are, zeros in the gap. A wave has up to 256 pieces of a row; source pieces
// start on any value (the hardware's unaligned loads).
struct PadArgs {
    PadCopy c[kMaxPads];
    long long first[kMaxPads];  // each copy's first wave
    int strips[kMaxPads];       // waves per row
    int n;
};

__global__ void __launch_bounds__(256) adapter_pad_kernel(PadArgs a)
{
    const long long unit = (long long)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int at = 0;
    for (int q = 1; q < a.n; ++q)
        if (unit >= a.first[q]) at = q;
    const PadCopy& p = a.c[at];
    const unsigned u = (unsigned)(unit - a.first[at]), n = (unsigned)a.strips[at];
    const long long row = u / n;
    if (row >= p.rows) return;
    const unsigned short* s = static_cast<const unsigned short*>(p.src) + row * p.lds;
    u4* d = reinterpret_cast<u4*>(static_cast<unsigned short*>(p.dst) + row * p.ldd);
    const int cols = (int)p.cols, pieces = (int)(p.ldd / 8);
    const int i0 = (int)(u % n) * 256 + (threadIdx.x & 63);
    u4 v[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        const int i = i0 + 64 * b;
        v[b] = u4{0u, 0u, 0u, 0u};
        if (8 * i + 8 <= cols) {
            __builtin_memcpy(&v[b], s + 8 * i, 16);
        } else if (8 * i < cols) {
#pragma unroll
            for (int k = 0; k < 7; ++k)
                if (8 * i + k < cols) v[b][k >> 1] |= (unsigned)s[8 * i + k] << (16 * (k & 1));
        }
    }
#pragma unroll
    for (int b = 0; b < 4; ++b)
        if (i0 + 64 * b < pieces) d[i0 + 64 * b] = v[b];
}

template <int DT>
hipError_t shrink_dt(const ShrinkArgs& a, hipStream_t s)
{
    const dim3 block(kShrinkWaves * 64);
    if (!a.wide) {
        hipLaunchKernelGGL((adapter_shrink_kernel<DT>), dim3((unsigned)shrink_all_wgs(a)), block, 0, s, a);
        return hipGetLastError();
    }
    const dim3 grid((unsigned)((a.M + kWideRows - 1) / kWideRows * a.slots * a.ksplit * a.sides + (a.order ? a.n : 0)));
    switch (a.rp) {
    case 16: hipLaunchKernelGGL((adapter_shrink_wide_kernel<DT, 1>), grid, block, 0, s, a); break;
    case 32: hipLaunchKernelGGL((adapter_shrink_wide_kernel<DT, 2>), grid, block, 0, s, a); break;
    case 64: hipLaunchKernelGGL((adapter_shrink_wide_kernel<DT, 4>), grid, block, 0, s, a); break;
    case 128: hipLaunchKernelGGL((adapter_shrink_wide_kernel<DT, 8>), grid, block, 0, s, a); break;
    default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

template <int DT>
hipError_t round_dt(const ShrinkArgs& a, hipStream_t s)
{
    const int rows = shrink_rounds(a) ? 0 : (a.M + 7) / 8;
    const dim3 grid((unsigned)(rows + (a.order ? 1 : 0)), (unsigned)(rows ? a.sides : 1)), block(256);
    if (!grid.x) return hipSuccess;
    switch ((a.rp + 31) / 32) {
    case 1: hipLaunchKernelGGL((adapter_round_kernel<DT, 1>), grid, block, 0, s, a); break;
    case 2: hipLaunchKernelGGL((adapter_round_kernel<DT, 2>), grid, block, 0, s, a); break;
    default: hipLaunchKernelGGL((adapter_round_kernel<DT, 4>), grid, block, 0, s, a); break;
    }
    return hipGetLastError();
}

// Four waves a row while that leaves CUs free (64 rows x 11008: 9.2 us with
// four, 6.8 with one; one row x 4096: 3.6 and 8.1).
bool share_rows(const FinishArgs& f) { return (f.N + 255) / 256 * (long long)f.M <= 1024; }

unsigned finish_wgs(const FinishArgs& f)
{
    return (unsigned)((f.N + 255) / 256 * (long long)(share_rows(f) ? f.M : (f.M + 3) / 4));
}

template <int DT>
hipError_t finish_dt(const FinishArgs& f, hipStream_t s)
{
    const dim3 grid(finish_wgs(f)), block(256);
    if (share_rows(f))
        hipLaunchKernelGGL((adapter_finish_kernel<DT, 4>), grid, block, 0, s, f);
    else
        hipLaunchKernelGGL((adapter_finish_kernel<DT, 1>), grid, block, 0, s, f);
    return hipGetLastError();
}

template <int DT, int NR>
void outer_nr(const OuterArgs& a, const FinishArgs* f, unsigned wgs, hipStream_t s)
{
    const dim3 block(256);
    if (!f)
        hipLaunchKernelGGL((adapter_outer_kernel<DT, NR>), dim3(wgs), block, 0, s, a);
    else if (share_rows(*f))
        hipLaunchKernelGGL((adapter_outer_finish_kernel<DT, NR, 4>), dim3(wgs + finish_wgs(*f)), block, 0, s, a, *f, (int)wgs);
    else
        hipLaunchKernelGGL((adapter_outer_finish_kernel<DT, NR, 1>), dim3(wgs + finish_wgs(*f)), block, 0, s, a, *f, (int)wgs);
}

template <int DT>
hipError_t outer_dt(const OuterArgs& a, const FinishArgs* f, hipStream_t s)
{
    const long long strips = (a.side[0].cols + kOuterCols - 1) / kOuterCols + (a.side[1].cols + kOuterCols - 1) / kOuterCols;
    const unsigned wgs = (unsigned)(strips * a.max_chunks);
    switch (a.rp) {
    case 16: outer_nr<DT, 1>(a, f, wgs, s); break;
    case 32: outer_nr<DT, 2>(a, f, wgs, s); break;
    case 64: outer_nr<DT, 4>(a, f, wgs, s); break;
    case 128: outer_nr<DT, 8>(a, f, wgs, s); break;
    default: return hipErrorInvalidValue;
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.M <= a.chunk) return e;   // no adapter has a second chunk
    // Four waves a value where the adapters have many chunks: 512 of 8192
    // values 10 us (one wave each, a value at a time, 57); 16 of 131072 values
    // 6.9 with four waves, 5.1 with one.
    const long long chunks = (a.M + a.chunk - 1) / a.chunk;
    const bool share = chunks > 32 && chunks > 4ll * a.n;
    const int vals = share ? 256 : 1024;
    const long long b = ((long long)a.r * a.side[0].cols + vals - 1) / vals + ((long long)a.r * a.side[1].cols + vals - 1) / vals;
    const dim3 grid((unsigned)(a.n * b));
    if (share)
        hipLaunchKernelGGL(adapter_outer_sum_kernel<4>, grid, dim3(256), 0, s, a);
    else
        hipLaunchKernelGGL(adapter_outer_sum_kernel<1>, grid, dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_adapter_shrink(int dtype, const ShrinkArgs& a, hipStream_t s)
{
    return dtype == DT_BF16 ? shrink_dt<DT_BF16>(a, s) : shrink_dt<DT_F16>(a, s);
}

hipError_t launch_adapter_round(int dtype, const ShrinkArgs& a, hipStream_t s)
{
    return dtype == DT_BF16 ? round_dt<DT_BF16>(a, s) : round_dt<DT_F16>(a, s);
}

hipError_t launch_adapter_finish(int dtype, const FinishArgs& a, hipStream_t s)
{
    return dtype == DT_BF16 ? finish_dt<DT_BF16>(a, s) : finish_dt<DT_F16>(a, s);
}

hipError_t launch_adapter_pad(const PadCopy* c, int n, hipStream_t s)
{
    PadArgs a{};
    long long waves = 0;
    for (int i = 0; i < n; ++i) {
        a.c[i] = c[i];
        a.first[i] = waves;
        a.strips[i] = (int)((c[i].ldd / 8 + 255) / 256);
        waves += c[i].rows * a.strips[i];
        if (c[i].rows * a.strips[i] >= 1ll << 32) return hipErrorInvalidValue;
    }
    a.n = n;
    if (waves) hipLaunchKernelGGL(adapter_pad_kernel, dim3((unsigned)((waves + 3) / 4)), dim3(256), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_adapter_outer(int dtype, const OuterArgs& a, const FinishArgs* f, hipStream_t s)
{
    return dtype == DT_BF16 ? outer_dt<DT_BF16>(a, f, s) : outer_dt<DT_F16>(a, f, s);
}

}  // namespace sam
