// Kernels around the shared projection of rows that carry low-rank adapters:
// the rank-r intermediate T (shrink), the sum of a split projection's
// partials with the adapters' term (finish), and the gradients of the
// adapters (outer). sam_adapter.h has the formulas.
#include "sam_adapter.h"
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

constexpr int kShrinkWaves = 8;

// Rows sorted by adapter, one workgroup per adapter: it counts the valid ids
// below its own (where its rows start) and writes its rows in row order.
__device__ __forceinline__ void group_rows(const ShrinkArgs& a, int ad)
{
    constexpr int NT = kShrinkWaves * 64;
    __shared__ int sums[kShrinkWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int below = 0;
    for (int m = tid; m < a.M; m += NT) below += (unsigned)a.ids[m] < (unsigned)ad;
#pragma unroll
    for (int d = 32; d; d >>= 1) below += __shfl_xor(below, d);
    if (lane == 0) sums[wave] = below;
    __syncthreads();
    int at = 0;
#pragma unroll
    for (int w = 0; w < kShrinkWaves; ++w) at += sums[w];
    if (tid == 0) a.seg[ad] = at;
    for (int m0 = 0; m0 < a.M; m0 += NT) {
        const int m = m0 + tid;
        const bool mine = m < a.M && a.ids[m] == ad;
        const unsigned long long b = __ballot(mine);
        __syncthreads();   // the last step's sums are read
        if (lane == 0) sums[wave] = __popcll(b);
        __syncthreads();
        int before = at;
#pragma unroll
        for (int w = 0; w < kShrinkWaves; ++w) {
            before += w < wave ? sums[w] : 0;
            at += sums[w];
        }
        if (mine) a.order[before + __popcll(b & ((1ull << lane) - 1))] = m;
    }
    if (tid == 0 && ad == a.n - 1) a.seg[a.n] = at;
}

// T of 16 rows: for each distinct adapter among them (a slot), X A[ad]^T on
// 16x16x32 blocks, the workgroup's eight waves taking pieces of 64 values of
// K in turn and adding up through LDS in wave order. Both operands are
// K-contiguous, so fragments come straight from memory: a lane holds 16
// consecutive values of K of one row (32 bytes), the first eight for one MFMA
// and the others for the next, the same for both operands. Rows of other
// adapters read zeros and are not written.
// Bound by reading X once; A[ad] comes from L2.
template <int DT, int NR>
__global__ void __launch_bounds__(kShrinkWaves * 64) adapter_shrink_kernel(ShrinkArgs a)
{
    using namespace dma;
    constexpr int NW = kShrinkWaves;
    constexpr int RP = 16 * NR;
    constexpr int BATCH = NR <= 2 ? 4 : (NR <= 4 ? 2 : 1);   // pieces of K loaded ahead of their MFMAs
    __shared__ float part[NW][16][RP + 4];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int blocks = (a.M + 15) / 16;
    int wg = blockIdx.x;
    const int per_side = blocks * a.slots * a.ksplit;
    if (wg >= per_side * a.sides) {
        group_rows(a, wg - per_side * a.sides);
        return;
    }
    const ShrinkSide& sd = a.side[wg >= per_side];
    if (wg >= per_side) wg -= per_side;
    const int split = wg / (blocks * a.slots);
    wg -= split * blocks * a.slots;
    const int m0 = (wg / a.slots) * 16;
    const int slot = wg % a.slots;
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
        v4f acc[NR];
#pragma unroll
        for (int q = 0; q < NR; ++q) acc[q] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
        for (int p = p0 + wave; p < p1; p += NW * BATCH) {
            u4 fx[BATCH][2], fa[BATCH][NR][2];
#pragma unroll
            for (int b = 0; b < BATCH; ++b) {
                const int k = (p + b * NW) * 64 + 16 * grp;
                const bool in = p + b * NW < p1;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const bool ok = in && k + 8 * h < K;
                    fx[b][h] = __builtin_amdgcn_raw_buffer_load_b128(rX, ok && xrow != kOOB ? xrow + (k + 8 * h) * 2 : kOOB, 0, 0);
#pragma unroll
                    for (int q = 0; q < NR; ++q)
                        fa[b][q][h] = __builtin_amdgcn_raw_buffer_load_b128(
                            rA, ok && 16 * q + row < a.r ? (int)(((16 * q + row) * sd.lda + k + 8 * h) * 2) : kOOB, 0, 0);
                }
            }
#pragma unroll
            for (int b = 0; b < BATCH; ++b)
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int q = 0; q < NR; ++q) Mf<DT, 16>::mfma(acc[q], fx[b][h], fa[b][q][h]);
        }
        __syncthreads();   // the last slot's sums are read
#pragma unroll
        for (int q = 0; q < NR; ++q)
#pragma unroll
            for (int v = 0; v < 4; ++v) part[wave][4 * grp + v][16 * q + row] = acc[q][v];
        __syncthreads();
        // 32 threads per row.
        const int orow = tid >> 5, c0 = tid & 31;
        const bool mine = (same >> orow) & 1;
        const float f = a.scale ? a.scale[ad] : 1.0f;
        float t[(RP + 31) / 32], big = 0.0f;
        bool odd = false;   // an Inf or a NaN in the row
#pragma unroll
        for (int q = 0; q < (RP + 31) / 32; ++q) {
            const int c = c0 + 32 * q;
            float v = 0.0f;
            if (c < RP)
#pragma unroll
                for (int w = 0; w < NW; ++w) v += part[w][orow][c];
            t[q] = c < a.r ? v * f : 0.0f;   // ranks past r: zeros also where X holds Inf
            big = fmaxf(big, fabsf(t[q]));
            odd |= !(fabsf(t[q]) < INFINITY);
        }
        const long long m = m0 + orow;
        if (sd.t32 && mine)
#pragma unroll
            for (int q = 0; q < (RP + 31) / 32; ++q)
                if (c0 + 32 * q < RP) sd.t32[((long long)split * a.M + m) * RP + c0 + 32 * q] = t[q];
        if (sd.factor) {
#pragma unroll
            for (int s = 16; s; s >>= 1) {
                big = fmaxf(big, __shfl_xor(big, s));
                odd |= __shfl_xor((int)odd, s) != 0;
            }
            // Divide by the power of two below the row's largest value. A row
            // of zeros gets the smallest one (it then never sets the scale of
            // rows that are added up with it), one with Inf or NaN gets 1.
            int e = big > 0.0f ? ilogbf(big) : -126;
            e = odd ? 0 : (e < -126 ? -126 : e);
            if (mine && c0 == 0) sd.factor[m] = ldexpf(1.0f, e);
            if (mine && sd.t16) {
                unsigned short* o = static_cast<unsigned short*>(sd.t16) + m * 2 * RP;
#pragma unroll
                for (int q = 0; q < (RP + 31) / 32; ++q) {
                    const int c = c0 + 32 * q;
                    unsigned short hi, lo;
                    split_bits<DT>(ldexpf(t[q], -e), hi, lo);
                    if (c < RP) {
                        o[c] = hi;
                        o[RP + c] = lo;
                    }
                }
            }
        }
    }
}

// Y[m][c] = sum over splits of part, in split order, + sum_i T[m][i] B[a][i][c].
// One wave per 256 columns of four rows; rows of one adapter share its loads.
template <int DT>
__device__ __forceinline__ void load_h4(const unsigned short* p, bool vec, int left, float (&o)[4])
{
    unsigned short b[4] = {0, 0, 0, 0};
    if (vec) {
        const uint2 w = *reinterpret_cast<const uint2*>(p);
        b[0] = (unsigned short)w.x; b[1] = (unsigned short)(w.x >> 16);
        b[2] = (unsigned short)w.y; b[3] = (unsigned short)(w.y >> 16);
    } else {
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (q < left) b[q] = p[q];
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) o[q] = from_bits<DT>(b[q]);
}

template <int DT, int ROWS>
__global__ void __launch_bounds__(64) adapter_finish_kernel(FinishArgs a)
{
    __shared__ float t[ROWS][kMaxRank];
    const int lane = threadIdx.x;
    const int strips = (a.N + 255) / 256;
    const int m0 = (blockIdx.x / strips) * ROWS, c = (blockIdx.x % strips) * 256 + 4 * lane;
    const int rows = min(ROWS, a.M - m0);
    int id[ROWS];
    bool same = true;
#pragma unroll
    for (int q = 0; q < ROWS; ++q) {
        id[q] = q < rows ? a.ids[m0 + q] : -1;
        if ((unsigned)id[q] >= (unsigned)a.n) id[q] = -1;
        same &= id[q] == id[0];
    }
#pragma unroll
    for (int q = 0; q < ROWS; ++q)
        for (int i = lane; i < a.r; i += 64) {
            float v = 0.0f;
            if (id[q] >= 0)
                for (int s = 0; s < a.tsplit; ++s) v += a.t32[((long long)s * a.M + m0 + q) * a.rp + i];
            t[q][i] = v;
        }
    __syncthreads();
    if (c >= a.N) return;
    const int left = a.N - c;
    float y[ROWS][4];
#pragma unroll
    for (int q = 0; q < ROWS; ++q) {
#pragma unroll
        for (int v = 0; v < 4; ++v) y[q][v] = 0.0f;
        if (q >= rows) continue;
        for (int s = 0; s < a.split; ++s) {
            const float4 w = *reinterpret_cast<const float4*>(a.part + ((long long)s * a.M + m0 + q) * a.ldp + c);
            y[q][0] += w.x; y[q][1] += w.y; y[q][2] += w.z; y[q][3] += w.w;
        }
    }
    const unsigned short* B = static_cast<const unsigned short*>(a.B);
    const bool vb = a.ldb % 4 == 0 && left >= 4;
    float z[ROWS][4];
#pragma unroll
    for (int q = 0; q < ROWS; ++q)
#pragma unroll
        for (int v = 0; v < 4; ++v) z[q][v] = 0.0f;
    if (same) {
        if (id[0] >= 0)
            for (int i = 0; i < a.r; ++i) {
                float b[4];
                load_h4<DT>(B + ((long long)id[0] * a.r + i) * a.ldb + c, vb, left, b);
#pragma unroll
                for (int q = 0; q < ROWS; ++q)
#pragma unroll
                    for (int v = 0; v < 4; ++v) z[q][v] = fmaf(t[q][i], b[v], z[q][v]);
            }
    } else {
#pragma unroll
        for (int q = 0; q < ROWS; ++q) {
            if (id[q] < 0) continue;
            for (int i = 0; i < a.r; ++i) {
                float b[4];
                load_h4<DT>(B + ((long long)id[q] * a.r + i) * a.ldb + c, vb, left, b);
#pragma unroll
                for (int v = 0; v < 4; ++v) z[q][v] = fmaf(t[q][i], b[v], z[q][v]);
            }
        }
    }
    const bool vy = a.N % 4 == 0 && a.ldy % 4 == 0;
#pragma unroll
    for (int q = 0; q < ROWS; ++q) {
        if (q >= rows) continue;
#pragma unroll
        for (int v = 0; v < 4; ++v) y[q][v] += z[q][v];
        const long long off = (long long)(m0 + q) * a.ldy + c;
        if (a.out16) {
            unsigned short h[4];
#pragma unroll
            for (int v = 0; v < 4; ++v) h[v] = to_bits<DT>(y[q][v]);
            unsigned short* o = static_cast<unsigned short*>(a.Y) + off;
            if (vy)
                *reinterpret_cast<uint2*>(o) = make_uint2(h[0] | (unsigned)h[1] << 16, h[2] | (unsigned)h[3] << 16);
            else
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    if (v < left) o[v] = h[v];
        } else {
            float* o = static_cast<float*>(a.Y) + off;
            if (vy)
                *reinterpret_cast<float4*>(o) = make_float4(y[q][0], y[q][1], y[q][2], y[q][3]);
            else
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    if (v < left) o[v] = y[q][v];
        }
    }
}

// Which adapter's chunk `want` is, and which of its chunks: adapters' rows
// are cut into chunks of `chunk` rows, numbered in adapter order. Every lane
// of the wave gets the answer; ad = -1 past the last chunk.
struct Chunk {
    int ad, first, count;   // adapter, its first chunk's number, its chunks
};

__device__ __forceinline__ Chunk find_chunk(const int* seg, int n, int chunk, int want)
{
    const int lane = threadIdx.x & 63;
    int base = 0;
    for (int a0 = 0; a0 < n; a0 += 64) {
        const int ad = a0 + lane;
        const int c = ad < n ? (seg[ad + 1] - seg[ad] + chunk - 1) / chunk : 0;
        int sum = c;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(sum, d);
            if (lane >= d) sum += o;
        }
        const unsigned long long hit = __ballot(want < base + sum);
        if (hit) {
            const int l = __ffsll((long long)hit) - 1;
            return {a0 + l, base + __shfl(sum - c, l), __shfl(c, l)};
        }
        base += __shfl(sum, 63);
    }
    return {-1, 0, 0};
}

// The adapter's chunks and the number of its first one.
__device__ __forceinline__ Chunk chunks_of(const int* seg, int n, int chunk, int want_ad)
{
    const int lane = threadIdx.x & 63;
    int first = 0, count = 0;
    for (int a0 = 0; a0 <= want_ad; a0 += 64) {
        const int ad = a0 + lane;
        const int c = ad < n ? (seg[ad + 1] - seg[ad] + chunk - 1) / chunk : 0;
        int s = ad < want_ad ? c : 0;
#pragma unroll
        for (int d = 32; d; d >>= 1) s += __shfl_xor(s, d);
        first += s;
        if (want_ad - a0 < 64) count = __shfl(c, want_ad - a0);
    }
    return {want_ad, first, count};
}

constexpr int kOuterCols = 256;

// out[ad][i][c] = sum over a chunk's rows m of T[m][i] X[m][c], for 256
// columns c: MFMA with the rows as its K, 32 a step. X rows come through
// registers into LDS (their order is the grouping's, so each lane has its own
// address) and are read with the transposing LDS read; T is divided by a
// power of two common to the chunk (from the rows' factors, so that binary16
// keeps it), split into a 16-bit value and its 16-bit remainder and read the
// same way: two MFMAs a block, the sum right to 2^-17 (bf16) or 2^-22.
// Bound by reading X once. Chunks of adapters with one chunk go to `out`,
// others to `part`, which outer_sum adds in order.
template <int DT, int NR>
__global__ void __launch_bounds__(256) adapter_outer_kernel(OuterArgs a)
{
    using namespace dma;
    constexpr int RP = 16 * NR;
    constexpr int TROW = 2 * RP < 64 ? 64 : 2 * RP;           // values per T row in LDS
    constexpr int XB = 32 * kOuterCols * 2, TB = 32 * TROW * 2;
    __shared__ __attribute__((aligned(1024))) unsigned char lds[2][XB + TB];
    __shared__ float fmax_s[4];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int strips0 = (a.side[0].cols + kOuterCols - 1) / kOuterCols;
    const int wgs0 = strips0 * a.max_chunks;
    const bool second = (int)blockIdx.x >= wgs0;
    const OuterSide& sd = a.side[second];
    const int wg = second ? blockIdx.x - wgs0 : blockIdx.x;
    const int ch = wg % a.max_chunks, c0 = (wg / a.max_chunks) * kOuterCols;
    const Chunk w = find_chunk(a.seg, a.n, a.chunk, ch);
    const int ad = __builtin_amdgcn_readfirstlane(w.ad);
    if (ad < 0) return;
    const int begin = a.seg[ad] + (ch - w.first) * a.chunk;
    const int rows = min(a.chunk, a.seg[ad + 1] - begin);
    const int* order = a.order + begin;

    // The chunk's scale: the largest of its rows' factors.
    float big = 0.0f;
    for (int m = tid; m < rows; m += 256) big = fmaxf(big, sd.factor[order[m]]);
#pragma unroll
    for (int d = 32; d; d >>= 1) big = fmaxf(big, __shfl_xor(big, d));
    if (lane == 0) fmax_s[wave] = big;
    __syncthreads();
    big = fmaxf(fmaxf(fmax_s[0], fmax_s[1]), fmaxf(fmax_s[2], fmax_s[3]));
    const int e = ilogbf(big);   // factors are powers of two, at least 2^-126

    // Loads of step s into registers: X 32 rows x 512 bytes, four 16-byte
    // pieces a thread; T 32 rows x RP floats, RP / 8 a thread.
    constexpr int TP = RP / 8;
    u4 rx[4];
    float rt[TP];
    const int trow = tid >> 3, tc = (tid & 7) * TP;
    auto load = [&](int s) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int i = s * 32 + q * 8 + (tid >> 5), c = c0 + (tid & 31) * 8;
            rx[q] = u4{0u, 0u, 0u, 0u};
            if (i < rows && c < sd.cols)
                rx[q] = *reinterpret_cast<const u4*>(static_cast<const unsigned short*>(sd.X) + (long long)order[i] * sd.ldx + c);
        }
        const int i = s * 32 + trow;
#pragma unroll
        for (int q = 0; q < TP; ++q) rt[q] = 0.0f;
        if (i < rows) {
            const float* p = sd.t32 + (long long)order[i] * RP + tc;
#pragma unroll
            for (int q = 0; q < TP; q += 2) {
                const float2 v = *reinterpret_cast<const float2*>(p + q);
                rt[q] = v.x;
                rt[q + 1] = v.y;
            }
        }
    };
    auto put = [&](int s) {
        unsigned char* xb = lds[s & 1];
        unsigned char* tb = xb + XB;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int row = q * 8 + (tid >> 5), c = (tid & 31) ^ nsw(row);
            *reinterpret_cast<u4*>(xb + row * kOuterCols * 2 + c * 16) = rx[q];
        }
#pragma unroll
        for (int q = 0; q < TP; q += 2) {
            unsigned short h0, l0, h1, l1;
            split_bits<DT>(ldexpf(rt[q], -e), h0, l0);
            split_bits<DT>(ldexpf(rt[q + 1], -e), h1, l1);
            *reinterpret_cast<unsigned*>(tb + (trow * TROW + tc + q) * 2) = h0 | (unsigned)h1 << 16;
            *reinterpret_cast<unsigned*>(tb + (trow * TROW + RP + tc + q) * 2) = l0 | (unsigned)l1 << 16;
        }
    };
    const int grp = lane >> 4, s16 = lane & 15;
    v4f acc[NR][4];
#pragma unroll
    for (int i = 0; i < NR; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    const int steps = (rows + 31) / 32;
    load(0);
    for (int s = 0; s < steps; ++s) {
        put(s);
        if (s + 1 < steps) load(s + 1);
        __syncthreads();
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
        for (int i = 0; i < 2 * NR; ++i) {
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
    }
    const bool direct = w.count == 1;
    float* o = direct ? sd.out + (long long)ad * a.r * sd.cols : sd.part + (long long)ch * a.r * sd.cols;
    const float back = ldexpf(1.0f, e);
#pragma unroll
    for (int i = 0; i < NR; ++i)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const int row = 16 * i + 4 * grp + v;
            if (row >= a.r) continue;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int c = c0 + wave * 64 + 16 * j + s16;
                if (c < sd.cols) o[(long long)row * sd.cols + c] = acc[i][j][v] * back;
            }
        }
}

// Adapters without rows get zeros, those with several chunks the sum of
// their partials in chunk order. 1024 values a workgroup.
__global__ void __launch_bounds__(256) adapter_outer_sum_kernel(OuterArgs a)
{
    const long long v0 = (long long)a.r * a.side[0].cols, v1 = (long long)a.r * a.side[1].cols;
    const int b0 = (int)((v0 + 1023) / 1024), b1 = (int)((v1 + 1023) / 1024);
    const int ad = blockIdx.x / (b0 + b1), b = blockIdx.x % (b0 + b1);
    const Chunk w = chunks_of(a.seg, a.n, a.chunk, ad);
    if (w.count == 1) return;
    const bool second = b >= b0;
    const OuterSide& sd = a.side[second];
    const long long vals = second ? v1 : v0;
    const long long at = (long long)(second ? b - b0 : b) * 1024 + threadIdx.x;
    float* out = sd.out + (long long)ad * vals;
    const float* part = sd.part + (long long)w.first * vals;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const long long i = at + 256 * q;
        if (i >= vals) continue;
        float v = 0.0f;
        for (int c = 0; c < w.count; ++c) v += part[(long long)c * vals + i];
        out[i] = v;
    }
}

template <int DT>
hipError_t shrink_dt(const ShrinkArgs& a, hipStream_t s)
{
    const int blocks = (a.M + 15) / 16;
    const dim3 grid((unsigned)(blocks * a.slots * a.ksplit * a.sides + (a.order ? a.n : 0)));
    const dim3 block(kShrinkWaves * 64);
    switch (a.rp / 16) {
    case 1: hipLaunchKernelGGL((adapter_shrink_kernel<DT, 1>), grid, block, 0, s, a); break;
    case 2: hipLaunchKernelGGL((adapter_shrink_kernel<DT, 2>), grid, block, 0, s, a); break;
    case 3: hipLaunchKernelGGL((adapter_shrink_kernel<DT, 3>), grid, block, 0, s, a); break;
    case 4: hipLaunchKernelGGL((adapter_shrink_kernel<DT, 4>), grid, block, 0, s, a); break;
    case 8: hipLaunchKernelGGL((adapter_shrink_kernel<DT, 8>), grid, block, 0, s, a); break;
    default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

template <int DT>
hipError_t outer_dt(const OuterArgs& a, hipStream_t s)
{
    const long long strips = (a.side[0].cols + kOuterCols - 1) / kOuterCols + (a.side[1].cols + kOuterCols - 1) / kOuterCols;
    const dim3 grid((unsigned)(strips * a.max_chunks)), block(256);
    if (grid.x) switch (a.rp / 16) {
    case 1: hipLaunchKernelGGL((adapter_outer_kernel<DT, 1>), grid, block, 0, s, a); break;
    case 2: hipLaunchKernelGGL((adapter_outer_kernel<DT, 2>), grid, block, 0, s, a); break;
    case 3: hipLaunchKernelGGL((adapter_outer_kernel<DT, 3>), grid, block, 0, s, a); break;
    case 4: hipLaunchKernelGGL((adapter_outer_kernel<DT, 4>), grid, block, 0, s, a); break;
    case 8: hipLaunchKernelGGL((adapter_outer_kernel<DT, 8>), grid, block, 0, s, a); break;
    default: return hipErrorInvalidValue;
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const long long b = ((long long)a.r * a.side[0].cols + 1023) / 1024 + ((long long)a.r * a.side[1].cols + 1023) / 1024;
    hipLaunchKernelGGL(adapter_outer_sum_kernel, dim3((unsigned)(a.n * b)), block, 0, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_adapter_shrink(int dtype, const ShrinkArgs& a, hipStream_t s)
{
    return dtype == DT_BF16 ? shrink_dt<DT_BF16>(a, s) : shrink_dt<DT_F16>(a, s);
}

hipError_t launch_adapter_finish(int dtype, const FinishArgs& a, hipStream_t s)
{
    const long long strips = (a.N + 255) / 256;
    const int rows = a.M >= 16 ? 4 : 1;
    const dim3 grid((unsigned)(strips * ((a.M + rows - 1) / rows)));
    if (rows == 4) {
        if (dtype == DT_BF16)
            hipLaunchKernelGGL((adapter_finish_kernel<DT_BF16, 4>), grid, dim3(64), 0, s, a);
        else
            hipLaunchKernelGGL((adapter_finish_kernel<DT_F16, 4>), grid, dim3(64), 0, s, a);
    } else {
        if (dtype == DT_BF16)
            hipLaunchKernelGGL((adapter_finish_kernel<DT_BF16, 1>), grid, dim3(64), 0, s, a);
        else
            hipLaunchKernelGGL((adapter_finish_kernel<DT_F16, 1>), grid, dim3(64), 0, s, a);
    }
    return hipGetLastError();
}

hipError_t launch_adapter_outer(int dtype, const OuterArgs& a, hipStream_t s)
{
    return dtype == DT_BF16 ? outer_dt<DT_BF16>(a, s) : outer_dt<DT_F16>(a, s);
}

}  // namespace sam
