// Kernels that make MXFP4 tensors and read them back (formulas in
// sam_mxfp4.h).
//
// Bound by memory: 2 or 4 bytes a value on one side, 17 / 32 of a byte on the
// other. The scaled conversions of gfx950 take a pair of values by a power of
// two to E2M1 (to nearest, ties to even, saturating) and back; the tests hold
// them against the definition for every 16-bit pattern at four distances from
// its block's largest value, for 262144 FP32 bit patterns, and on and next to
// the borders between codes. A scale of code 0 (2^-127) is the float with all
// bits zero to them.
#include "sam_mxfp4.h"
#include "sam_quant4.h"

namespace sam {

namespace {

using namespace quant4;

constexpr int kQuantThreads = 256, kQuantEach = 2;

constexpr int kPlanesEach = 4;

// 256 rows of scales, kPlanesEach dwords of each, to their planes: a lane
// reads neighbours in a row, a wave writes lines.
__device__ __forceinline__ void to_planes(const Quant4Args& a, unsigned wg)
{
    const unsigned groups = (a.kb / 4 + kPlanesEach - 1) / kPlanesEach;
    const long long row = (long long)(wg / groups) * kQuantThreads + threadIdx.x;
    const int p0 = wg % groups * kPlanesEach;
    if (row >= a.plane_rows) return;
    // Whole words around the row's bytes, shifted into place; words past the
    // row's last byte are its last word, and dropped.
    const unsigned long long at = reinterpret_cast<unsigned long long>(a.from + row * a.from_kb);
    const unsigned* from = reinterpret_cast<const unsigned*>(at & ~3ull);
    const int skew = (int)(at & 3), last = (skew + a.from_kb - 1) >> 2;
    unsigned w[kPlanesEach + 1], d[kPlanesEach];
#pragma unroll
    for (int i = 0; i <= kPlanesEach; ++i) w[i] = from[min(p0 + i, last)];
#pragma unroll
    for (int i = 0; i < kPlanesEach; ++i) {
        const int left = a.from_kb - 4 * (p0 + i);
        const unsigned v = __builtin_amdgcn_alignbit(w[i + 1], w[i], 8 * skew);
        d[i] = left >= 4 ? v : (left > 0 ? v & ((1u << (8 * left)) - 1) : 0u);
    }
#pragma unroll
    for (int i = 0; i < kPlanesEach; ++i)
        if (p0 + i < a.kb / 4) reinterpret_cast<unsigned*>(a.to)[(p0 + i) * scale_rows(a.plane_rows) + row] = d[i];
}

// A quarter of a block a lane: 16 (FP32: 32) bytes in, 4 out, both whole
// lines a wave. The first `copies` workgroups bring other scales into planes.
template <int DT, bool ALIGNED>
__global__ void __launch_bounds__(kQuantThreads) quant4_rows_kernel(Quant4Args a, unsigned copies)
{
    if (blockIdx.x < copies) {
        to_planes(a, blockIdx.x);
        return;
    }
    typedef typename Ty<DT>::T T;
    constexpr int W = DT == DT_F32 ? 8 : 4;
    const unsigned per_row = 4u * a.kb;
    const long long first = (long long)(blockIdx.x - copies) * (kQuantThreads * kQuantEach);
    const long long row0 = first / per_row;
    const unsigned rem0 = (unsigned)(first - row0 * per_row);
    unsigned x[kQuantEach][W];
    long long row[kQuantEach];
    unsigned q[kQuantEach];
#pragma unroll
    for (int i = 0; i < kQuantEach; ++i) {
        const unsigned at = rem0 + threadIdx.x + i * kQuantThreads;
        const unsigned down = at / per_row;
        row[i] = row0 + down;
        q[i] = at - down * per_row;
        // Lanes past the last row: no values, and nothing is stored.
        const int n = row[i] < a.rows ? a.K - (int)q[i] * 8 : 0;
        load_words<DT, ALIGNED>(static_cast<const T*>(a.x) + (n > 0 ? row[i] * a.ldx + q[i] * 8 : 0), n, x[i]);
    }
#pragma unroll
    for (int i = 0; i < kQuantEach; ++i) {
        unsigned m = 0;
#pragma unroll
        for (int j = 0; j < W; ++j) m = max_bits<DT>(m, x[i][j]);
        if (DT != DT_F32) m = max(m & 0xFFFFu, m >> 16);
        m = max(m, quad<0xB1>(m));   // lanes 1 0 3 2
        m = max(m, quad<0x4E>(m));   // lanes 2 3 0 1
        const unsigned code = scale_code<DT>(m);
        const unsigned c = to_codes<DT>(x[i], code);
        if (a.planes) {   // a dword of four blocks: 16 lanes of one row
            unsigned d = code << (8 * (q[i] >> 2 & 3));
            d |= __builtin_amdgcn_update_dpp(0u, d, 0x124, 0xF, 0xF, true);   // of 4, then 8 lanes round
            d |= __builtin_amdgcn_update_dpp(0u, d, 0x128, 0xF, 0xF, true);
            if ((q[i] & 15) == 0 && row[i] < a.rows) reinterpret_cast<unsigned*>(a.scales)[(q[i] >> 4) * scale_rows(a.rows) + row[i]] = d;
        }
        if (row[i] < a.rows) {
            reinterpret_cast<unsigned*>(a.codes)[row[i] * per_row + q[i]] = c;
            if (!a.planes && (q[i] & 3) == 0) a.scales[row[i] * a.kb + (q[i] >> 2)] = (unsigned char)code;
        }
    }
}

// X given as K rows: a lane takes 16 bytes (C columns) of the 32 rows of a
// block, eight lanes a 128-byte line, eight blocks a wave: what a wave stores
// for a column is 128 bytes again. All 32 loads of a lane are under way at
// once (32 KB a wave).
template <int DT, bool ALIGNED>
__global__ void __launch_bounds__(256) quant4_cols_kernel(Quant4Args a, int groups)
{
    typedef typename Ty<DT>::T T;
    constexpr int C = DT == DT_F32 ? 4 : 8;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int down = blockIdx.x / groups, over = blockIdx.x - down * groups;
    const int kb = down * 8 + lane / 8;
    const long long c0 = ((long long)over * 4 + wave) * 8 * C + (lane % 8) * C;
    const long long left = a.rows - c0;
    if (kb >= a.kb || left <= 0) return;
    const int n = left < C ? (int)left : C;
    unsigned r[32][4];
    const T* p = static_cast<const T*>(a.x) + (long long)kb * 32 * a.ldx + c0;
#pragma unroll
    for (int k = 0; k < 32; ++k) {
        const bool in = kb * 32 + k < a.K;
        load_words<DT, ALIGNED>(in ? p + k * a.ldx : p, in ? n : 0, r[k]);
    }
    unsigned m[4] = {0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < 32; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) m[j] = max_bits<DT>(m[j], r[k][j]);
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int w = C == 8 ? c / 2 : c;
        const unsigned code = scale_code<DT>(C == 8 && (c & 1) ? m[w] >> 16 : m[w]);
        u4 out;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            if constexpr (DT == DT_F32) {
                unsigned v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = r[8 * g + i][w];
                out[g] = to_codes<DT>(v, code);
            } else {
                unsigned v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)   // the column's values of two rows
                    v[i] = __builtin_amdgcn_perm(r[8 * g + 2 * i + 1][w], r[8 * g + 2 * i][w], c & 1 ? 0x07060302u : 0x05040100u);
                out[g] = to_codes<DT>(v, code);
            }
        }
        if (c < n) {
            *reinterpret_cast<u4*>(a.codes + ((c0 + c) * a.kb + kb) * 16) = out;
            a.scales[(c0 + c) * a.kb + kb] = (unsigned char)code;
        }
    }
}

// Eight codes to eight values, a quarter of a block a lane as above.
template <int DT, int W>
__device__ __forceinline__ void from_codes(unsigned c, unsigned code, unsigned (&x)[W])
{
    const float s = __uint_as_float(code << 23);
    if constexpr (DT == DT_F32) {
        const f2 v[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 0), __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 1),
                         __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 2), __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 3)};
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = code == 255 ? 0x7FC00000u : __float_as_uint(v[i / 2][i % 2]);
    } else if constexpr (DT == DT_BF16) {
        x[0] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 0));
        x[1] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 1));
        x[2] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 2));
        x[3] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 3));
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = code == 255 ? 0x7FC07FC0u : x[i];
    } else {
        x[0] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, s, 0));
        x[1] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, s, 1));
        x[2] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, s, 2));
        x[3] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, s, 3));
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = code == 255 ? 0x7E007E00u : x[i];
    }
}

// Eight packed values to p, the first `n` of them; 16-bit values that start
// inside a word as two halves and the three words between.
template <int DT, bool ALIGNED, int W>
__device__ __forceinline__ void store_words(typename Ty<DT>::T* p, int n, const unsigned (&r)[W])
{
    unsigned* w = reinterpret_cast<unsigned*>(p);
    if (n >= 8) {
        if constexpr (DT == DT_F32) {
            if (ALIGNED) {
                *reinterpret_cast<u4*>(w) = u4{r[0], r[1], r[2], r[3]};
                *reinterpret_cast<u4*>(w + 4) = u4{r[4], r[5], r[6], r[7]};
            } else {
                *reinterpret_cast<u4w*>(w) = u4{r[0], r[1], r[2], r[3]};
                *reinterpret_cast<u4w*>(w + 4) = u4{r[4], r[5], r[6], r[7]};
            }
        } else if (ALIGNED) {
            *reinterpret_cast<u4*>(w) = u4{r[0], r[1], r[2], r[3]};
        } else if ((reinterpret_cast<unsigned long long>(p) & 2) == 0) {
            *reinterpret_cast<u4w*>(w) = u4{r[0], r[1], r[2], r[3]};
        } else {
            unsigned short* h = reinterpret_cast<unsigned short*>(p);
            h[0] = (unsigned short)r[0];
            *reinterpret_cast<u3w*>(h + 1) = u3w{__builtin_amdgcn_alignbit(r[1], r[0], 16), __builtin_amdgcn_alignbit(r[2], r[1], 16),
                                                 __builtin_amdgcn_alignbit(r[3], r[2], 16)};
            h[7] = (unsigned short)(r[3] >> 16);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 7; ++i) {
        if (i >= n) return;
        if constexpr (DT == DT_F32) w[i] = r[i];
        else reinterpret_cast<unsigned short*>(p)[i] = (unsigned short)(i & 1 ? r[i / 2] >> 16 : r[i / 2]);
    }
}

template <int DT, bool ALIGNED>
__global__ void __launch_bounds__(kQuantThreads) dequant4_kernel(Dequant4Args a)
{
    typedef typename Ty<DT>::T T;
    constexpr int W = DT == DT_F32 ? 8 : 4;
    const unsigned per_row = 4u * a.kb;
    const long long first = (long long)blockIdx.x * (kQuantThreads * kQuantEach);
    const long long row0 = first / per_row;
    const unsigned rem0 = (unsigned)(first - row0 * per_row);
    unsigned c[kQuantEach], s[kQuantEach], q[kQuantEach];
    long long row[kQuantEach];
#pragma unroll
    for (int i = 0; i < kQuantEach; ++i) {
        const unsigned at = rem0 + threadIdx.x + i * kQuantThreads;
        const unsigned down = at / per_row;
        row[i] = row0 + down;
        q[i] = at - down * per_row;
        const bool in = row[i] < a.rows;
        c[i] = reinterpret_cast<const unsigned*>(a.codes)[in ? row[i] * per_row + q[i] : 0];
        s[i] = a.scales[in ? row[i] * a.kb + (q[i] >> 2) : 0];
    }
#pragma unroll
    for (int i = 0; i < kQuantEach; ++i) {
        unsigned x[W];
        from_codes<DT>(c[i], s[i], x);
        const int n = row[i] < a.rows ? a.K - (int)q[i] * 8 : 0;
        if (n > 0) store_words<DT, ALIGNED>(static_cast<T*>(a.x) + row[i] * a.ldx + q[i] * 8, n, x);
    }
}

// Four values a lane where the results' rows allow one store for them.
template <int DT, int E>
__global__ void __launch_bounds__(256) join4_kernel(Join4Args a)
{
    typedef typename Ty<DT>::T T;
    typedef float Fe __attribute__((ext_vector_type(E)));
    typedef T Te __attribute__((ext_vector_type(E)));
    const long long n = a.rows * a.cols;
    for (long long i = (blockIdx.x * 256ll + threadIdx.x) * E; i < n; i += gridDim.x * 256ll * E) {
        Fe v = *reinterpret_cast<const Fe*>(a.src + i);
        for (int p = 1; p < a.parts; ++p) v += *reinterpret_cast<const Fe*>(a.src + p * n + i);
        const long long row = i / a.cols;
        Te r;
#pragma unroll
        for (int e = 0; e < E; ++e) r[e] = (T)v[e];
        *reinterpret_cast<Te*>(static_cast<T*>(a.dst) + row * a.ldd + (i - row * a.cols)) = r;
    }
}

bool on16(const void* p, long long ld, int es) { return (reinterpret_cast<unsigned long long>(p) & 15) == 0 && ld * es % 16 == 0; }

}  // namespace

hipError_t launch_quant4(int dtype, bool trans, const Quant4Args& a, hipStream_t s)
{
    const int es = dtype == DT_F32 ? 4 : 2;
    const bool al = on16(a.x, a.ldx, es);
    if (trans) {
        const long long cols = 4 * 8 * 16 / es;
        const long long groups = (a.rows + cols - 1) / cols, down = (a.kb + 7) / 8;
        typedef void (*Fn)(Quant4Args, int);
        static const Fn fn[3][2] = {{quant4_cols_kernel<DT_F32, false>, quant4_cols_kernel<DT_F32, true>},
                                    {quant4_cols_kernel<DT_BF16, false>, quant4_cols_kernel<DT_BF16, true>},
                                    {quant4_cols_kernel<DT_F16, false>, quant4_cols_kernel<DT_F16, true>}};
        hipLaunchKernelGGL(fn[dtype][al], dim3((unsigned)(groups * down)), dim3(256), 0, s, a, (int)groups);
        return hipGetLastError();
    }
    const long long pieces = a.rows * a.kb * 4, each = kQuantThreads * kQuantEach;
    const long long blocks = (pieces + each - 1) / each;
    const long long copies = (a.plane_rows + kQuantThreads - 1) / kQuantThreads * ((a.kb / 4 + kPlanesEach - 1) / kPlanesEach);
    typedef void (*Fn)(Quant4Args, unsigned);
    static const Fn fn[3][2] = {{quant4_rows_kernel<DT_F32, false>, quant4_rows_kernel<DT_F32, true>},
                                {quant4_rows_kernel<DT_BF16, false>, quant4_rows_kernel<DT_BF16, true>},
                                {quant4_rows_kernel<DT_F16, false>, quant4_rows_kernel<DT_F16, true>}};
    hipLaunchKernelGGL(fn[dtype][al], dim3((unsigned)(blocks + copies)), dim3(kQuantThreads), 0, s, a,
                       (unsigned)copies);
    return hipGetLastError();
}

hipError_t launch_dequant4(int dtype, const Dequant4Args& a, hipStream_t s)
{
    const bool al = on16(a.x, a.ldx, dtype == DT_F32 ? 4 : 2);
    const long long pieces = a.rows * a.kb * 4, each = kQuantThreads * kQuantEach;
    typedef void (*Fn)(Dequant4Args);
    static const Fn fn[3][2] = {{dequant4_kernel<DT_F32, false>, dequant4_kernel<DT_F32, true>},
                                {dequant4_kernel<DT_BF16, false>, dequant4_kernel<DT_BF16, true>},
                                {dequant4_kernel<DT_F16, false>, dequant4_kernel<DT_F16, true>}};
    hipLaunchKernelGGL(fn[dtype][al], dim3((unsigned)((pieces + each - 1) / each)), dim3(kQuantThreads), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_join4(int dtype, const Join4Args& a, hipStream_t s)
{
    const int es = dtype == DT_F32 ? 4 : 2;
    const bool four = a.cols % 4 == 0 && a.ldd % 4 == 0 && (unsigned long long)a.dst % (4 * es) == 0;
    const long long n = (a.rows * a.cols / (four ? 4 : 1) + 255) / 256;
    typedef void (*Fn)(Join4Args);
    static const Fn fn[3][2] = {{join4_kernel<DT_F32, 1>, join4_kernel<DT_F32, 4>}, {join4_kernel<DT_BF16, 1>, join4_kernel<DT_BF16, 4>},
                                {join4_kernel<DT_F16, 1>, join4_kernel<DT_F16, 4>}};
    hipLaunchKernelGGL(fn[dtype][four], dim3((unsigned)(n < 8192 ? n : 8192)), dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace sam
