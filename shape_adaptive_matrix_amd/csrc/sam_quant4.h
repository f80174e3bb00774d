// Values to MXFP4 codes on the GPU: loads of a row's pieces, the largest value
// of a block, its scale, the codes.
#pragma once

#include "sam_internal.h"

namespace sam {
namespace quant4 {

typedef unsigned int u4 __attribute__((ext_vector_type(4)));
typedef u4 u4w __attribute__((aligned(4)));            // 16 bytes at any whole word
typedef unsigned int u3w __attribute__((ext_vector_type(3), aligned(4)));
typedef unsigned short us2 __attribute__((ext_vector_type(2)));
typedef float f2 __attribute__((ext_vector_type(2)));
typedef __bf16 b2 __attribute__((ext_vector_type(2)));
typedef _Float16 h2 __attribute__((ext_vector_type(2)));

template <int DT> struct Ty;
template <> struct Ty<DT_F32> { typedef float T; };
template <> struct Ty<DT_BF16> { typedef __bf16 T; };
template <> struct Ty<DT_F16> { typedef _Float16 T; };

// W words of values, loaded as 16-byte pieces: `n` values at p are there
// (all, unless the row ends inside), zeros behind them. ALIGNED: p is on 16
// bytes. Otherwise p is on a value, and pieces are loaded from whole words
// (16-bit values that start inside a word are shifted into place; the word
// behind then holds the last of them, so nothing outside the row's own words
// is touched).
template <int DT, bool ALIGNED, int W>
__device__ __forceinline__ void load_words(const typename Ty<DT>::T* p, int n, unsigned (&r)[W])
{
    constexpr int E = DT == DT_F32 ? W : 2 * W;
    if (n >= E) {
        if (ALIGNED || DT == DT_F32) {
#pragma unroll
            for (int i = 0; i < W; i += 4) {
                const u4 v = ALIGNED ? *reinterpret_cast<const u4*>(reinterpret_cast<const unsigned*>(p) + i)
                                     : *reinterpret_cast<const u4w*>(reinterpret_cast<const unsigned*>(p) + i);
#pragma unroll
                for (int j = 0; j < 4; ++j) r[i + j] = v[j];
            }
        } else {
            const unsigned long long at = reinterpret_cast<unsigned long long>(p);
            const unsigned* w = reinterpret_cast<const unsigned*>(at & ~3ull);
            const unsigned shift = (unsigned)(at & 2) * 8;
            unsigned v[W + 1];
#pragma unroll
            for (int i = 0; i < W; i += 4) {
                const u4 x = *reinterpret_cast<const u4w*>(w + i);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[i + j] = x[j];
            }
            v[W] = shift ? w[W] : 0;
#pragma unroll
            for (int i = 0; i < W; ++i) r[i] = __builtin_amdgcn_alignbit(v[i + 1], v[i], shift);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < W; ++i) {
        if constexpr (DT == DT_F32) {
            r[i] = i < n ? reinterpret_cast<const unsigned*>(p)[i] : 0u;
        } else {
            const unsigned short* h = reinterpret_cast<const unsigned short*>(p);
            r[i] = 2 * i < n ? h[2 * i] : 0u;
            if (2 * i + 1 < n) r[i] |= (unsigned)h[2 * i + 1] << 16;
        }
    }
}

// The largest |x| of packed words as bits that order like the values (16-bit
// types: in each half), Inf and NaN above all others.
template <int DT>
__device__ __forceinline__ unsigned max_bits(unsigned a, unsigned x)
{
    if constexpr (DT == DT_F32) {
        x &= 0x7FFFFFFFu;
        return a > x ? a : x;
    } else {
        return __builtin_bit_cast(unsigned, __builtin_elementwise_max(__builtin_bit_cast(us2, a), __builtin_bit_cast(us2, x & 0x7FFF7FFFu)));
    }
}

// Of the largest value's bits (16-bit types: in the low half), the scale byte.
template <int DT>
__device__ __forceinline__ unsigned scale_code(unsigned bits)
{
    unsigned e;
    if constexpr (DT == DT_F32) e = bits >> 23;
    else if constexpr (DT == DT_BF16) e = (bits & 0xFFFF) >> 7;
    else e = __float_as_uint((float)__builtin_bit_cast(_Float16, (unsigned short)bits)) >> 23;
    return e == 255 ? 255 : (e > 2 ? e - 2 : 0);
}

// Eight values to eight codes: pairs x[0..3] of 16-bit values, or eight floats.
template <int DT, int W>
__device__ __forceinline__ unsigned to_codes(const unsigned (&x)[W], unsigned code)
{
    const float s = __uint_as_float(code << 23);
    unsigned r = 0;
    if constexpr (DT == DT_F32) {
        static_assert(W == 8, "eight values");
        r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, __uint_as_float(x[0]), __uint_as_float(x[1]), s, 0);
        r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, __uint_as_float(x[2]), __uint_as_float(x[3]), s, 1);
        r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, __uint_as_float(x[4]), __uint_as_float(x[5]), s, 2);
        r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, __uint_as_float(x[6]), __uint_as_float(x[7]), s, 3);
    } else if constexpr (DT == DT_BF16) {
        static_assert(W == 4, "eight values");
        r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(b2, x[0]), s, 0);
        r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(b2, x[1]), s, 1);
        r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(b2, x[2]), s, 2);
        r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(b2, x[3]), s, 3);
    } else {
        static_assert(W == 4, "eight values");
        r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(r, __builtin_bit_cast(h2, x[0]), s, 0);
        r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(r, __builtin_bit_cast(h2, x[1]), s, 1);
        r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(r, __builtin_bit_cast(h2, x[2]), s, 2);
        r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(r, __builtin_bit_cast(h2, x[3]), s, 3);
    }
    return code == 255 ? 0u : r;
}

template <int CTRL>
__device__ __forceinline__ unsigned quad(unsigned v)   // of another lane of the four
{
    return __builtin_amdgcn_update_dpp(0u, v, CTRL, 0xF, 0xF, true);
}

}  // namespace quant4
}  // namespace sam
