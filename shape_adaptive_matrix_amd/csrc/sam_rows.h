// What the kernels over rows of logits share: 16-byte pieces of values as
// floats, a row's aligned pieces, reductions over a wave.
#pragma once

#include "sam_dma.h"

namespace sam {
namespace rows {

typedef unsigned int u4 __attribute__((ext_vector_type(4)));

template <int DT> struct Ty;
template <> struct Ty<DT_F32> { typedef float T; };
template <> struct Ty<DT_BF16> { typedef __bf16 T; };
template <> struct Ty<DT_F16> { typedef _Float16 T; };

// 16 bytes of logits as floats and back.
template <int DT>
struct Piece {
    typedef typename Ty<DT>::T T;
    static constexpr int E = 16 / sizeof(T);
    static __device__ __forceinline__ void get(const u4& r, float (&v)[E])
    {
        if constexpr (DT == DT_F32) {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(r[i]);
        } else if constexpr (DT == DT_BF16) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = __uint_as_float(r[i] << 16);
                v[2 * i + 1] = __uint_as_float(r[i] & 0xFFFF0000u);
            }
        } else {
            typedef _Float16 h8 __attribute__((ext_vector_type(8)));
            const h8 h = __builtin_bit_cast(h8, r);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = (float)h[i];
        }
    }
    static __device__ __forceinline__ u4 put(const float (&v)[E])
    {
        if constexpr (DT == DT_F32) {
            return u4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
        } else {
            typedef T h8 __attribute__((ext_vector_type(8)));
            h8 h;
#pragma unroll
            for (int i = 0; i < 8; ++i) h[i] = (T)v[i];
            return __builtin_bit_cast(u4, h);
        }
    }
    static __device__ __forceinline__ u4 masked()   // -inf throughout
    {
        const unsigned w = DT == DT_F32 ? 0xFF800000u : (DT == DT_BF16 ? 0xFF80FF80u : 0xFC00FC00u);
        return u4{w, w, w, w};
    }
};

// Rows are read once and written once: past the caches (a buffer access's
// non-temporal bit). Measured without it, loss and gradient: 4096 x 32768
// bf16 124 us, not 110; 1024 x 131072 FP32 234, not 219.
constexpr int kOnce = 2;

// Stores take their whole offset in the vector register. With part of it in
// the scalar one the compiler lets the next instruction overwrite the data's
// registers, and some of the 16 bytes came out as what was written there.
__device__ __forceinline__ void store_once(const u4& v, __amdgpu_buffer_rsrc_t r, int off)
{
    __builtin_amdgcn_raw_buffer_store_b128(v, r, off, 0, kOnce);
}

// 2^x with the hardware's instruction (x <= 0 here but for a pivot that is
// not the largest value): within 1 unit in the last place of FP32, results
// under 2^-126 become zero.
__device__ __forceinline__ float pow2(float x) { return __builtin_amdgcn_exp2f(x); }

// The part of a row that is whole aligned 16-byte pieces, and the values
// before it.
struct Span {
    int head, pieces, tail0;   // values before, pieces, first value behind
};

template <int DT>
__device__ __forceinline__ Span span_of(const void* p, int V)
{
    constexpr int E = Piece<DT>::E;
    const int off = (int)(((unsigned long long)p & 15) / (16 / E));
    int head = off ? E - off : 0;
    head = head < V ? head : V;
    const int pieces = (V - head) / E;
    return {head, pieces, head + pieces * E};
}

// A reduction over the wave: rows of 16 lanes by shifts, then across them;
// lane 63's result, held by the wave. id: the operation's neutral value.
template <int CTRL, int ROWS, class F>
__device__ __forceinline__ float dpp_step(float v, float id, F op)
{
    return op(v, __uint_as_float(__builtin_amdgcn_update_dpp(__float_as_uint(id), __float_as_uint(v), CTRL, ROWS, 0xF, false)));
}

template <class F>
__device__ __forceinline__ float wave_reduce(float v, float id, F op)
{
    v = dpp_step<0x111, 0xF>(v, id, op);   // from 1, 2, 4, 8 lanes below
    v = dpp_step<0x112, 0xF>(v, id, op);
    v = dpp_step<0x114, 0xF>(v, id, op);
    v = dpp_step<0x118, 0xF>(v, id, op);
    v = dpp_step<0x142, 0xA>(v, id, op);   // lane 15 of the row below
    v = dpp_step<0x143, 0xC>(v, id, op);   // lane 31
    return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), 63));
}

__device__ __forceinline__ float wave_max(float v) { return wave_reduce(v, -INFINITY, [](float x, float y) { return fmaxf(x, y); }); }
__device__ __forceinline__ float wave_sum(float v) { return wave_reduce(v, 0.0f, [](float x, float y) { return x + y; }); }

// A value that no kernel call in flight writes, by a scalar load (a vector
// load would queue behind the row's).
__device__ __forceinline__ float constant(const float* p, long long i)
{
    return reinterpret_cast<const __attribute__((address_space(4))) float*>(reinterpret_cast<unsigned long long>(p))[i];
}

}  // namespace rows
}  // namespace sam
