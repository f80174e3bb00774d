// MXFP4 tensors made, read back, and multiplied by rows of X: kernel
// arguments and launchers (sam_kernels_mxfp4.hip; entry points in
// sam_mxfp4.cpp).
//
// A row of K values is blocks of 32 (zeros behind the last):
//   s = floor(log2(max |x|)) - 2, at least -127;  code = E2M1(x / 2^s)
// rounded to nearest, ties to the even code, at most 6; the scale byte is s +
// 127, and 255 (all codes 0) where the block holds an Inf or NaN.
#pragma once

#include "sam_internal.h"

namespace sam {

struct Quant4Args {
    const void* x;           // rows of K, stride ldx; transposed: K rows of `rows`
    long long ldx;
    long long rows;
    int K, kb;               // values and blocks a row
    unsigned char* codes;    // rows x kb x 16
    unsigned char* scales;   // rows x kb
    // For the tiles (rows' form; kb is a multiple of four then): scales as kb / 4
    // planes of scale_rows() dwords, and beside it those of another tensor,
    // plane_rows of from_kb, zeros behind a row.
    int planes;
    const unsigned char* from;
    unsigned char* to;
    long long plane_rows;
    int from_kb;
};

struct Dequant4Args {
    const unsigned char* codes;
    const unsigned char* scales;
    long long rows;
    int K, kb;
    void* x;                 // rows of K, stride ldx
    long long ldx;
};

// Partial sums added in their order, into rows of the result's type and stride.
struct Join4Args {
    const float* src;        // [parts][rows][cols]
    int parts;
    void* dst;               // stride ldd
    long long ldd;
    long long rows;
    int cols;
};

// Y = q(X) Wq^T for few rows, W streamed past them.
struct Stream4Args {
    const void* x;                  // M rows of K, stride ldx, rounded on the way; or
    long long ldx;
    const unsigned char* xc;        // ... their codes (M x kb x 16)
    const unsigned char* xs;        // and scales (M x kb)
    const unsigned char* codes;     // N x kb x 16
    const unsigned char* scales;    // N x kb
    int M, N, K, kb;
    void* y;                        // M rows of N, stride ldy
    long long ldy;
    int out;                        // type of y
};

// Whether the streaming kernels take M rows of kb blocks: up to 32, or 64
// whose codes fit into LDS (read from memory, 48 rows of 11008 values take as
// long as through the tiles).
bool stream4_takes(long long M, long long kb);
// Whether the rows are rounded in the product's own launch (xc, xs unused).
bool stream4_rounds(long long M, long long kb);
hipError_t launch_stream4(int dtype, const Stream4Args& a, hipStream_t s);

hipError_t launch_quant4(int dtype, bool trans, const Quant4Args& a, hipStream_t s);
hipError_t launch_dequant4(int dtype, const Dequant4Args& a, hipStream_t s);
hipError_t launch_join4(int dtype, const Join4Args& a, hipStream_t s);
// A product of E2M1 operands by its plan: C (or the partial sums) of type
// `out` at a.out with row stride a.ldc, Bt's rows of a.ldb values, scales in
// planes.
hipError_t launch_tile4(const Plan& p, const GemmArgs& a, int out, hipStream_t s);

}  // namespace sam
