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
};

struct Dequant4Args {
    const unsigned char* codes;
    const unsigned char* scales;
    long long rows;
    int K, kb;
    void* x;                 // rows of K, stride ldx
    long long ldx;
};

// FP32 rows into rows of another type or stride.
struct Convert4Args {
    const float* src;        // rows x cols, compact
    void* dst;               // stride ldd
    long long ldd;
    long long rows;
    int cols;
};

hipError_t launch_quant4(int dtype, bool trans, const Quant4Args& a, hipStream_t s);
hipError_t launch_dequant4(int dtype, const Dequant4Args& a, hipStream_t s);
hipError_t launch_convert4(int dtype, const Convert4Args& a, hipStream_t s);

}  // namespace sam
