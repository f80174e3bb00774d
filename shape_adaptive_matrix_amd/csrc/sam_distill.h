// Distillation from a teacher's top logits: kernel arguments and launchers
// (sam_kernels_distill.hip; entry points in sam_distill.cpp).
//
//   p = softmax(t / T) over a row's valid entries, q = softmax(z / T)
//   loss = w T^2 sum_j p_j (log p_j - log q_j),   dz = w T (q - p)
#pragma once

#include "sam_internal.h"

namespace sam {

constexpr int kMaxTop = 1024;

struct DistillArgs {
    const void* z;       // student's logits: rows of V, stride ldz
    long long ldz;
    const void* t;       // teacher's [rows][top]
    const int* index;    // [rows][top]; outside 0 .. V - 1: an empty entry
    const float* weight; // [rows] or null (1)
    float* loss;         // [rows] or null
    float* lse;          // [rows], of z / T: written by the loss, read by the gradient alone
    void* grad;          // rows of V, stride ldg, z's type; null: no gradient
    long long ldg;
    long long rows;
    int V, top;
    int t_dtype;
    float T;
    float inv_hi, inv_lo;   // 1 / T in two pieces
    float scale;            // log2(e) / T
};

// Loss (and lse), with the gradient when a.grad is set.
hipError_t launch_distill(int dtype, const DistillArgs& a, hipStream_t s);
// The gradient from a given lse.
hipError_t launch_distill_grad(int dtype, const DistillArgs& a, hipStream_t s);

}  // namespace sam
