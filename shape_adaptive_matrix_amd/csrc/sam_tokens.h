// Log probabilities of given tokens, entropy and the most likely entries of
// rows of logits, and their gradient: kernel arguments and launchers
// (sam_kernels_tokens.hip; entry points in sam_tokens.cpp).
//
//   log p_j = (z_j - m) / T - L,  m = max z,  L = log sum exp((z - m) / T)
//   logprob = log p[token],  entropy = - sum_j p_j log p_j
//   dz_j = (u (1[j = token] - p_j) - v p_j (log p_j + entropy)) / T
#pragma once

#include "sam_internal.h"

namespace sam {

constexpr int kMaxAlternatives = 128;

struct TokenArgs {
    const void* z;         // logits: rows of V, stride ldz
    long long ldz;
    const int* token;      // [rows]; outside 0 .. V - 1: none
    long long rows;
    int V, top;
    float T;
    float inv_hi, inv_lo;  // 1 / T in two pieces
    float scale;           // log2(e) / T
    float* logprob;        // [rows]
    float* entropy;        // [rows]
    float* norm;           // [rows][2]: m, L
    float* top_logprob;    // [rows][top]
    int* top_index;        // [rows][top]
    // Rows cut over workgroups: what each leaves of its part of a row, and
    // then `top` candidates of each, the best first.
    int parts;
    float4* part;          // [rows][parts]: m, sum exp without m's own 1, sum of exp times exponent, number of candidates
    float* z_token;        // [rows]: the token's logit
    unsigned long long* list;   // [rows][parts][top]
};

// Workgroups that a row is cut over.
int tokens_parts(int dtype, long long rows, long long V, long long top);
constexpr int kMaxParts = 64;

struct TokenGradArgs {
    const void* z;
    long long ldz;
    const int* token;
    long long rows;
    int V;
    float T;
    float inv;             // 1 / T
    float scale;           // log2(e) / T
    const float* norm;     // [rows][2]
    const float* entropy;  // [rows]; null where dentropy is
    const float* u;        // gradient of logprob, [rows] or null
    const float* v;        // gradient of entropy, [rows] or null
    void* grad;            // rows of V, stride ldg, z's type
    long long ldg;
};

hipError_t launch_tokens(int dtype, const TokenArgs& a, hipStream_t s);
hipError_t launch_tokens_grad(int dtype, const TokenGradArgs& a, hipStream_t s);

}  // namespace sam
