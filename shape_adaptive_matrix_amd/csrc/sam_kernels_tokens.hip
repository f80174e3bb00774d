// Kernels of the token log probabilities (formulas in sam_tokens.h).
#include "sam_tokens.h"

namespace sam {

namespace {

template <int DT> struct Ty;
template <> struct Ty<DT_F32> { typedef float T; };
template <> struct Ty<DT_BF16> { typedef __bf16 T; };
template <> struct Ty<DT_F16> { typedef _Float16 T; };

constexpr int kThreads = 256;

// Whole numbers that order values: NaN above all, the two zeros equal.
__device__ __forceinline__ unsigned order_of(float v)
{
    const unsigned b = __float_as_uint(v + 0.0f);
    if (v != v) return 0xFFFFFFF0u;
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float value_of(unsigned k)
{
    return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}

template <class V, class F>
__device__ __forceinline__ V block_reduce(V v, V* s, F op)
{
    __syncthreads();
    s[threadIdx.x] = v;
    __syncthreads();
    for (int d = kThreads / 2; d; d >>= 1) {
        if ((int)threadIdx.x < d) s[threadIdx.x] = op(s[threadIdx.x], s[threadIdx.x + d]);
        __syncthreads();
    }
    return s[0];
}

template <int DT>
__global__ void __launch_bounds__(kThreads) tokens_kernel(TokenArgs a)
{
    typedef typename Ty<DT>::T T;
    typedef unsigned long long u64;
    __shared__ float sf[kThreads];
    __shared__ u64 su[kThreads];
    const long long row = blockIdx.x;
    const T* z = static_cast<const T*>(a.z) + row * a.ldz;
    float m = -INFINITY;
    for (int j = threadIdx.x; j < a.V; j += kThreads) m = fmaxf(m, (float)z[j]);
    m = block_reduce(m, sf, [](float x, float y) { return fmaxf(x, y); });
    const float pivot = m == -INFINITY ? 0.0f : m;
    float s = 0.0f, h = 0.0f;
    for (int j = threadIdx.x; j < a.V; j += kThreads) {
        const float d = ((float)z[j] - pivot) * a.scale;
        const float e = exp2f(d);
        s += e;
        h += e == 0.0f ? 0.0f : e * d;
    }
    auto add = [](float x, float y) { return x + y; };
    s = block_reduce(s, sf, add);
    h = block_reduce(h, sf, add);
    const float L = logf(s), ln2 = 0.69314718f;
    auto logp = [&](float v) { return v == -INFINITY ? v - L : (v - pivot) * a.inv_hi + (v - pivot) * a.inv_lo - L; };
    if (threadIdx.x == 0) {
        const int t = a.token[row];
        a.logprob[row] = (unsigned)t < (unsigned)a.V ? (L == -INFINITY ? L : logp((float)z[t])) : 0.0f;
        a.entropy[row] = L == -INFINITY ? 0.0f : L - ln2 * h / s;
        a.norm[2 * row] = m;
        a.norm[2 * row + 1] = L;
    }
    u64 last = ~0ull;
    for (int k = 0; k < a.top; ++k) {
        u64 best = 0;
        for (int j = threadIdx.x; j < a.V; j += kThreads) {
            const u64 c = (u64)order_of((float)z[j]) << 32 | (unsigned)~j;
            if (c < last && c > best) best = c;
        }
        last = block_reduce(best, su, [](u64 x, u64 y) { return x > y ? x : y; });
        if (threadIdx.x == 0) {
            const float v = value_of((unsigned)(last >> 32));
            a.top_logprob[row * a.top + k] = L == -INFINITY ? L : logp(v);
            a.top_index[row * a.top + k] = (int)~(unsigned)last;
        }
    }
}

template <int DT>
__global__ void __launch_bounds__(kThreads) tokens_grad_kernel(TokenGradArgs a)
{
    typedef typename Ty<DT>::T T;
    const long long row = blockIdx.x;
    const T* z = static_cast<const T*>(a.z) + row * a.ldz;
    T* g = static_cast<T*>(a.grad) + row * a.ldg;
    const int t = a.token[row];
    const bool has = (unsigned)t < (unsigned)a.V;
    const float u = a.u && has ? a.u[row] : 0.0f, v = a.v ? a.v[row] : 0.0f;
    const float m = a.norm[2 * row], L = a.norm[2 * row + 1], H = v != 0.0f ? a.entropy[row] : 0.0f;
    const bool off = (u == 0.0f && v == 0.0f) || L == -INFINITY;
    for (int j = threadIdx.x; j < a.V; j += kThreads) {
        float r = 0.0f;
        if (!off) {
            const float lp = ((float)z[j] - m) * a.scale * 0.69314718f - L;
            const float p = expf(lp);
            r = p == 0.0f ? 0.0f : -p * (u + v * (lp + H));
            if (j == t) r += u;
        }
        g[j] = (T)(r * a.inv);
    }
}

}  // namespace

hipError_t launch_tokens(int dtype, const TokenArgs& a, hipStream_t s)
{
    typedef void (*Fn)(TokenArgs);
    static const Fn fn[3] = {tokens_kernel<DT_F32>, tokens_kernel<DT_BF16>, tokens_kernel<DT_F16>};
    hipLaunchKernelGGL(fn[dtype], dim3((unsigned)a.rows), dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_tokens_grad(int dtype, const TokenGradArgs& a, hipStream_t s)
{
    typedef void (*Fn)(TokenGradArgs);
    static const Fn fn[3] = {tokens_grad_kernel<DT_F32>, tokens_grad_kernel<DT_BF16>, tokens_grad_kernel<DT_F16>};
    hipLaunchKernelGGL(fn[dtype], dim3((unsigned)a.rows), dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

}  // namespace sam
