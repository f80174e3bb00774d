// Kernels of the distillation loss (formulas in sam_distill.h).
//
// Bound by memory: a row's logits are read once and its gradient written
// once. The loss kernel gives a row to one workgroup, which keeps it in
// registers between the softmax's sum and the gradient; of a row too long for
// registers and LDS the rest is read again.
#include "sam_distill.h"

namespace sam {

namespace {

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

// The registers as they are, not what an earlier use made of them: without it
// the compiler keeps 16-bit rows as floats from one use to the next, twice
// the registers.
template <int P>
__device__ __forceinline__ void as_read(u4 (&r)[P])
{
#pragma unroll
    for (int q = 0; q < P; ++q) asm volatile("" : "+v"(r[q]));
}

// 2^x with the hardware's instruction (x <= 0 here but for a pivot that is
// not the largest value): within 1 unit in the last place of FP32, results
// under 2^-126 become zero.
__device__ __forceinline__ float pow2(float x) { return __builtin_amdgcn_exp2f(x); }

__device__ __forceinline__ float teacher_at(const DistillArgs& a, long long i)
{
    if (a.t_dtype == DT_F32) return static_cast<const float*>(a.t)[i];
    if (a.t_dtype == DT_BF16) return (float)static_cast<const __bf16*>(a.t)[i];
    return (float)static_cast<const _Float16*>(a.t)[i];
}

template <int NT, class F>
__device__ __forceinline__ float block_reduce(float v, float* s, F op)
{
#pragma unroll
    for (int d = 32; d; d >>= 1) v = op(v, __shfl_xor(v, d));
    if constexpr (NT > 64) {
        __syncthreads();   // the last use of s is over
        if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
        __syncthreads();
        v = s[0];
#pragma unroll
        for (int w = 1; w < NT / 64; ++w) v = op(v, s[w]);
    }
    return v;
}

// A row's teacher distribution: p[j] and index[j] (-1: empty) in LDS. Returns
// the sum of the unnormalised weights, 0 if no entry is valid; best: their
// pivot.
template <int NT>
__device__ __forceinline__ float teacher_row(const DistillArgs& a, long long row, float* p, int* idx, float* red, float& best)
{
    float m = -INFINITY;
    for (int j = threadIdx.x; j < a.top; j += NT) {
        const int i = a.index[row * a.top + j];
        const bool ok = (unsigned)i < (unsigned)a.V;
        const float t = ok ? teacher_at(a, row * a.top + j) : -INFINITY;
        idx[j] = ok ? i : -1;
        p[j] = t;
        m = fmaxf(m, t);
    }
    best = block_reduce<NT>(m, red, [](float x, float y) { return fmaxf(x, y); });
    const float pivot = best > -INFINITY ? best : 0.0f;
    float sum = 0.0f;
    for (int j = threadIdx.x; j < a.top; j += NT) {
        const float e = expf((p[j] - pivot) / a.T);
        sum += e;
    }
    return block_reduce<NT>(sum, red, [](float x, float y) { return x + y; });
}

// p of all entries with entry j's index, or a negative value unless j is the
// first of them.
__device__ __forceinline__ float total_p(const DistillArgs& a, const float* p, const int* idx, int j)
{
    const int i = idx[j];
    if (i < 0) return -1.0f;
    float sum = 0.0f;
    bool first = true;
    for (int o = 0; o < a.top; ++o)
        if (idx[o] == i) {
            first &= o >= j;
            sum += p[o];
        }
    return first ? sum : -1.0f;
}

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

// P pieces of a row stay in each thread's registers and L more in its own
// place in LDS; what is left of a longer row is read again for the gradient.
template <int DT, int NT, int P, int L, bool GRAD>
__global__ void __launch_bounds__(NT) distill_kernel(DistillArgs a)
{
    typedef Piece<DT> Pc;
    typedef typename Pc::T T;
    constexpr int E = Pc::E;
    __shared__ u4 hold[L > 0 ? L * NT : 1];
    __shared__ float p[kMaxTop];
    __shared__ int idx[kMaxTop];
    __shared__ float red[2][NT / 64];
    const int tid = threadIdx.x;
    const long long row = blockIdx.x;
    const T* z = static_cast<const T*>(a.z) + row * a.ldz;
    T* g = static_cast<T*>(a.grad) + row * a.ldg;
    const float w = a.weight ? a.weight[row] : 1.0f;
    const Span sp = span_of<DT>(z, a.V);
    const u4* zb = reinterpret_cast<const u4*>(z + sp.head);
    u4* gb = reinterpret_cast<u4*>(g + sp.head);
    const bool whole = (((unsigned long long)gb) & 15) == 0;
    auto write = [&](int i, const u4& x) {
        if (whole) {
            gb[i] = x;
        } else {
            const T* h = reinterpret_cast<const T*>(&x);
#pragma unroll
            for (int k = 0; k < E; ++k) g[sp.head + (long long)i * E + k] = h[k];
        }
    };
    // Values outside the pieces: at most E - 1 at either end, a thread each.
    int edge_at = -1;
    if (tid < sp.head) edge_at = tid;
    if (tid >= 32 && tid - 32 < a.V - sp.tail0) edge_at = sp.tail0 + tid - 32;
    if (GRAD && w == 0.0f) {
        // A row that is not trained on: its logits are not read.
        for (int i = tid; i < sp.pieces; i += NT) write(i, u4{0u, 0u, 0u, 0u});
        if (edge_at >= 0) g[edge_at] = (T)0.0f;
        if (a.loss && tid == 0) a.loss[row] = 0.0f;
        return;
    }

    // The row's loads first; the teacher's part runs while they are under way.
    u4 r[P];
#pragma unroll
    for (int q = 0; q < P; ++q) {
        const int i = tid + q * NT;
        r[q] = Pc::masked();
        if (i < sp.pieces) r[q] = zb[i];
    }
    float edge = -INFINITY;
    if (edge_at >= 0) edge = (float)z[edge_at];

    float best;
    const float psum = teacher_row<NT>(a, row, p, idx, red[0], best);

    // This thread's largest value, then the row's, and the row's sum of
    // 2^((z - m) scale). Values not in registers: a running maximum and sum,
    // four pieces at a time.
    float m = edge;
#pragma unroll
    for (int q = 0; q < P; ++q) {
        float v[E];
        Pc::get(r[q], v);
#pragma unroll
        for (int i = 0; i < E; ++i) m = fmaxf(m, v[i]);
    }
    float mx = -INFINITY, sx = 0.0f;
    auto running = [&](const u4 (&x)[4]) {
        float n = mx;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            float v[E];
            Pc::get(x[b], v);
#pragma unroll
            for (int i = 0; i < E; ++i) n = fmaxf(n, v[i]);
        }
        const float pv = n > -INFINITY ? n : 0.0f;
        if (mx > -INFINITY) sx *= pow2((mx - pv) * a.scale);
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            float v[E];
            Pc::get(x[b], v);
#pragma unroll
            for (int i = 0; i < E; ++i) sx += pow2((v[i] - pv) * a.scale);
        }
        mx = n;
    };
#pragma unroll
    for (int o = 0; o < L; o += 4) {
        u4 x[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const int i = tid + (P + o + b) * NT;
            x[b] = Pc::masked();
            if (i < sp.pieces) x[b] = zb[i];
        }
#pragma unroll
        for (int b = 0; b < 4; ++b) hold[(o + b) * NT + tid] = x[b];
        running(x);
    }
    for (int i0 = tid + (P + L) * NT; i0 < sp.pieces; i0 += 4 * NT) {
        u4 x[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            x[b] = Pc::masked();
            if (i0 + b * NT < sp.pieces) x[b] = zb[i0 + b * NT];
        }
        running(x);
    }
    as_read(r);
    m = block_reduce<NT>(fmaxf(m, mx), red[1], [](float x, float y) { return fmaxf(x, y); });
    const float pivot = m > -INFINITY ? m : 0.0f;
    // mx = -inf with a sum: NaN values, which stay.
    float s = pow2((edge - pivot) * a.scale) + (mx > -INFINITY ? sx * pow2((mx - pivot) * a.scale) : sx);
#pragma unroll
    for (int q = 0; q < P; ++q) {
        float v[E];
        Pc::get(r[q], v);
#pragma unroll
        for (int i = 0; i < E; ++i) s += pow2((v[i] - pivot) * a.scale);
    }
    as_read(r);
    s = block_reduce<NT>(s, red[0], [](float x, float y) { return x + y; });

    // The loss, entry by entry; p[j] becomes the probability. A row takes
    // part if the teacher has an entry and the student a logit above -inf.
    const bool on = w != 0.0f && !(psum == 0.0f) && !(s == 0.0f);
    const float ls = logf(s), lp = logf(psum);
    const float tp = best > -INFINITY ? best : 0.0f;
    float sum = 0.0f;
    for (int j = tid; j < a.top; j += NT) {
        const float lt = (p[j] - tp) / a.T;
        const float pj = idx[j] >= 0 ? expf(lt) / psum : 0.0f;
        if (on && !(pj == 0.0f)) sum += pj * (lt - lp - (((float)z[idx[j]] - pivot) / a.T - ls));
        p[j] = pj;
    }
    sum = block_reduce<NT>(sum, red[1], [](float x, float y) { return x + y; });
    if (tid == 0) {
        if (a.loss) a.loss[row] = on ? w * a.T * a.T * sum : 0.0f;
        if (a.lse) a.lse[row] = s == 0.0f ? -INFINITY : (float)((double)pivot / a.T + (double)ls);
    }
    if constexpr (GRAD) {
        const float wt = w * a.T, f = on ? wt / s : 0.0f;
        // The entries' own logits are read before any of the row is written
        // (the gradient may take the logits' place). Every index is written
        // once more after the row, by its first entry.
        constexpr int MORE = (kMaxTop + NT - 1) / NT;
        float gv[MORE];
        int gat[MORE];
#pragma unroll
        for (int o = 0; o < MORE; ++o) {
            const int j = tid + o * NT;
            gat[o] = -1;
            if (on && j < a.top) {
                const float pt = total_p(a, p, idx, j);
                if (!(pt < 0.0f)) {
                    gat[o] = idx[j];
                    gv[o] = wt * (pow2(((float)z[idx[j]] - pivot) * a.scale) / s - pt);
                }
            }
        }
        __syncthreads();
        auto grad_of = [&](const u4& x) {
            float v[E];
            Pc::get(x, v);
#pragma unroll
            for (int i = 0; i < E; ++i) v[i] = on ? f * pow2((v[i] - pivot) * a.scale) : 0.0f;
            return Pc::put(v);
        };
#pragma unroll
        for (int q = 0; q < P; ++q) {
            const int i = tid + q * NT;
            if (i < sp.pieces) write(i, grad_of(r[q]));
        }
#pragma unroll
        for (int o = 0; o < L; ++o) {
            const int i = tid + (P + o) * NT;
            if (i < sp.pieces) write(i, grad_of(hold[o * NT + tid]));
        }
        for (int i0 = tid + (P + L) * NT; i0 < sp.pieces; i0 += 4 * NT) {
            u4 x[4];
#pragma unroll
            for (int b = 0; b < 4; ++b)
                if (i0 + b * NT < sp.pieces) x[b] = zb[i0 + b * NT];
#pragma unroll
            for (int b = 0; b < 4; ++b)
                if (i0 + b * NT < sp.pieces) write(i0 + b * NT, grad_of(x[b]));
        }
        if (edge_at >= 0) g[edge_at] = (T)(on ? f * pow2((edge - pivot) * a.scale) : 0.0f);
        __syncthreads();
#pragma unroll
        for (int o = 0; o < MORE; ++o)
            if (gat[o] >= 0) g[gat[o]] = (T)gv[o];
    }
}

// The gradient from a given lse: no sum over the row, so a row is cut into
// strips of 64 KB, a workgroup each.
constexpr int kGradThreads = 256, kGradPieces = 16;

template <int DT>
__global__ void __launch_bounds__(kGradThreads) distill_grad_kernel(DistillArgs a, int strips)
{
    typedef Piece<DT> Pc;
    typedef typename Pc::T T;
    constexpr int E = Pc::E, NT = kGradThreads, P = kGradPieces;
    __shared__ float p[kMaxTop];
    __shared__ int idx[kMaxTop];
    __shared__ float red[NT / 64];
    const int tid = threadIdx.x;
    const long long row = blockIdx.x / strips;
    const int strip = blockIdx.x % strips;
    const T* z = static_cast<const T*>(a.z) + row * a.ldz;
    T* g = static_cast<T*>(a.grad) + row * a.ldg;
    const float w = a.weight ? a.weight[row] : 1.0f;
    const float lse = a.lse[row];
    const Span sp = span_of<DT>(z, a.V);
    const u4* zb = reinterpret_cast<const u4*>(z + sp.head);
    u4* gb = reinterpret_cast<u4*>(g + sp.head);
    const bool whole = (((unsigned long long)gb) & 15) == 0;
    const int first = strip * NT * P;
    u4 r[P];
#pragma unroll
    for (int q = 0; q < P; ++q) {
        const int i = first + tid + q * NT;
        r[q] = Pc::masked();
        if (i < sp.pieces) r[q] = zb[i];
    }
    // The first strip takes the values before the pieces, the last those behind.
    float edge = 0.0f;
    int edge_at = -1;
    if (strip == 0 && tid < sp.head) edge_at = tid;
    if (strip == strips - 1 && tid >= 32 && tid - 32 < a.V - sp.tail0) edge_at = sp.tail0 + tid - 32;
    if (edge_at >= 0) edge = (float)z[edge_at];
    const int begin = strip == 0 ? 0 : sp.head + first * E;
    const int end = strip == strips - 1 ? a.V : sp.head + (first + NT * P) * E;

    float best;
    const float psum = teacher_row<NT>(a, row, p, idx, red, best);
    const bool on = w != 0.0f && !(psum == 0.0f) && !(lse == -INFINITY);
    const float tp = best > -INFINITY ? best : 0.0f;
    for (int j = tid; j < a.top; j += NT) p[j] = idx[j] >= 0 ? expf((p[j] - tp) / a.T) / psum : 0.0f;
    __syncthreads();
    const float wt = w * a.T;
    // lse is at least every v / T; where its rounding says otherwise (it is
    // coarse for logits next to a type's lowest value) q is 1, not more. A NaN
    // stays one.
    auto q_of = [&](float v) {
        const float d = fmaf(v, a.inv_hi, -lse) + v * a.inv_lo;
        return pow2((d > 0.0f ? 0.0f : d) * 1.44269504088896341f);
    };
    constexpr int MORE = kMaxTop / NT;
    float gv[MORE];
    int gat[MORE];
#pragma unroll
    for (int o = 0; o < MORE; ++o) {
        const int j = tid + o * NT;
        gat[o] = -1;
        if (on && j < a.top && idx[j] >= begin && idx[j] < end) {
            const float pt = total_p(a, p, idx, j);
            if (!(pt < 0.0f)) {
                gat[o] = idx[j];
                const float v = (float)z[idx[j]];
                gv[o] = wt * ((v == -INFINITY ? 0.0f : q_of(v)) - pt);
            }
        }
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < P; ++q) {
        const int i = first + tid + q * NT;
        if (i < sp.pieces) {
            float v[E];
            Pc::get(r[q], v);
#pragma unroll
            for (int k = 0; k < E; ++k) v[k] = !on || v[k] == -INFINITY ? 0.0f : wt * q_of(v[k]);
            const u4 x = Pc::put(v);
            if (whole) {
                gb[i] = x;
            } else {
                const T* h = reinterpret_cast<const T*>(&x);
#pragma unroll
                for (int k = 0; k < E; ++k) g[sp.head + (long long)i * E + k] = h[k];
            }
        }
    }
    if (edge_at >= 0) g[edge_at] = (T)(!on || edge == -INFINITY ? 0.0f : wt * q_of(edge));
    __syncthreads();
#pragma unroll
    for (int o = 0; o < MORE; ++o)
        if (gat[o] >= 0) g[gat[o]] = (T)gv[o];
}

template <int DT, int NT, int P, int L>
hipError_t run(const DistillArgs& a, hipStream_t s)
{
    const dim3 grid((unsigned)a.rows), block(NT);
    if (a.grad)
        hipLaunchKernelGGL((distill_kernel<DT, NT, P, L, true>), grid, block, 0, s, a);
    else   // the loss alone has no use for what it has read
        hipLaunchKernelGGL((distill_kernel<DT, NT, P, 0, false>), grid, block, 0, s, a);
    return hipGetLastError();
}

// Threads and registers by the row's length; few rows: as many threads as
// fit, for latency.
template <int DT>
hipError_t pick(const DistillArgs& a, hipStream_t s)
{
    const long long pieces = ((long long)a.V + Piece<DT>::E - 1) / Piece<DT>::E;
    const bool few = a.rows <= 256;
    if (pieces <= 256 * 4) return run<DT, 256, 4, 0>(a, s);
    if (few && pieces <= 1024 * 4) return run<DT, 1024, 4, 0>(a, s);
    if (few && pieces <= 1024 * 8) return run<DT, 1024, 8, 0>(a, s);
    if (pieces <= 256 * 8) return run<DT, 256, 8, 0>(a, s);
    if (pieces <= 256 * 16) return run<DT, 256, 16, 0>(a, s);
    if (pieces <= 512 * 16) return run<DT, 512, 16, 0>(a, s);
    if (pieces <= 1024 * 16) return run<DT, 1024, 16, 0>(a, s);
    return run<DT, 1024, 20, 8>(a, s);
}

}  // namespace

hipError_t launch_distill(int dtype, const DistillArgs& a, hipStream_t s)
{
    if (dtype == DT_F32) return pick<DT_F32>(a, s);
    return dtype == DT_BF16 ? pick<DT_BF16>(a, s) : pick<DT_F16>(a, s);
}

hipError_t launch_distill_grad(int dtype, const DistillArgs& a, hipStream_t s)
{
    const long long e = dtype == DT_F32 ? 4 : 8;
    const long long per = (long long)kGradThreads * kGradPieces * e;
    const int strips = (int)((a.V + per - 1) / per);
    const dim3 grid((unsigned)(a.rows * strips)), block(kGradThreads);
    if (dtype == DT_F32)
        hipLaunchKernelGGL((distill_grad_kernel<DT_F32>), grid, block, 0, s, a, strips);
    else if (dtype == DT_BF16)
        hipLaunchKernelGGL((distill_grad_kernel<DT_BF16>), grid, block, 0, s, a, strips);
    else
        hipLaunchKernelGGL((distill_grad_kernel<DT_F16>), grid, block, 0, s, a, strips);
    return hipGetLastError();
}

}  // namespace sam
