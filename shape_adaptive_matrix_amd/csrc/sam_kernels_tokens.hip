// Kernels of the token log probabilities (formulas in sam_tokens.h).
//
// Bound by memory: a row's logits are read once for its results and once more
// for its gradient. One pass holds a thread's largest value, its sum of
// exponentials and the sum of these times their exponents (for the entropy),
// and finds the most likely entries on the way:
//
//  * Of the first segment of a row (what the workgroup's registers hold) each
//    thread has its largest value. The top-th largest of these, found by one
//    wave bit by bit while the others add up exponentials, is a lower bound
//    for the row's top-th largest value, and few values reach it.
//  * Those go to a list in LDS, later segments' too. A list that fills up
//    (more alternatives than a segment gives, many equal values) is cut to its
//    best `top` and the bound with it; a segment that does not fit in one go
//    is taken again, a value a thread at a time.
//  * Entries are compared as 64-bit numbers, the value's order above the
//    index's complement: all different, so that the order in which they
//    reached the list does not matter. An entry's place among the results is
//    how many are larger.
#include "sam_rows.h"
#include "sam_tokens.h"

namespace sam {

namespace {

using namespace rows;
typedef unsigned long long u64;

constexpr int kList = 1536;             // candidates of a workgroup
constexpr float kLn2 = 0.693147180559945f;

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

__device__ __forceinline__ u64 entry_of(float v, int index) { return (u64)order_of(v) << 32 | (unsigned)~index; }

// The largest of three, of numbers where there are any (the compiler's own
// maximum would first quieten each operand).
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
    return r;
}

template <int E>
__device__ __forceinline__ float max_of(const float (&v)[E], float m)
{
#pragma unroll
    for (int i = 0; i < E; i += 2) m = max3(m, v[i], v[i + 1]);
    return m;
}

// Sums over some values relative to their largest, m: s of 2^d and h of d
// 2^d, d = (z - m) log2(e) / T.
struct Sums {
    float m, s, h;
};

// The same relative to M >= m. Where nothing was counted m is -inf.
__device__ __forceinline__ void to_largest(Sums& x, float M, float scale)
{
    const float d = (x.m - M) * scale, f = pow2(d);
    const bool none = x.s == 0.0f;
    x.h = none ? 0.0f : f * (x.h + fmaxf(d, -1000.0f) * x.s);
    x.s = none ? 0.0f : f * x.s;
    x.m = M;
}

__device__ __forceinline__ Sums wave_total(Sums x, float scale)
{
    to_largest(x, wave_max(x.m), scale);
    return {x.m, wave_sum(x.s), wave_sum(x.h)};
}

// log p of a value of a row with norm (m, L); with m = -inf the pivot is 0.
__device__ __forceinline__ float log_p(float v, float m, float L, const TokenArgs& a)
{
    if (L == -INFINITY) return L;
    if (v == -INFINITY) return v - L;
    const float d = v - (m == -INFINITY ? 0.0f : m);
    return d * a.inv_hi + d * a.inv_lo - L;
}

// What a row's results are made of, by one thread.
__device__ __forceinline__ void write_row(const TokenArgs& a, long long row, const Sums& x, float L, float z_token)
{
    const bool has = (unsigned)a.token[row] < (unsigned)a.V;
    a.logprob[row] = has ? log_p(z_token, x.m, L, a) : 0.0f;
    a.entropy[row] = L == -INFINITY ? 0.0f : fmaxf(L - kLn2 * (x.h / x.s), L != L ? L : 0.0f);
    a.norm[2 * row] = x.m;
    a.norm[2 * row + 1] = L;
}

// The workgroup's list in LDS cut to its `top` best: the bits of the top-th
// largest entry are found one by one, until exactly `top` are as large.
// Returns a bound that the kept entries reach. n > top entries; every thread
// calls it, and the list's last use lies behind a barrier.
template <int NT, int CAP>
__device__ u64 cut_list(u64* list, int* count, int n, int top)
{
    __shared__ int more[NT / 64];
    constexpr int EACH = (CAP + NT - 1) / NT;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    u64 own[EACH];
#pragma unroll
    for (int i = 0; i < EACH; ++i) own[i] = (int)threadIdx.x + i * NT < n ? list[threadIdx.x + i * NT] : 0;
    u64 bound = 0;
    for (int bit = 63; bit >= 0; --bit) {
        const u64 t = bound | 1ull << bit;
        int c = 0;
#pragma unroll
        for (int i = 0; i < EACH; ++i) c += __popcll(__ballot(own[i] >= t));
        if (lane == 0) more[wave] = c;
        __syncthreads();
        int total = 0;
#pragma unroll
        for (int w = 0; w < NT / 64; ++w) total += more[w];
        if (total >= top) bound = t;
        __syncthreads();
        if (total == top) break;
    }
    if (threadIdx.x == 0) *count = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < EACH; ++i)
        if (own[i] && own[i] >= bound) list[atomicAdd(count, 1)] = own[i];
    __syncthreads();
    return bound;
}

// How many of a list's n entries are larger than e.
__device__ __forceinline__ int larger(const u64* list, int n, u64 e)
{
    int r = 0;
    for (int j = 0; j < n; ++j) r += list[j] > e;
    return r;
}

__device__ __forceinline__ void write_entry(const TokenArgs& a, long long row, int place, u64 e, float m, float L)
{
    a.top_logprob[row * a.top + place] = log_p(value_of((unsigned)(e >> 32)), m, L, a);
    a.top_index[row * a.top + place] = (int)~(unsigned)e;
}

// Entries of -inf, where there are fewer than `top` others (n, all of them in
// the list): the first ones of the row, which lie among its first `top`. The
// first wave calls it.
template <int DT>
__device__ __forceinline__ void write_masked(const TokenArgs& a, long long row, int n, float m, float L)
{
    const typename Ty<DT>::T* z = static_cast<const typename Ty<DT>::T*>(a.z) + row * a.ldz;
    for (int j0 = 0; j0 < a.top && n < a.top; j0 += 64) {
        const int j = j0 + (int)(threadIdx.x & 63);
        const bool masked = j < a.top && (float)z[j] == -INFINITY;
        const u64 who = __ballot(masked);
        const int place = n + __popcll(who & ((1ull << (threadIdx.x & 63)) - 1));
        if (masked && place < a.top) write_entry(a, row, place, entry_of(-INFINITY, j), m, L);
        n += __popcll(who);
    }
}

// A row, or a part of one (a.parts > 1), on NT threads that hold P pieces each.
template <int DT, int NT, int P, bool TOP>
__global__ void __launch_bounds__(NT) tokens_kernel(TokenArgs a)
{
    typedef Piece<DT> Pc;
    typedef typename Pc::T T;
    constexpr int E = Pc::E, NW = NT / 64;
    __shared__ u64 list[TOP ? kList : 1];
    __shared__ unsigned short best[TOP ? NT : 1];
    __shared__ int count;
    __shared__ float bound_s;
    __shared__ Sums wave_sums[NW];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const long long row = blockIdx.x / (unsigned)a.parts;
    const int part = blockIdx.x - (unsigned)row * a.parts;
    const T* z = static_cast<const T*>(a.z) + row * a.ldz;
    const Span sp = span_of<DT>(z, a.V);
    const u4* zb = reinterpret_cast<const u4*>(z + sp.head);
    const int each = a.parts == 1 ? sp.pieces : (sp.pieces / a.parts + 64) & ~63;
    const int p0 = min(part * each, sp.pieces), p1 = min(p0 + each, sp.pieces);

    // The first part takes the values outside the pieces, one a thread, and
    // the row's token.
    int edge_at = -1;
    if (part == 0) {
        if (tid < sp.head) edge_at = tid;
        if (tid >= 32 && tid - 32 < a.V - sp.tail0) edge_at = sp.tail0 + tid - 32;
    }
    const float edge = edge_at >= 0 ? (float)z[edge_at] : -INFINITY;
    float z_token = 0.0f;
    if (a.parts == 1 && tid == 0) {
        const int t = a.token[row];
        z_token = (float)z[(unsigned)t < (unsigned)a.V ? t : 0];
    }
    Sums x = {edge, edge == -INFINITY ? 0.0f : 1.0f + (edge - edge), 0.0f};   // NaN for an Inf or NaN

    int n = 0;             // candidates
    u64 least = 0;         // entries under it are out
    float bound = 0.0f;    // ... and values
    if (TOP && tid == 0) count = 0;
    auto push = [&](float v, int index) {
        const u64 e = entry_of(v, index);
        if (e >= least) {
            const int at = atomicAdd(&count, 1);
            if (at < kList) list[at] = e;
        }
    };

    for (int seg = p0; seg < p1 || seg == p0; seg += NT * P) {
        u4 r[P];
        const __amdgpu_buffer_rsrc_t rs = dma::make_rsrc(zb + seg, 16ll * (p1 - seg));
#pragma unroll
        for (int q = 0; q < P; ++q) r[q] = __builtin_amdgcn_raw_buffer_load_b128(rs, tid * 16, q * NT * 16, kOnce);
        if (seg + NT * P > p1) {   // the part's end: nothing there
#pragma unroll
            for (int q = 0; q < P; ++q)
                if (seg + q * NT + tid >= p1) r[q] = Pc::masked();
        }
        float pm[P], tm = -INFINITY;
#pragma unroll
        for (int q = 0; q < P; ++q) {
            float v[E];
            Pc::get(r[q], v);
            pm[q] = max_of(v, -INFINITY);
            tm = fmaxf(tm, pm[q]);
        }
        const bool select = TOP && n < a.top;
        if (select) {
            best[tid] = (unsigned short)(order_of(fmaxf(tm, seg == p0 ? edge : -INFINITY)) >> 16);
            __syncthreads();
            if (wave == 0) {
                unsigned k[NW], t = 0;
#pragma unroll
                for (int i = 0; i < NW; ++i) k[i] = best[lane + 64 * i];
#pragma unroll
                for (int bit = 15; bit >= 0; --bit) {
                    int c = 0;
#pragma unroll
                    for (int i = 0; i < NW; ++i) c += __popcll(__ballot(k[i] >= (t | 1u << bit)));
                    if (c >= a.top) t |= 1u << bit;
                }
                // Values of -inf are no candidates.
                if (lane == 0) bound_s = t <= 0x7F ? -3.402823466e38f : value_of(t << 16);
            }
        }

        // The segment's sums, relative to the thread's largest value so far.
        if (tm > x.m || x.s == 0.0f) {
            const float M = fmaxf(tm, x.m);
            to_largest(x, M, a.scale);
        }
        const float pivot = x.m == -INFINITY ? 0.0f : x.m, c = pivot * a.scale;
        float s = 0.0f, h = 0.0f;
        if (!__any(!(fabsf(c) <= 16384.0f))) {
            // d = z scale - c in one operation. c is rounded: all exponents
            // are off by the same, which is taken out of the sums.
#pragma unroll
            for (int q = 0; q < P; ++q) {
                float v[E];
                Pc::get(r[q], v);
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    const float d = __fmaf_rn(v[i], a.scale, -c), e = pow2(d);
                    s += e;
                    h = __fmaf_rn(e, fmaxf(d, -1000.0f), h);
                }
            }
            const float off = __fmaf_rn(pivot, a.scale, -c), g = pow2(-off);
            h = g * (h - off * s);
            s *= g;
        } else {
#pragma unroll
            for (int q = 0; q < P; ++q) {
                float v[E];
                Pc::get(r[q], v);
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    const float d = (v[i] - pivot) * a.scale, e = pow2(d);
                    s += e;
                    h = __fmaf_rn(e, fmaxf(d, -1000.0f), h);
                }
            }
        }
        x.s += s;
        x.h += h;

        if constexpr (TOP) {
            if (select) {
                __syncthreads();
                bound = fmaxf(bound_s, n ? bound : bound_s);
            }
            const bool odd = x.s != x.s;   // NaN among the values: pieces' largest do not show it
            if (seg == p0 && edge_at >= 0 && edge != -INFINITY && !(edge < bound)) push(edge, edge_at);
#pragma unroll
            for (int q = 0; q < P; ++q) {
                if (pm[q] < bound && !odd) continue;
                float v[E];
                Pc::get(r[q], v);
#pragma unroll
                for (int i = 0; i < E; ++i)
                    if (!(v[i] < bound)) push(v[i], sp.head + (seg + q * NT + tid) * E + i);
            }
            __syncthreads();
            int now = count;
            __syncthreads();
            if (now > kList) {
                // Too many at once: the segment again, a value a thread at a
                // time, and the list cut whenever it could not take the next.
                if (tid == 0) count = n;
                __syncthreads();
                if (seg == p0 && edge_at >= 0 && edge != -INFINITY) push(edge, edge_at);
                for (int i = 0; i < P * E; ++i) {
                    const int piece = seg + i / E * NT + tid;
                    if (piece < p1) {
                        const int index = sp.head + piece * E + i % E;
                        const float v = (float)z[index];
                        if (v != -INFINITY) push(v, index);
                    }
                    __syncthreads();
                    now = count;
                    __syncthreads();
                    if (now + NT > kList) {
                        least = cut_list<NT, kList>(list, &count, now, a.top);
                        now = a.top;
                    }
                }
            }
            n = now;
            if (n > kList / 2) {
                least = cut_list<NT, kList>(list, &count, n, a.top);
                n = a.top;
            }
            if (least) bound = fmaxf(bound, value_of((unsigned)(least >> 32)));
        }
    }

    x = wave_total(x, a.scale);
    if (NW > 1) {
        if (lane == 0) wave_sums[wave] = x;
        __syncthreads();
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < NW; ++w) M = fmaxf(M, wave_sums[w].m);
        Sums all = {M, 0.0f, 0.0f};
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            Sums y = wave_sums[w];
            to_largest(y, M, a.scale);
            all.s += y.s;
            all.h += y.h;
        }
        x = all;
    }
    if (TOP && n > kList / 4) {
        cut_list<NT, kList>(list, &count, n, a.top);
        n = a.top;
    }
    if (a.parts > 1) {
        const long long at = row * a.parts + part;
        if (tid == 0) a.part[at] = make_float4(x.m, x.s, x.h, __int_as_float(min(n, a.top)));
        if constexpr (TOP) {
            for (int i = tid; i < n; i += NT) {
                const int place = larger(list, n, list[i]);
                if (place < a.top) a.list[at * a.top + place] = list[i];
            }
        }
        return;
    }
    const float L = logf(x.s);
    if (tid == 0) write_row(a, row, x, L, z_token);
    if constexpr (TOP) {
        for (int i = tid; i < n; i += NT) {
            const int place = larger(list, n, list[i]);
            if (place < a.top) write_entry(a, row, place, list[i], x.m, L);
        }
        if (n < a.top && wave == 0) write_masked<DT>(a, row, n, x.m, L);
    }
}

// A row from its parts: sums joined, and the candidates that can be among the
// best: with full lists (top entries, sorted), the least of the entries at
// place ceil(top / lists) - 1 of each is reached by at least `top` of them.
template <int DT, bool TOP>
__global__ void __launch_bounds__(256) tokens_join_kernel(TokenArgs a)
{
    typedef typename Ty<DT>::T T;
    constexpr int NT = 256, CAP = TOP ? kMaxParts * kMaxAlternatives : 1;
    __shared__ u64 list[CAP];
    __shared__ int count, held[kMaxParts];
    const int tid = threadIdx.x, lane = tid & 63;
    const long long row = blockIdx.x;
    const int t = a.token[row];
    const float z_token = (float)(static_cast<const T*>(a.z) + row * a.ldz)[(unsigned)t < (unsigned)a.V ? t : 0];
    const float4 mine = lane < a.parts ? a.part[row * a.parts + lane] : make_float4(-INFINITY, 0.0f, 0.0f, 0.0f);
    const Sums x = wave_total({mine.x, mine.y, mine.z}, a.scale);   // every wave the same
    const float L = logf(x.s);
    if (tid == 0) write_row(a, row, x, L, z_token);
    if constexpr (TOP) {
        const int have = __float_as_int(mine.w);
        const u64* from = a.list + row * a.parts * a.top;
        const int full = __popcll(__ballot(lane < a.parts && have == a.top));
        u64 least = 0;
        if (full) {
            const int at = (a.top + full - 1) / full - 1;
            u64 e = lane < a.parts && have == a.top ? from[lane * a.top + at] : ~0ull;
#pragma unroll
            for (int d = 32; d; d >>= 1) {
                const u64 o = __shfl_xor(e, d);
                e = o < e ? o : e;
            }
            least = e;
        }
        if (tid == 0) count = 0;
        if (tid < 64) held[lane] = have;
        __syncthreads();
        for (int i = tid; i < a.parts * a.top; i += NT) {
            const int s = i / a.top, k = i - s * a.top;
            const u64 e = k < held[s] ? from[i] : 0;
            if (e && e >= least) list[atomicAdd(&count, 1)] = e;
        }
        __syncthreads();
        int n = count;
        __syncthreads();
        if (n > kList / 4) {
            cut_list<NT, CAP>(list, &count, n, a.top);
            n = min(n, a.top);
        }
        for (int i = tid; i < n; i += NT) {
            const int place = larger(list, n, list[i]);
            if (place < a.top) write_entry(a, row, place, list[i], x.m, L);
        }
        if (n < a.top && tid < 64) write_masked<DT>(a, row, n, x.m, L);
    }
}

// A strip of a row on a workgroup. Pieces are whole in the gradient's memory;
// where the logits lie otherwise (`shift`) they are loaded from whole words.
constexpr int kStripThreads = 256, kStripEach = 4;

template <int DT>
__global__ void __launch_bounds__(kStripThreads) tokens_grad_kernel(TokenGradArgs a, int strips)
{
    typedef Piece<DT> Pc;
    typedef typename Pc::T T;
    constexpr int E = Pc::E;
    const int tid = threadIdx.x;
    const long long row = blockIdx.x / (unsigned)strips;
    const int strip = blockIdx.x - (unsigned)row * strips;
    const T* z = static_cast<const T*>(a.z) + row * a.ldz;
    T* g = static_cast<T*>(a.grad) + row * a.ldg;
    const Span sp = span_of<DT>(g, a.V);
    const int t = a.token[row];
    const bool has = (unsigned)t < (unsigned)a.V;
    const float u = a.u && has ? a.u[row] : 0.0f, v = a.v ? a.v[row] : 0.0f;
    const float m = a.norm[2 * row], L = a.norm[2 * row + 1], H = v != 0.0f ? a.entropy[row] : 0.0f;
    // Rows without a gradient are not looked at.
    const bool off = (u == 0.0f && v == 0.0f) || L == -INFINITY;
    const float pivot = m == -INFINITY ? 0.0f : m;
    // dz = p (c0 + c1 log2 p) with both over T.
    const float l2 = L * 1.44269504088896f, c0 = -(u + v * H) * a.inv, c1 = -v * kLn2 * a.inv;
    auto one = [&](float x) {
        const float lp = (x - pivot) * a.scale - l2, p = pow2(lp);
        return p * (c0 + c1 * fmaxf(lp, -1000.0f));
    };
    u4 r[kStripEach];
    const int first = strip * kStripThreads * kStripEach + tid;
    const unsigned long long at = reinterpret_cast<unsigned long long>(z + sp.head);
    const bool same = (at & 15) == 0;
#pragma unroll
    for (int q = 0; q < kStripEach; ++q) {
        const int piece = first + q * kStripThreads;
        if (off || piece >= sp.pieces) continue;
        if (same) {
            r[q] = __builtin_nontemporal_load(reinterpret_cast<const u4*>(at) + piece);
        } else {
            typedef u4 u4w __attribute__((aligned(4)));
            const unsigned* w = reinterpret_cast<const unsigned*>((at & ~3ull) + 16ull * piece);
            r[q] = *reinterpret_cast<const u4w*>(w);
            if (DT != DT_F32 && (at & 2)) {
                const unsigned next = w[4];
                r[q] = u4{__builtin_amdgcn_alignbit(r[q][1], r[q][0], 16), __builtin_amdgcn_alignbit(r[q][2], r[q][1], 16),
                          __builtin_amdgcn_alignbit(r[q][3], r[q][2], 16), __builtin_amdgcn_alignbit(next, r[q][3], 16)};
            }
        }
    }
    // In the logits' place a piece is read by the thread that writes it; with
    // a shift the two share no memory.
#pragma unroll
    for (int q = 0; q < kStripEach; ++q) {
        const int piece = first + q * kStripThreads;
        if (piece >= sp.pieces) continue;
        float x[E];
        if (off) {
#pragma unroll
            for (int i = 0; i < E; ++i) x[i] = 0.0f;
        } else {
            Pc::get(r[q], x);
#pragma unroll
            for (int i = 0; i < E; ++i) x[i] = one(x[i]);
            const int k = t - (sp.head + piece * E);
            if (u != 0.0f && (unsigned)k < (unsigned)E) {
#pragma unroll
                for (int i = 0; i < E; ++i) x[i] += i == k ? u * a.inv : 0.0f;
            }
        }
        __builtin_nontemporal_store(Pc::put(x), reinterpret_cast<u4*>(g + sp.head) + piece);
    }
    if (strip == 0) {
        int j = -1;
        if (tid < sp.head) j = tid;
        if (tid >= 32 && tid - 32 < a.V - sp.tail0) j = sp.tail0 + tid - 32;
        if (j >= 0) g[j] = (T)(off ? 0.0f : one((float)z[j]) + (j == t ? u * a.inv : 0.0f));
    }
}

struct Form {
    int nt, p;
};

template <int DT, bool TOP>
hipError_t run(const TokenArgs& a, hipStream_t s)
{
    const unsigned grid = (unsigned)(a.rows * a.parts);
    const long long bytes = (long long)a.V * (DT == DT_F32 ? 4 : 2) / a.parts;
    if (!TOP && bytes <= 4096)
        hipLaunchKernelGGL((tokens_kernel<DT, 64, 4, TOP>), dim3(grid), dim3(64), 0, s, a);
    else if (bytes <= 32768)
        hipLaunchKernelGGL((tokens_kernel<DT, 256, 8, TOP>), dim3(grid), dim3(256), 0, s, a);
    else
        hipLaunchKernelGGL((tokens_kernel<DT, 512, 8, TOP>), dim3(grid), dim3(512), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.parts == 1) return e;
    hipLaunchKernelGGL((tokens_join_kernel<DT, TOP>), dim3((unsigned)a.rows), dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace

// Rows for fewer than two workgroups a CU are cut, into parts of 16 KB at least.
int tokens_parts(int dtype, long long rows, long long V)
{
    const long long bytes = V * (dtype == DT_F32 ? 4 : 2);
    long long p = 512 / rows;
    const long long most = bytes / 16384;
    p = p > most ? most : p;
    p = p > kMaxParts ? kMaxParts : p;
    return p < 2 ? 1 : (int)p;
}

hipError_t launch_tokens(int dtype, const TokenArgs& a, hipStream_t s)
{
    typedef hipError_t (*Fn)(const TokenArgs&, hipStream_t);
    static const Fn fn[3][2] = {{run<DT_F32, false>, run<DT_F32, true>}, {run<DT_BF16, false>, run<DT_BF16, true>},
                                {run<DT_F16, false>, run<DT_F16, true>}};
    return fn[dtype][a.top > 0](a, s);
}

hipError_t launch_tokens_grad(int dtype, const TokenGradArgs& a, hipStream_t s)
{
    const int each = kStripThreads * kStripEach * (dtype == DT_F32 ? 4 : 8);
    const int strips = (a.V + each - 1) / each;
    typedef void (*Fn)(TokenGradArgs, int);
    static const Fn fn[3] = {tokens_grad_kernel<DT_F32>, tokens_grad_kernel<DT_BF16>, tokens_grad_kernel<DT_F16>};
    hipLaunchKernelGGL(fn[dtype], dim3((unsigned)(a.rows * strips)), dim3(kStripThreads), 0, s, a, strips);
    return hipGetLastError();
}

}  // namespace sam
