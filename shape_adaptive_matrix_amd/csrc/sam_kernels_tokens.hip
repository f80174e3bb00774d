// Kernels of the token log probabilities (formulas in sam_tokens.h).
//
// Bound by memory: a row's logits are read once for its results and once more
// for its gradient. One pass holds a thread's largest value, its sum of
// exponentials and the sum of these times their exponents (for the entropy),
// and finds the most likely entries on the way:
//
//  * Every thread keeps, in 16 bits each, the largest value of its 16-byte
//    pieces (of rows too long for that, of the four pieces of a turn, or of
//    those of several turns: at most 32 numbers). Behind the row the
//    top-th largest of the threads' own largest values, found bit by bit, is a
//    lower bound of the row's top-th largest value that few pieces reach.
//  * Those pieces are read again (of 32768 values and 64 alternatives about 75
//    of 4096) and their values over the bound compared as 64-bit numbers, the
//    value's order above the index's complement: all different, so that their
//    order in the list does not matter. An entry's place among the results is
//    how many are larger.
//  * Rows with more such pieces or values than fit (equal values) are taken
//    again from the front, a piece a thread at a time, through a list that is
//    cut to its best whenever it could not take the next.
#include "sam_rows.h"
#include "sam_tokens.h"

namespace sam {

namespace {

using namespace rows;
typedef unsigned long long u64;

constexpr int kEntries = 512;           // entries whose places are found by comparing all with all
constexpr float kLowest = -3.402823466e38f;
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

// The register as it is, not what an earlier use made of it: without it the
// compiler keeps 16-bit rows as floats from one use to the next, twice the
// registers.
__device__ __forceinline__ void as_read(u4& x) { asm volatile("" : "+v"(x)); }

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

// Sums of several threads. The largest value's own 1 is left out of r, so that
// beside it nothing of the others is lost where they come to little (p near 1);
// with no value r is -1. h as in Sums.
struct Rest {
    float m, r, h;
};

// What y adds to a sum relative to M >= y.m: all of it, or (own) what is left
// beside the 1 of M itself.
__device__ __forceinline__ void relative_to(Rest& y, float M, bool own, float scale)
{
    if (own) return;
    Sums x = {y.m, 1.0f + y.r, y.h};
    to_largest(x, M, scale);
    y.r = x.s;
    y.h = x.h;
}

// The first of the lanes whose value is the largest, M.
__device__ __forceinline__ int lane_of(float v, float M)
{
    const u64 who = __ballot(v == M);
    return who ? __builtin_ctzll(who) : 0;
}

__device__ __forceinline__ Rest wave_total(Rest y, float scale)
{
    const float M = wave_max(y.m);
    relative_to(y, M, (int)(threadIdx.x & 63) == lane_of(y.m, M), scale);
    return {M, wave_sum(y.r), wave_sum(y.h)};
}

// log(1 + r), also where 1 + r is rounded: what that takes from r it takes from
// the logarithm too, in the same proportion (W. Kahan's way).
__device__ __forceinline__ float log_of_sum(float r)
{
    const float w = 1.0f + r;
    return w == 1.0f ? r : logf(w) * (r / (w - 1.0f));
}

// Below this rest the thread that has the largest value is summed once more
// without it, by its wave: its own sum, which holds that 1, is off by some
// 2^-24 (of 256 values some 2^-22), and with it log p, the entropy and 1 - p of a
// row whose p is near 1. One more trip to memory for such rows: 4096 x 32768
// bf16, all of them so, 52 us instead of 49; 2048 x 131072 FP32 160, 155.
constexpr float kSmallRest = 0.25f;

// log p of a value of a row with norm (m, L); with m = -inf the pivot is 0.
__device__ __forceinline__ float log_p(float v, float m, float L, const TokenArgs& a)
{
    if (L == -INFINITY) return L;
    if (v == -INFINITY) return v - L;
    const float pivot = m == -INFINITY ? 0.0f : m, d = v - pivot;
    if (d == -INFINITY) return 2.0f * ((0.5f * v - 0.5f * pivot) * a.inv_hi) - L;   // over FP32's range before the division
    return d * a.inv_hi + d * a.inv_lo - L;
}

// What a row's results are made of, by one thread.
__device__ __forceinline__ void write_row(const TokenArgs& a, long long row, const Rest& x, float L, float z_token)
{
    const bool has = (unsigned)a.token[row] < (unsigned)a.V;
    a.logprob[row] = has ? log_p(z_token, x.m, L, a) : 0.0f;
    a.entropy[row] = L == -INFINITY ? 0.0f : fmaxf(L - kLn2 * (x.h / (1.0f + x.r)), L != L ? L : 0.0f);
    a.norm[2 * row] = x.m;
    a.norm[2 * row + 1] = L;
}

// An LDS barrier that leaves global loads under way.
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

__device__ __forceinline__ int lanes_below(u64 who)
{
    return __builtin_amdgcn_mbcnt_hi((unsigned)(who >> 32), __builtin_amdgcn_mbcnt_lo((unsigned)who, 0));
}

// The top-th largest of the numbers that the workgroup's threads hold, G each
// (zero: none): bit by bit, until exactly `top` are as large; zero with fewer.
// `count`: LDS for a number a wave.
template <int NT, int G>
__device__ __forceinline__ u64 bound_together(const u64 (&own)[G], int top, int* count)
{
    u64 bound = 0;
    for (int bit = 63; bit >= 0; --bit) {
        const u64 t = bound | 1ull << bit;
        int c = 0;
#pragma unroll
        for (int i = 0; i < G; ++i) c += __popcll(__ballot(own[i] >= t));
        lds_barrier();
        if ((threadIdx.x & 63) == 0) count[threadIdx.x >> 6] = c;
        lds_barrier();
        c = 0;
#pragma unroll
        for (int w = 0; w < NT / 64; ++w) c += count[w];
        if (c >= top) bound = t;
        if (c == top) break;
    }
    return bound;
}

// Calls f(entry, its place) for the list's n entries, by the workgroup: a
// place is how many are larger. Lists of up to 64 (128) have four (two) lanes
// to an entry. Zeros follow the last entry up to a multiple of eight.
template <int NT, class F>
__device__ __forceinline__ void for_places(const u64* list, int n, F f)
{
    const int split = n <= NT / 4 ? 2 : (n <= NT / 2 ? 1 : 0);
    const int sub = threadIdx.x & ((1 << split) - 1);
    for (int i = threadIdx.x >> split; i < n; i += NT >> split) {
        const u64 e = list[i];
        int r = 0;
        for (int j = 8 * sub; j < n; j += 8 << split) {
            u64 o[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) o[k] = list[j + k];
#pragma unroll
            for (int k = 0; k < 8; ++k) r += o[k] > e;
        }
        if (split) r += __builtin_amdgcn_update_dpp(0, r, 0xB1, 0xF, 0xF, true);       // lanes 1 0 3 2
        if (split == 2) r += __builtin_amdgcn_update_dpp(0, r, 0x4E, 0xF, 0xF, true);  // lanes 2 3 0 1
        if (sub == 0) f(e, r);
    }
}

// Sum over the lanes up to this one.
__device__ __forceinline__ int sum_up_to(int v)
{
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, true);   // from 1, 2, 4, 8 lanes below
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);  // lane 15 of the row below
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);  // lane 31
    return v;
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

// A lower bound of the top-th largest of 64 G values, by the upper 16 bits of
// numbers that order them (G a lane; zero: none), found by one wave.
template <int G>
__device__ __forceinline__ float bound_of(const unsigned (&k)[G], int top)
{
    unsigned hi = k[0], lo = k[0];
#pragma unroll
    for (int i = 1; i < G; ++i) {
        hi = max(hi, k[i]);
        lo = min(lo, k[i]);
    }
    // The bits that all have in common need no search.
    hi = (unsigned)wave_max((float)hi);
    lo = (unsigned)-wave_max(-(float)lo);
    unsigned bit = hi == lo ? 0 : 1u << (31 - __builtin_clz(hi ^ lo));
    unsigned t = bit ? hi & ~(2 * bit - 1) : hi;
    for (; bit; bit >>= 1) {
        int c = 0;
#pragma unroll
        for (int i = 0; i < G; ++i) c += __popcll(__ballot(k[i] >= (t | bit)));
        t = c >= top ? t | bit : t;
    }
    return t <= 0x7F ? kLowest : value_of(t << 16);   // values of -inf are no candidates
}

// A row, or a part of one (a.parts > 1), on NT threads that hold P pieces
// each of it, and the next P on the way.
template <int DT, int NT, int P, bool TOP>
__global__ void __launch_bounds__(NT) __attribute__((amdgpu_waves_per_eu(!TOP ? 8 : (NT == 64 ? 4 : 6)))) tokens_kernel(TokenArgs a)
{
    typedef Piece<DT> Pc;
    typedef typename Pc::T T;
    constexpr int E = Pc::E, NW = NT / 64, FINE = 32 / P;   // segments whose pieces each have a bit of 32
    // top <= NT: that many threads' largest values bound it.
    static_assert(P == 4 && FINE * P == 32, "a thread's pieces, or groups of segments, are 32 bits");
    // The pieces' largest values, [segment][thread][P], or those of `step`
    // segments, [.][thread];
    // entries; and in the place of both the list of the long way.
    constexpr int KEYS = 32 * NT / 4, LIST = NT * E + kEntries;
    constexpr int ROOM = KEYS + kEntries > LIST ? KEYS + kEntries : LIST;
    __shared__ __attribute__((aligned(16))) u64 room[TOP ? ROOM + 8 : 1];
    __shared__ unsigned short ids[TOP ? kEntries : 1], best[TOP ? NT : 1];
    __shared__ int counts[NW], pieces_found, entries;
    __shared__ Rest wave_sums[NW];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const long long row = blockIdx.x / (unsigned)a.parts;
    const int part = blockIdx.x - (unsigned)row * a.parts;
    const T* z = static_cast<const T*>(a.z) + row * a.ldz;
    const Span sp = span_of<DT>(z, a.V);
    const u4* zb = reinterpret_cast<const u4*>(z + sp.head);
    const int each = (sp.pieces + a.parts - 1) / a.parts;
    const int p0 = min(part * each, sp.pieces), p1 = min(p0 + each, sp.pieces);
    const int segments = (p1 - p0 + NT * P - 1) / (NT * P);
    const bool fine = segments <= FINE;
    const int step = fine ? 1 : (segments + 31) / 32;   // segments that share a bit

    u4 r[2][P];
    auto fetch = [&](u4 (&x)[P], int seg) {   // past the part's end: zeros, and no traffic
        const __amdgpu_buffer_rsrc_t rs = dma::make_rsrc(zb + seg, seg < p1 ? 16ll * (p1 - seg) : 0);
#pragma unroll
        for (int q = 0; q < P; ++q) x[q] = __builtin_amdgcn_raw_buffer_load_b128(rs, tid * 16, q * NT * 16, kOnce);
    };
    fetch(r[0], p0);

    // The first part takes the values outside the pieces, one a thread, and
    // the row's token.
    int edge_at = -1;
    if (part == 0) {
        if (tid < sp.head) edge_at = tid;
        if (tid >= 32 && tid - 32 < a.V - sp.tail0) edge_at = sp.tail0 + tid - 32;
    }
    const float edge = edge_at >= 0 ? (float)z[edge_at] : -INFINITY;
    float z_token = 0.0f;
    if (part == 0 && tid == 0) {
        const int t = a.token[row];
        z_token = (float)z[(unsigned)t < (unsigned)a.V ? t : 0];
    }
    Sums x = {edge, edge == -INFINITY ? 0.0f : 1.0f + (edge - edge), 0.0f};   // NaN for an Inf or NaN

    float so_far = -INFINITY;   // of the segments that share a bit
    bool plain = true;          // the wave's values so far are finite and near enough to zero
    if constexpr (TOP)
        for (int i = tid; i < kEntries + 8; i += NT) room[KEYS + i] = 0;
    auto segment = [&](u4 (&r)[P], u4 (&next)[P], int at) {
        const int seg = p0 + at * (NT * P);
        fetch(next, seg + NT * P);
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
        }
        tm = max3(max3(pm[0], pm[1], pm[2]), pm[3], tm);
#pragma unroll
        for (int q = 0; q < P; ++q) as_read(r[q]);

        // The segment's sums, relative to the thread's largest value so far.
        if (tm > x.m || x.s == 0.0f) to_largest(x, fmaxf(tm, x.m), a.scale);
        const float pivot = x.m == -INFINITY ? 0.0f : x.m, c = pivot * a.scale;
        float s = 0.0f, h = 0.0f;
        plain = plain && !__any(!(fabsf(c) <= 16384.0f));
        if (plain) {
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
                    h = __fmaf_rn(e, d, h);
                }
            }
            const float off = __fmaf_rn(pivot, a.scale, -c), g = pow2(-off);
            h = g * (h - off * s);
            s *= g;
            plain = !__any(h != h);
        }
        // Values of -inf (their 0 times -inf should be 0), and far from zero:
        // here, and for the rest of the row.
        if (!plain) {
            s = h = 0.0f;
#pragma unroll
            for (int q = 0; q < P; ++q) as_read(r[q]);
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
            // NaN among the values does not show in their largest: a NaN.
            const bool odd = x.s != x.s;
            unsigned k[P];
#pragma unroll
            for (int q = 0; q < P; ++q) k[q] = odd ? 0x7FC00000u : __float_as_uint(pm[q]);
            if (fine) {
                reinterpret_cast<uint2*>(room)[at * NT + tid] = make_uint2(__builtin_amdgcn_perm(k[1], k[0], 0x07060302u),
                                                                           __builtin_amdgcn_perm(k[3], k[2], 0x07060302u));
            } else {
                const int group = at / step;
                so_far = group * step == at ? tm : fmaxf(so_far, tm);
                reinterpret_cast<unsigned short*>(room)[group * NT + tid] = odd ? 0x7FC0 : (unsigned short)(__float_as_uint(so_far) >> 16);
            }
        }
    };
    int at = 0;
#pragma clang loop unroll(disable)
    for (; at + 2 <= segments; at += 2) {
        segment(r[0], r[1], at);
        segment(r[1], r[0], at + 1);
    }
    if (at < segments) segment(r[0], r[1], at);

    if constexpr (TOP) {
        best[tid] = x.s != x.s ? 0xFFFF : (unsigned short)(order_of(x.m) >> 16);
        if (tid == 0) pieces_found = entries = 0;
    }
    // The wave's sums, without the largest value.
    const float largest = wave_max(x.m);
    const int owner = lane_of(x.m, largest);
    to_largest(x, largest, a.scale);
    Rest rest = {largest, wave_sum(lane == owner ? x.s - 1.0f : x.s), wave_sum(x.h)};
    if (fabsf(rest.r) < kSmallRest) {
        float s = lane == owner ? 0.0f : x.s, h = lane == owner ? 0.0f : x.h;
        auto take = [&](float v) {
            const float d = (v - largest) * a.scale, e = v != largest ? pow2(d) : 0.0f;
            s += e;
            h = __fmaf_rn(e, fmaxf(d, -1000.0f), h);
        };
        const float its_edge = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(edge), owner));
        if (lane == 0) take(its_edge);
        for (int i = lane; i < segments * P; i += 64) {
            const int piece = p0 + i * NT + 64 * wave + owner;
            if (piece >= p1) continue;
            float v[E];
            Pc::get(zb[piece], v);
#pragma unroll
            for (int j = 0; j < E; ++j) take(v[j]);
        }
        rest.r = wave_sum(s);
        rest.h = wave_sum(h);
    }
    if (NW > 1 || TOP) {
        if (lane == 0) wave_sums[wave] = rest;
        lds_barrier();
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < NW; ++w) M = fmaxf(M, wave_sums[w].m);
        Rest all = {M, 0.0f, 0.0f};
        bool found = false;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            Rest y = wave_sums[w];
            const bool own = !found && y.m == M;
            found |= own;
            relative_to(y, M, own, a.scale);
            all.r += y.r;
            all.h += y.h;
        }
        rest = all;
    }
    const float L = log_of_sum(rest.r);
    int total = 0;
    if constexpr (TOP) {
        u64* list = room + KEYS;
        float bound;
        {
            unsigned k[NW];
#pragma unroll
            for (int i = 0; i < NW; ++i) k[i] = best[lane + 64 * i];
            bound = bound_of(k, a.top);   // every wave the same
        }
        // A place for each of `n` of every lane, counted in `count`.
        auto places = [&](int n, int* count) {
            const int up = sum_up_to(n);
            int to = 0;
            if (lane == 63 && up) to = atomicAdd(count, up);
            return __builtin_amdgcn_readlane(to, 63) + up - n;
        };
        auto taken = [&](float v) { return v != -INFINITY && !(v < bound); };
        // The values of a thread's pieces (d[q] at index[q]), and at the edge
        // of the row, that reach the bound.
        auto gather = [&](auto& d, auto& index, unsigned look, bool with_edge) {   // look: a bit for each piece
            constexpr int Q = sizeof(index) / sizeof(index[0]);
            const int edges = with_edge && edge_at >= 0 && taken(edge) ? 1 : 0;
            int n = edges;
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                if (!__any(look >> q & 1)) continue;
                float v[E];
                Pc::get(d[q], v);
#pragma unroll
                for (int j = 0; j < E; ++j) n += taken(v[j]);
            }
            int to = places(n, &entries);
            if (n == 0) return;
            if (edges && to < kEntries) list[to] = entry_of(edge, edge_at);
            to += edges;
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                if (!(look >> q & 1)) continue;
                float v[E];
                Pc::get(d[q], v);
#pragma unroll
                for (int j = 0; j < E; ++j) {
                    if (taken(v[j]) && to < kEntries) list[to] = entry_of(v[j], index[q] + j);
                    to += taken(v[j]);
                }
            }
        };
        // A bit for each of the thread's pieces (segments) that reach it.
        unsigned mine = 0;
        for (int s = 0; s * step < segments; ++s) {
            auto reaches = [&](unsigned upper) { return !(__uint_as_float(upper) < bound) ? 1u : 0u; };
            if (fine) {
                const uint2 k = reinterpret_cast<const uint2*>(room)[s * NT + tid];
                mine |= (reaches(k.x << 16) | reaches(k.x & 0xFFFF0000u) << 1 | reaches(k.y << 16) << 2 |
                         reaches(k.y & 0xFFFF0000u) << 3) << (4 * s);
            } else {
                mine |= reaches((unsigned)reinterpret_cast<const unsigned short*>(room)[s * NT + tid] << 16) << s;
            }
        }
        int found = 0;
        if (segments <= 1) {   // the pieces are still there
            int index[P];
#pragma unroll
            for (int q = 0; q < P; ++q) index[q] = sp.head + (p0 + q * NT + tid) * E;
            gather(r[0], index, mine, true);
            lds_barrier();
            total = entries;
        } else {
            int to = places(__popc(mine), &pieces_found);
            for (; mine; mine &= mine - 1, ++to)
                if (to < kEntries) ids[to] = (unsigned short)((__ffs(mine) - 1) * NT + tid);
            lds_barrier();
            found = pieces_found;
            if (found <= kEntries) {
                const int per = fine ? 1 : P * step, items = found * per;
                for (int i0 = 0; i0 < items || i0 == 0; i0 += NT) {
                    const int i = i0 + tid;
                    u4 d[1] = {Pc::masked()};
                    int index[1] = {0};
                    if (i < items) {
                        const int id = ids[i / per], bit = id / NT, rest = i % per;
                        const int at = fine ? bit / P : bit * step + rest / P, q = fine ? bit % P : rest % P;
                        const int piece = p0 + at * (NT * P) + q * NT + id % NT;
                        if (piece < p1) {
                            d[0] = zb[piece];
                            index[0] = sp.head + piece * E;
                        }
                    }
                    gather(d, index, 1, i0 == 0);
                }
                lds_barrier();
                total = entries;
            }
        }
        if (found > kEntries || total > kEntries) {
            list = room;
            u64 least = 0;
            lds_barrier();
            if (tid == 0) entries = 0;
            lds_barrier();
            auto push = [&](float v, int index) {
                const u64 e = entry_of(v, index);
                if (v != -INFINITY && e >= least) list[atomicAdd(&entries, 1)] = e;
            };
            if (edge_at >= 0) push(edge, edge_at);
            for (int p = p0; p < p1; p += NT) {
                if (p + tid < p1) {
                    float v[E];
                    Pc::get(zb[p + tid], v);
#pragma unroll
                    for (int j = 0; j < E; ++j) push(v[j], sp.head + (p + tid) * E + j);
                }
                lds_barrier();
                total = entries;
                lds_barrier();
                if (total <= kEntries - 2 * E) continue;   // room for a step's and the edges'
                constexpr int G = (LIST + NT - 1) / NT;
                u64 own[G];
#pragma unroll
                for (int i = 0; i < G; ++i) own[i] = tid + i * NT < total ? list[tid + i * NT] : 0;
                least = bound_together<NT>(own, a.top, counts);
                if (tid == 0) entries = 0;
                lds_barrier();
#pragma unroll
                for (int i = 0; i < G; ++i)
                    if (own[i] && own[i] >= least) list[atomicAdd(&entries, 1)] = own[i];
                lds_barrier();
                total = entries;
            }
            if (tid < (-total & 7)) list[total + tid] = 0;
            lds_barrier();
        }
        const long long out = row * a.parts + part;
        for_places<NT>(list, total, [&](u64 e, int place) {
            if (place >= a.top) return;
            if (a.parts > 1) a.list[out * a.top + place] = e;
            else write_entry(a, row, place, e, rest.m, L);
        });
        if (a.parts == 1 && total < a.top && wave == 0) write_masked<DT>(a, row, total, rest.m, L);
    }
    if (tid == 0) {
        if (a.parts == 1) {
            write_row(a, row, rest, L, z_token);
        } else {
            a.part[row * a.parts + part] = make_float4(rest.m, rest.r, rest.h, __int_as_float(min(total, a.top)));
            if (part == 0) a.z_token[row] = z_token;
        }
    }
}

// A row from its parts: sums joined, and the candidates that can be among the
// best: with full lists (top entries, sorted), the least of the entries at
// place ceil(top / lists) - 1 of each is reached by at least `top` of them.
template <int DT, bool TOP>
__global__ void __launch_bounds__(256) tokens_join_kernel(TokenArgs a)
{
    constexpr int CAP = TOP ? kMaxParts * kMaxAlternatives : 1;
    __shared__ __attribute__((aligned(16))) u64 list[CAP + 8];
    __shared__ int count, held[kMaxParts];
    constexpr int EARLY = 4;
    const int tid = threadIdx.x, lane = tid & 63;
    const long long row = blockIdx.x;
    const u64* from = a.list + row * a.parts * a.top;
    // Everything that most calls need is asked for at once; what a list holds
    // past its end is dropped later.
    const float4 mine = lane < a.parts ? a.part[row * a.parts + lane] : make_float4(-INFINITY, -1.0f, 0.0f, 0.0f);
    const float z_token = a.z_token[row];
    const int all = a.parts * a.top;
    u64 own[EARLY], low = 0;
    if constexpr (TOP) {
        low = from[min(lane, a.parts - 1) * a.top + (a.top + a.parts - 1) / a.parts - 1];
#pragma unroll
        for (int i = 0; i < EARLY; ++i) own[i] = from[min(tid + 256 * i, all - 1)];
    }
    const int have = __float_as_int(mine.w);
    const Rest x = wave_total({mine.x, mine.y, mine.z}, a.scale);   // every wave the same
    const float L = log_of_sum(x.r);
    if constexpr (TOP) {
        const bool is_full = lane < a.parts && have == a.top;
        const int full = __popcll(__ballot(is_full));
        u64 least = 0;
        if (full) {
            if (full < a.parts && is_full) low = from[lane * a.top + (a.top + full - 1) / full - 1];
            least = is_full ? low : ~0ull;
#pragma unroll
            for (int d = 32; d; d >>= 1) {
                const u64 o = __shfl_xor(least, d);
                least = o < least ? o : least;
            }
        }
        if (tid == 0) count = 0;
        if (tid < 64) held[lane] = have;
        for (int i = tid; i < min(all, kEntries) + 8; i += 256) list[i] = 0;
        lds_barrier();
        auto add = [&](u64 e, int i) {
            const int s = i / a.top;
            const bool in = i < all && i - s * a.top < held[min(s, a.parts - 1)] && e >= least;
            const u64 who = __ballot(in);
            int at = 0;
            if (lane == 0 && who) at = atomicAdd(&count, __popcll(who));
            at = __builtin_amdgcn_readfirstlane(at);
            if (in) list[at + lanes_below(who)] = e;
        };
#pragma unroll
        for (int i = 0; i < EARLY; ++i) add(own[i], tid + 256 * i);
        for (int i = 256 * EARLY; i < all; i += 256) add(i + tid < all ? from[i + tid] : 0, i + tid);
        lds_barrier();
        int n = count;
        if (n > kEntries) {   // the best lie in few parts
            __shared__ int counts[4];
            constexpr int G = (CAP + 255) / 256;
            u64 some[G];
#pragma unroll
            for (int i = 0; i < G; ++i) some[i] = tid + 256 * i < n ? list[tid + 256 * i] : 0;
            const u64 last = bound_together<256>(some, a.top, counts);
            if (tid == 0) count = 0;
            lds_barrier();
#pragma unroll
            for (int i = 0; i < G; ++i)
                if (some[i] && some[i] >= last) list[atomicAdd(&count, 1)] = some[i];
            lds_barrier();
            n = count;
            if (tid < (-n & 7)) list[n + tid] = 0;
            lds_barrier();
        }
        for_places<256>(list, n, [&](u64 e, int place) {
            if (place < a.top) write_entry(a, row, place, e, x.m, L);
        });
        if (n < a.top && tid < 64) write_masked<DT>(a, row, n, x.m, L);
    }
    if (tid == 0) write_row(a, row, x, L, z_token);
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
    // The token: u (1 - p) by expm1, which loses nothing where p is near 1.
    auto own = [&](float x) {
        const float lp = (x - pivot) * a.scale - l2, p = pow2(lp);
        return p * (c1 * fmaxf(lp, -1000.0f) - v * H * a.inv) - u * a.inv * expm1f(lp * kLn2);
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
                float y[E], w = 0.0f;
                Pc::get(r[q], y);
#pragma unroll
                for (int i = 0; i < E; ++i) w = i == k ? y[i] : w;
                w = own(w);
#pragma unroll
                for (int i = 0; i < E; ++i) x[i] = i == k ? w : x[i];
            }
        }
        __builtin_nontemporal_store(Pc::put(x), reinterpret_cast<u4*>(g + sp.head) + piece);
    }
    if (strip == 0) {
        int j = -1;
        if (tid < sp.head) j = tid;
        if (tid >= 32 && tid - 32 < a.V - sp.tail0) j = sp.tail0 + tid - 32;
        if (j >= 0) g[j] = (T)(off ? 0.0f : (u != 0.0f && j == t ? own((float)z[j]) : one((float)z[j])));
    }
}

template <int DT, bool TOP>
hipError_t run(const TokenArgs& a, hipStream_t s)
{
    const unsigned grid = (unsigned)(a.rows * a.parts);
    const long long bytes = (long long)a.V * (DT == DT_F32 ? 4 : 2);
    // Short rows: a wave each, which waits for no other (4096 x 2000 bf16, 5
    // alternatives: 14 us, with four waves 29; 4096 x 8192: 20 and 26), as long
    // as its 64 lanes' largest values make a close bound.
    const bool wave = a.top <= 24 && a.parts == 1 && (bytes <= 4096 || (bytes <= 16384 && a.rows >= 512));
    if (wave)
        hipLaunchKernelGGL((tokens_kernel<DT, 64, 4, TOP>), dim3(grid), dim3(64), 0, s, a);
    else
        hipLaunchKernelGGL((tokens_kernel<DT, 256, 4, TOP>), dim3(grid), dim3(256), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.parts == 1) return e;
    hipLaunchKernelGGL((tokens_join_kernel<DT, TOP>), dim3((unsigned)a.rows), dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace

// Rows for fewer than two workgroups a CU are cut, into parts of 16 KB at
// least, with alternatives 32 KB (16 x 131072 FP32, 20 of them: 13.3 us, with
// 16 KB 16 us, for twice the lists to join).
int tokens_parts(int dtype, long long rows, long long V, long long top)
{
    const long long bytes = V * (dtype == DT_F32 ? 4 : 2), most = bytes / (top ? 32768 : 16384);
    long long p = 512 / rows;
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
