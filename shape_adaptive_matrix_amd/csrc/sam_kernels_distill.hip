// Kernels of the distillation loss (formulas in sam_distill.h).
//
// Bound by memory: a row's logits are read once and its gradient written
// once. The loss kernel gives a row to one workgroup, which keeps it in
// registers between the softmax's sum and the gradient; of a row too long for
// registers and LDS the rest is read again.
#include "sam_distill.h"
#include "sam_dma.h"

namespace sam {

namespace {

typedef unsigned int u4 __attribute__((ext_vector_type(4)));

constexpr int kFewTop = 128;

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
__device__ __forceinline__ void as_read(u4& a, u4& b, u4& c, u4& d)
{
    asm volatile("" : "+v"(a), "+v"(b), "+v"(c), "+v"(d));
}

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

// A teacher's or a student's value as it is stored, and as a float: loads
// that are not waited for where they are issued.
__device__ __forceinline__ unsigned raw_at(const void* p, int dtype, long long i)
{
    if (dtype == DT_F32) return static_cast<const unsigned*>(p)[i];
    return static_cast<const unsigned short*>(p)[i];
}

__device__ __forceinline__ float value_of(unsigned raw, int dtype)
{
    if (dtype == DT_F32) return __uint_as_float(raw);
    if (dtype == DT_BF16) return __uint_as_float(raw << 16);
    return (float)__builtin_bit_cast(_Float16, (unsigned short)raw);
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

// How many of a row's entries have index i. Their list is -1 up to a multiple of four.
__device__ __forceinline__ int repeats(const int* idx, int top, int i)
{
    int n = 0;
    for (int k = 0; k < top; k += 4) {
        const int4 v = *reinterpret_cast<const int4*>(idx + k);
        n += (v.x == i) + (v.y == i) + (v.z == i) + (v.w == i);
    }
    return n;
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

// A row's part of the arguments. `read`: its logits are wanted; otherwise its
// pieces read zeros, which costs nothing.
template <int DT>
struct Row {
    typedef typename Ty<DT>::T T;
    long long at;
    const T* z;
    float w;
    Span sp;
    const u4* zb;
    long long bytes;
    __device__ __forceinline__ Row(const DistillArgs& a, long long row, bool grad, bool read)
        : at(row), z(static_cast<const T*>(a.z) + row * a.ldz), w(a.weight ? constant(a.weight, row) : 1.0f), sp(span_of<DT>(z, a.V)),
          zb(reinterpret_cast<const u4*>(z + sp.head)), bytes(read && !(grad && w == 0.0f) ? 16ll * sp.pieces : 0) {}
    // Values outside the pieces: at most E - 1 at either end, a thread each.
    __device__ __forceinline__ int edge_at(int V) const
    {
        const int tid = threadIdx.x;
        if (tid < sp.head) return tid;
        return tid >= 32 && tid - 32 < V - sp.tail0 ? sp.tail0 + tid - 32 : -1;
    }
};

// P pieces of a row stay in each thread's registers and L more in its own
// place in LDS; what is left of a longer row (REST) is read again for the
// gradient. With the gradient a workgroup takes row after row: as soon as a
// piece of one row's gradient is stored its registers take the next row's
// logits, so that loads and stores are under way together all the time, and
// the sums run on pieces as they arrive. For that no load may sit behind a
// condition (the compiler could not count how many follow it, and would wait
// for all): pieces past a row's end read zeros, entries past the last read
// the last, and what they hold is dropped when it is used.
// A row has one barrier, between its sums and what follows from them: the
// teacher's entries go 64 to a wave (more than the waves take at once have
// their logits read behind it, and a second barrier before the row's stores),
// and what is to be written behind the whole row (the loss, the entries' own
// gradients) goes out behind the next row's barrier.
// Measured, loss and gradient: 4096 x 32768 bf16 100 us (rows on
// workgroups of their own, everything between barriers: 123), 1024 x 131072
// FP32 219 us (274).
// Waves a SIMD that the registers have to leave room for: with the gradient
// as many as `run` puts on a CU.
constexpr int distill_waves(int nt, int p, bool grad) { return !grad ? 1 : (nt == 512 && p == 8 ? 6 : nt == 64 && p <= 8 ? 5 : 4); }

template <int DT, int NT, int P, int L, bool REST, bool GRAD, int TOP>
__global__ void __launch_bounds__(NT) __attribute__((amdgpu_waves_per_eu(distill_waves(NT, P, GRAD))))
distill_kernel(DistillArgs a)
{
    typedef Piece<DT> Pc;
    typedef typename Pc::T T;
    constexpr int E = Pc::E, NW = NT / 64;
    static_assert(P % 4 == 0 && L % 4 == 0, "pieces are summed four at a time");
    __shared__ __attribute__((aligned(16))) u4 hold[L > 0 ? L * NT : 1];
    __shared__ float val[2][TOP];        // by row parity: the teacher's value
    __shared__ __attribute__((aligned(16))) int idx[2][TOP];   // its index, -1: empty
    __shared__ float gval[2][TOP];       // an entry's own gradient
    __shared__ unsigned long long gset[2][TOP / 64];   // and whether it is written, a bit each
    __shared__ float4 part[2][NW];       // a wave's largest logit and sum, its entries' largest and sum
    __shared__ float lsum[2][NW];        // its part of the loss
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int chunks = (a.top + 63) / 64;

    // What is loaded ahead of a row's turn: its pieces, its edge value, the
    // wave's first entries and their logits (for which the entries themselves
    // come two rows ahead).
    u4 r[P];
    unsigned t, t_next, zr, edge;
    int ix, ix_next;
    auto entry_at = [&](const Row<DT>& c, int o) { return c.at * a.top + min(lane + 64 * o, a.top - 1); };
    auto entry_of = [&](const Row<DT>& c, int o) {
        const int i = a.index[entry_at(c, o)];
        return lane + 64 * o >= a.top || (unsigned)i >= (unsigned)a.V ? -1 : i;
    };
    auto fetch_entries = [&](const Row<DT>& c, long long then) {   // row c's turn is next, row `then`'s after that
        ix = ix_next;
        t = t_next;
        if (lane + 64 * wave >= a.top || (unsigned)ix >= (unsigned)a.V) ix = -1;
        zr = raw_at(c.z, DT, max(ix, 0));
        edge = raw_at(c.z, DT, max(c.edge_at(a.V), 0));
        const long long j = then * a.top + min(lane + 64 * wave, a.top - 1);
        ix_next = a.index[j];
        t_next = raw_at(a.t, a.t_dtype, j);
    };
    auto fetch = [&](const Row<DT>& c, int q) {
        r[q] = __builtin_amdgcn_raw_buffer_load_b128(dma::make_rsrc(c.zb, c.bytes), tid * 16, q * NT * 16, kOnce);
    };
    auto fetch_hold = [&](const Row<DT>& c, int o) {   // straight into LDS; no registers for it
        dma::lds_load16(dma::rsrc_words(c.zb, c.bytes), dma::lds_addr(hold + o * NT + wave * 64), (tid + (P + o) * NT) * 16);
    };
    auto fetch_rest = [&](const Row<DT>& c, u4 (&x)[4], int at) {
        const __amdgpu_buffer_rsrc_t rs = dma::make_rsrc(c.zb + at, c.bytes - 16ll * at);
#pragma unroll
        for (int b = 0; b < 4; ++b) x[b] = __builtin_amdgcn_raw_buffer_load_b128(rs, tid * 16, b * NT * 16, 0);
    };
    // -inf in pieces past the row's end, of four that start at piece `at`, NT
    // apart. A branch, not selects, for whole groups pass it by.
    auto trim = [&](const Row<DT>& c, u4& x0, u4& x1, u4& x2, u4& x3, int at) {
        if (at + 4 * NT > c.sp.pieces) {
            as_read(x0, x1, x2, x3);
            const int left = c.sp.pieces - at - tid;
            if (left <= 0) x0 = Pc::masked();
            if (left <= NT) x1 = Pc::masked();
            if (left <= 2 * NT) x2 = Pc::masked();
            if (left <= 3 * NT) x3 = Pc::masked();
        }
    };
    // What follows a row that all waves have stored: each wave's entries, the loss.
    auto finish_row = [&](long long row, int par) {
        if (GRAD)
            for (int j = lane + 64 * wave; j < a.top; j += NT)
                if (gset[par][j / 64] >> lane & 1) static_cast<T*>(a.grad)[row * a.ldg + idx[par][j]] = (T)gval[par][j];
        if (tid == 0) {
            float sum = 0.0f;
            for (int w = 0; w < min(chunks, NW); ++w) sum += lsum[par][w];
            if (a.loss) a.loss[row] = sum;
        }
    };

    long long row = blockIdx.x, before = -1;
    Row<DT> c(a, row, GRAD, true);
    ix_next = a.index[entry_at(c, wave)];
    t_next = raw_at(a.t, a.t_dtype, entry_at(c, wave));
#pragma unroll
    for (int o = 0; o < L; ++o) fetch_hold(c, o);
#pragma unroll
    for (int q = 0; q < P; ++q) fetch(c, q);
    fetch_entries(c, min(row + (GRAD ? gridDim.x : 0), a.rows - 1));
    for (int par = 0;; par ^= 1) {
        const bool last = !GRAD || row + gridDim.x >= a.rows;
        const Row<DT> n(a, last ? row : row + gridDim.x, GRAD, !last);
        const int edge_at = c.edge_at(a.V);
        const float edge_v = edge_at >= 0 ? value_of(edge, DT) : -INFINITY;

        const bool look = !GRAD || c.w != 0.0f;   // a row that is not trained on: its logits are not looked at
        float z_own = 0.0f;                       // of the wave's first entries
        bool twice = false;                       // the lane's index comes more than once
        if (look) {
            float best = -INFINITY, psum = 0.0f;
            if (wave < chunks) {
                auto take = [&](int o, int i, unsigned raw) {
                    const int j = lane + 64 * o;
                    const float v = i >= 0 ? value_of(raw, a.t_dtype) : -INFINITY;
                    best = fmaxf(best, v);
                    idx[par][j] = i;
                    val[par][j] = v;
                };
                take(wave, ix, t);
                for (int o = wave + NW; o < chunks; o += NW) take(o, entry_of(c, o), raw_at(a.t, a.t_dtype, entry_at(c, o)));
                best = wave_max(best);
                for (int j = lane + 64 * wave; j < a.top; j += NT)
                    if (idx[par][j] >= 0) psum += expf((val[par][j] - (best > -INFINITY ? best : 0.0f)) / a.T);
                psum = wave_sum(psum);
                if (GRAD && chunks == 1) twice = ix >= 0 && repeats(idx[par], a.top, ix) > 1;   // while the row arrives
            }

            // A running maximum and sum of 2^((z - mx) scale), 16 values at a time.
            constexpr int GR = 16 / E;
            float mx = -INFINITY, sx = 0.0f;
            auto running = [&](const u4 (&x)[GR]) {
                float m = mx;
#pragma unroll
                for (int b = 0; b < GR; ++b) {
                    float v[E];
                    Pc::get(x[b], v);
#pragma unroll
                    for (int i = 0; i < E; ++i) m = fmaxf(m, v[i]);
                }
                const float pv = m > -INFINITY ? m : 0.0f;
                sx *= mx > -INFINITY ? pow2((mx - pv) * a.scale) : 1.0f;
#pragma unroll
                for (int b = 0; b < GR; ++b) {
                    float v[E];
                    Pc::get(x[b], v);
#pragma unroll
                    for (int i = 0; i < E; ++i) sx += pow2((v[i] - pv) * a.scale);
                }
                mx = m;
                asm volatile("" : "+v"(sx), "+v"(mx));   // here, not where the sum is used: registers
            };
            auto running4 = [&](const u4& x0, const u4& x1, const u4& x2, const u4& x3) {
                if constexpr (GR == 4) {
                    running({x0, x1, x2, x3});
                } else {
                    running({x0, x1});
                    running({x2, x3});
                }
            };
#pragma unroll
            for (int q = 0; q < P; q += 4) {
                trim(c, r[q], r[q + 1], r[q + 2], r[q + 3], q * NT);
                running4(r[q], r[q + 1], r[q + 2], r[q + 3]);
                as_read(r[q], r[q + 1], r[q + 2], r[q + 3]);
            }
            if constexpr (L > 0) asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
#pragma unroll
            for (int o = 0; o < L; o += 4) {
                u4 x[4];
#pragma unroll
                for (int b = 0; b < 4; ++b) x[b] = hold[(o + b) * NT + tid];
                trim(c, x[0], x[1], x[2], x[3], (P + o) * NT);
                running4(x[0], x[1], x[2], x[3]);
            }
            if constexpr (REST)
                for (int at = (P + L) * NT; at < c.sp.pieces; at += 4 * NT) {
                    u4 x[4];
                    fetch_rest(c, x, at);
                    trim(c, x[0], x[1], x[2], x[3], at);
                    running4(x[0], x[1], x[2], x[3]);
                }
            // The wave's. mx = -inf with a sum: NaN values, which stay.
            const float m = wave_max(fmaxf(mx, edge_v)), pv = m > -INFINITY ? m : 0.0f;
            const float s = wave_sum(pow2((edge_v - pv) * a.scale) + (mx > -INFINITY ? sx * pow2((mx - pv) * a.scale) : sx));
            if (lane == 0) part[par][wave] = make_float4(m, s, best, psum);
            z_own = value_of(zr, DT);
            asm volatile("" : "+v"(z_own));   // it is there; later it would be waited for behind stores
        }
        __syncthreads();

        float pivot = 0.0f, s = 1.0f;
        bool on = look;   // a row takes part if the teacher has an entry and the student a logit above -inf
        if (look) {
            const float4 w = part[par][lane & (NW - 1)];
            const bool mine = lane < NW;
            const float m = wave_max(w.x), best = wave_max(w.z), tp = best > -INFINITY ? best : 0.0f;
            pivot = m > -INFINITY ? m : 0.0f;
            s = wave_sum(!mine ? 0.0f : w.x > -INFINITY ? w.y * pow2((w.x - pivot) * a.scale) : w.y);
            const float psum = wave_sum(!mine ? 0.0f : w.z > -INFINITY ? w.w * expf((w.z - tp) / a.T) : w.w);
            on = __builtin_amdgcn_readfirstlane(c.w != 0.0f && !(psum == 0.0f) && !(s == 0.0f));
            const float ls = logf(s);
            if (tid == 0 && a.lse) a.lse[row] = s == 0.0f ? -INFINITY : (float)((double)pivot / a.T + (double)ls);
            if (on && wave < chunks) {
                // The loss, entry by entry, and the entries' gradients: an
                // index is written by its first entry, for all of them.
                const float lp = logf(psum);
                float sum = 0.0f;
                auto entry = [&](int o, float zj) {
                    const int j = lane + 64 * o;
                    const int i = j < a.top ? idx[par][j] : -1;
                    const float lt = i >= 0 ? (val[par][j] - tp) / a.T : -INFINITY;
                    const float pj = i >= 0 ? expf(lt) / psum : 0.0f;
                    if (!(pj == 0.0f)) sum += pj * (lt - lp - ((zj - pivot) / a.T - ls));
                    if constexpr (GRAD) {
                        float pt = pj;
                        bool first = i >= 0;
                        if (chunks > 1) twice = first && repeats(idx[par], a.top, i) > 1;
                        if (twice)
                            for (int k = 0; k < a.top; ++k)
                                if (idx[par][k] == i && k != j) {
                                    first &= k > j;
                                    pt += expf((val[par][k] - tp) / a.T) / psum;
                                }
                        const unsigned long long set = __ballot(first);
                        if (lane == 0) gset[par][o] = set;
                        if (first) gval[par][j] = c.w * a.T * (pow2((zj - pivot) * a.scale) / s - pt);
                    }
                };
                entry(wave, z_own);
                for (int o = wave + NW; o < chunks; o += NW)
                    entry(o, value_of(raw_at(c.z, DT, max(idx[par][lane + 64 * o], 0)), DT));
                sum = wave_sum(sum);
                if (lane == 0) lsum[par][wave] = c.w * a.T * a.T * sum;
            }
        }
        if (!on && tid == 0 && a.loss) a.loss[row] = 0.0f;
        if constexpr (!GRAD) {
            __syncthreads();
            if (on) finish_row(row, par);
            return;
        }
        // The gradient may take the logits' place: no wave stores any of it
        // while another still reads the logits of its further entries.
        if constexpr (NW > 1 && TOP > 64 * NW)
            if (chunks > NW) __syncthreads();

        T* g = static_cast<T*>(a.grad) + row * a.ldg;
        const T* gb = g + c.sp.head;   // aligned to a value: the hardware's unaligned stores
        const __amdgpu_buffer_rsrc_t rg = dma::make_rsrc(gb, 16ll * c.sp.pieces);
        const float f = c.w * a.T / s;
        auto grad_of = [&](const u4& x) {
            u4 o = {0u, 0u, 0u, 0u};
            if (on) {
                float v[E];
                Pc::get(x, v);
#pragma unroll
                for (int i = 0; i < E; ++i) v[i] = f * pow2((v[i] - pivot) * a.scale);
                o = Pc::put(v);
                asm volatile("" : "+v"(o));
            }
            return o;
        };
        if constexpr (REST)
            for (int at = (P + L) * NT; at < c.sp.pieces; at += 4 * NT) {
                u4 x[4];
                fetch_rest(c, x, at);
                const __amdgpu_buffer_rsrc_t rs = dma::make_rsrc(gb + (long long)at * E, 16ll * (c.sp.pieces - at));
#pragma unroll
                for (int b = 0; b < 4; ++b) store_once(grad_of(x[b]), rs, (tid + b * NT) * 16);
            }
        fetch_entries(n, min(row + 2 * (long long)gridDim.x, a.rows - 1));
        if (before >= 0) finish_row(before, par ^ 1);   // behind the loads: its stores need not be waited for
        before = on ? row : -1;
#pragma unroll
        for (int o = 0; o < L; ++o) {
            store_once(grad_of(hold[o * NT + tid]), rg, (tid + (P + o) * NT) * 16);
            fetch_hold(n, o);
        }
#pragma unroll
        for (int q = 0; q < P; ++q) {
            store_once(grad_of(r[q]), rg, (tid + q * NT) * 16);
            fetch(n, q);
            __builtin_amdgcn_sched_barrier(0);
        }
        if (edge_at >= 0) g[edge_at] = (T)(on ? f * pow2((edge_v - pivot) * a.scale) : 0.0f);
        if (last) {
            __syncthreads();
            if (on) finish_row(row, par);
            if constexpr (L > 0) asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // no load into LDS outlives the workgroup
            return;
        }
        row += gridDim.x;
        c = n;
    }
}

// The gradient from a given lse: no sum over the row, so a row is cut into
// strips of NT x P pieces, a workgroup each. Up to 128 entries: a wave a strip
// with no barrier, as many as fit a CU; a wave's chain of loads (entries,
// their logits) is a few microseconds long.
template <int DT, int NT, int P, int TOP>
__global__ void __launch_bounds__(NT) distill_grad_kernel(DistillArgs a, int strips)
{
    typedef Piece<DT> Pc;
    typedef typename Pc::T T;
    constexpr int E = Pc::E, MORE = TOP / NT;
    static_assert(TOP % NT == 0 && MORE * NT == TOP, "entries a thread");
    __shared__ float val[TOP];
    __shared__ __attribute__((aligned(16))) int idx[TOP];
    __shared__ float red[NT / 64];
    const int tid = threadIdx.x;
    const long long row = blockIdx.x / strips;
    const int strip = blockIdx.x % strips;
    const T* z = static_cast<const T*>(a.z) + row * a.ldz;
    T* g = static_cast<T*>(a.grad) + row * a.ldg;
    const Span sp = span_of<DT>(z, a.V);
    const int first = strip * NT * P, here = sp.pieces - first;
    // Entries first: what hangs on them is the longer chain.
    int ix[MORE];
    unsigned tr[MORE], zr[MORE];
#pragma unroll
    for (int o = 0; o < MORE; ++o) {
        const long long j = row * a.top + min(tid + o * NT, a.top - 1);
        ix[o] = a.index[j];
        tr[o] = raw_at(a.t, a.t_dtype, j);
    }
    const __amdgpu_buffer_rsrc_t rz = dma::make_rsrc(reinterpret_cast<const u4*>(z + sp.head) + first, 16ll * here);
    // Aligned to a value: the hardware's unaligned stores.
    const __amdgpu_buffer_rsrc_t rg = dma::make_rsrc(g + sp.head + (long long)first * E, 16ll * here);
    u4 r[P];
#pragma unroll
    for (int q = 0; q < P; ++q) r[q] = __builtin_amdgcn_raw_buffer_load_b128(rz, tid * 16, q * NT * 16, 0);
    // The first strip takes the values before the pieces, the last those behind.
    int edge_at = -1;
    if (strip == 0 && tid < sp.head) edge_at = tid;
    if (strip == strips - 1 && tid >= 32 && tid - 32 < a.V - sp.tail0) edge_at = sp.tail0 + tid - 32;
    const unsigned edge_r = raw_at(z, DT, max(edge_at, 0));
    // Entries go to the strip that writes their place: those behind the
    // pieces are the last strip's, also where a strip before it ends there.
    const int begin = strip == 0 ? 0 : min(sp.head + first * E, sp.tail0);
    const int end = strip == strips - 1 ? a.V : min(sp.head + (first + NT * P) * E, sp.tail0);
    const float w = a.weight ? constant(a.weight, row) : 1.0f, lse = a.lse[row];
#pragma unroll
    for (int o = 0; o < MORE; ++o) {
        if (tid + o * NT >= a.top || (unsigned)ix[o] >= (unsigned)a.V) ix[o] = -1;
        zr[o] = raw_at(z, DT, max(ix[o], 0));
    }

    float best = -INFINITY, psum = 0.0f;
#pragma unroll
    for (int o = 0; o < MORE; ++o)
        if (ix[o] >= 0) best = fmaxf(best, value_of(tr[o], a.t_dtype));
    best = block_reduce<NT>(best, red, [](float x, float y) { return fmaxf(x, y); });
    const float tp = best > -INFINITY ? best : 0.0f;
    float pj[MORE];
#pragma unroll
    for (int o = 0; o < MORE; ++o) {
        pj[o] = ix[o] >= 0 ? expf((value_of(tr[o], a.t_dtype) - tp) / a.T) : 0.0f;
        psum += pj[o];
    }
    psum = block_reduce<NT>(psum, red, [](float x, float y) { return x + y; });
#pragma unroll
    for (int o = 0; o < MORE; ++o) {
        pj[o] = ix[o] >= 0 ? pj[o] / psum : 0.0f;
        idx[tid + o * NT] = ix[o];
        val[tid + o * NT] = pj[o];
    }
    __syncthreads();
    const bool on = w != 0.0f && !(psum == 0.0f) && !(lse == -INFINITY);
    const float wt = w * a.T;
    // lse is at least every v / T; where its rounding says otherwise (it is
    // coarse for logits next to a type's lowest value) q is 1, not more. A NaN
    // stays one.
    auto q_of = [&](float v) {
        const float d = fmaf(v, a.inv_hi, -lse) + v * a.inv_lo;
        return pow2((d > 0.0f ? 0.0f : d) * 1.44269504088896341f);
    };
    // An index is written by its first entry, for all of them.
    float gv[MORE];
#pragma unroll
    for (int o = 0; o < MORE; ++o) {
        gv[o] = 0.0f;
        if (!on || ix[o] < begin || ix[o] >= end) ix[o] = -1;
        if (ix[o] < 0) continue;
        const int i = ix[o], j = tid + o * NT;
        float pt = pj[o];
        if (repeats(idx, a.top, i) > 1)
            for (int k = 0; k < a.top; ++k)
                if (idx[k] == i && k != j) {
                    pt += val[k];
                    if (k < j) ix[o] = -1;
                }
        const float v = value_of(zr[o], DT);
        gv[o] = wt * ((v == -INFINITY ? 0.0f : q_of(v)) - pt);
    }
    __syncthreads();   // a wave's logits are all read before any of the row is written
#pragma unroll
    for (int q = 0; q < P; ++q) {
        float v[E];
        Pc::get(r[q], v);
#pragma unroll
        for (int k = 0; k < E; ++k) v[k] = !on || v[k] == -INFINITY ? 0.0f : wt * q_of(v[k]);
        store_once(Pc::put(v), rg, (tid + q * NT) * 16);
    }
    if (edge_at >= 0) {
        const float edge = value_of(edge_r, DT);
        g[edge_at] = (T)(!on || edge == -INFINITY ? 0.0f : wt * q_of(edge));
    }
    __syncthreads();
#pragma unroll
    for (int o = 0; o < MORE; ++o)
        if (ix[o] >= 0) g[ix[o]] = (T)gv[o];
}

// per: workgroups of a CU that take rows in turn.
template <int DT, int NT, int P, int L, bool REST = false, int TOP = kMaxTop>
hipError_t run(const DistillArgs& a, int per, hipStream_t s)
{
    const dim3 block(NT);
    if (a.grad)
        hipLaunchKernelGGL((distill_kernel<DT, NT, P, L, REST, true, TOP>),
                           dim3((unsigned)(a.rows < 256 * per ? a.rows : 256 * per)), block, 0, s, a);
    else   // the loss alone has no use for what it has read
        hipLaunchKernelGGL((distill_kernel<DT, NT, P, 0, REST, false, TOP>), dim3((unsigned)a.rows), block, 0, s, a);
    return hipGetLastError();
}

// Threads and registers by the row's length, so that each holds a row and two
// to four workgroups share a CU. Loss and gradient, bf16, 32 entries, us:
// 4096 x 32768: three of 512 threads 96, two 101, three of 256 with twice the
// registers 108, one of 1024 111; 4096 x 16000: four of 256 57, three of 512 75.
// Up to one row a CU: as many threads as fit, for latency (64 x 32768: 1024
// threads 9.6, 512 10.3; 256 rows 11.2 and 11.8; 400 rows 17.4 and 15.5. 256 x
// 65536: 14.9 and 15.6; 400 rows 26.6 and 22.0).
template <int DT>
hipError_t pick(const DistillArgs& a, hipStream_t s)
{
    const long long pieces = ((long long)a.V + Piece<DT>::E - 1) / Piece<DT>::E;
    const bool few = a.rows <= 256;
    // Many short rows: a wave each and no barrier, so that a CU has 16 to 20
    // on their way (4096 x 4000: four of 256 threads 38 us, this 20; 1400 x
    // 8000: both 18; 1024 rows of 1500, 4000, 8000: 13.1, 13.1, 13.9 with 256
    // threads and 9.5, 10.7, 14.0 this way; 512 of 8000: 11.1 and 12.4).
    if (a.rows > 1024 && a.top <= kFewTop) {
        if (pieces <= 64 * 4) return run<DT, 64, 4, 0, false, kFewTop>(a, 20, s);
        if (pieces <= 64 * 8) return run<DT, 64, 8, 0, false, kFewTop>(a, 20, s);
        if (pieces <= 64 * 16) return run<DT, 64, 16, 0, false, kFewTop>(a, 16, s);
    }
    if (pieces <= 256 * 4) return run<DT, 256, 4, 0>(a, 4, s);
    if (few && pieces <= 1024 * 4) return run<DT, 1024, 4, 0>(a, 1, s);
    if (few && pieces <= 1024 * 8) return run<DT, 1024, 8, 0>(a, 1, s);
    if (pieces <= 256 * 8) return run<DT, 256, 8, 0>(a, 4, s);
    if (pieces <= 512 * 8) return run<DT, 512, 8, 0>(a, 3, s);
    if (pieces <= 512 * 16) return run<DT, 512, 16, 0>(a, 2, s);
    if (pieces <= 1024 * 16) return run<DT, 1024, 16, 0>(a, 1, s);
    return run<DT, 1024, 20, 8, true>(a, 1, s);
}

}  // namespace

hipError_t launch_distill(int dtype, const DistillArgs& a, hipStream_t s)
{
    if (dtype == DT_F32) return pick<DT_F32>(a, s);
    return dtype == DT_BF16 ? pick<DT_BF16>(a, s) : pick<DT_F16>(a, s);
}

namespace {

template <int DT, int NT, int P, int TOP>
hipError_t run_grad(const DistillArgs& a, hipStream_t s)
{
    const long long per = (long long)NT * P * Piece<DT>::E;
    const int strips = (int)((a.V + per - 1) / per);
    hipLaunchKernelGGL((distill_grad_kernel<DT, NT, P, TOP>), dim3((unsigned)(a.rows * strips)), dim3(NT), 0, s, a, strips);
    return hipGetLastError();
}

template <int DT>
hipError_t pick_grad(const DistillArgs& a, hipStream_t s)
{
    if (a.top > kFewTop) return run_grad<DT, 256, 16, kMaxTop>(a, s);
    const long long pieces = ((long long)a.V + Piece<DT>::E - 1) / Piece<DT>::E;
    if (pieces <= 64 * 4) return run_grad<DT, 64, 4, kFewTop>(a, s);
    // Strips of 8 pieces a lane while their number fits a grid (checked for strips of twice that).
    if (pieces <= 64 * 8 || a.rows * (pieces / 512 + 1) < (1ll << 31) - 1) return run_grad<DT, 64, 8, kFewTop>(a, s);
    return run_grad<DT, 256, 16, kMaxTop>(a, s);
}

}  // namespace

hipError_t launch_distill_grad(int dtype, const DistillArgs& a, hipStream_t s)
{
    if (dtype == DT_F32) return pick_grad<DT_F32>(a, s);
    return dtype == DT_BF16 ? pick_grad<DT_BF16>(a, s) : pick_grad<DT_F16>(a, s);
}

}  // namespace sam
