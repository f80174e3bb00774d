// Entry points of the adapter projection (declared in include/sam.h):
// argument checks, the choice between a product with the adapters' term
// inside its tiles and a split product with the term added by the pass that
// sums it, and the launches. Everything that can be rejected is rejected
// before any HIP call.
#include "sam_adapter.h"
#include "sam_check.h"

using namespace sam;

namespace {

constexpr int kBK = 64;         // K per ring stage
constexpr int kCUs = 256;

struct Region {
    unsigned long long off = 0, bytes = 0;
};

// A product rows x cols over `k` with the adapters' term, and how it runs.
struct Product {
    int tile;          // launch_adapter_ring's
    int split;         // 0: whole K with the term inside the tile; else K ranges
    int k_chunk;
    int tiles_m, tiles_n;
};

// Fused tiles take whole K, a round of them as long as the K loop; the rates
// are those the ring kernels reach with all CUs busy, as parts of the matrix
// peak. A split product fills the CUs with few tiles, but writes and reads its
// partials once more.
// `beside`: the pass that adds the partials has a launch to go with.
Product choose(long long rows, long long cols, long long k, bool beside)
{
    static const struct { int tile; double rate; } fused[] = {{0, 0.575}, {1, 0.545}, {2, 0.40}};
    Product best{};
    double best_cost = 0;
    for (const auto& f : fused) {
        const AdapterTile t = adapter_tile(f.tile);
        const long long tm = (rows + t.bm - 1) / t.bm, tn = (cols + t.bn - 1) / t.bn;
        const double cost = (double)((tm * tn + kCUs - 1) / kCUs) * t.bm * t.bn / f.rate;
        if (!best_cost || cost < best_cost) {
            best_cost = cost;
            best = {f.tile, 0, 0, (int)tm, (int)tn};
        }
    }
    if (rows == 0 || k <= 4 * kBK) return best;   // no rows: no tiles to share the CUs
    Product p{};
    p.tile = rows <= 16 ? 5 : (rows <= 32 ? 4 : (rows <= 64 ? 3 : 2));
    const AdapterTile t = adapter_tile(p.tile);
    p.tiles_m = (int)((rows + t.bm - 1) / t.bm);
    p.tiles_n = (int)((cols + t.bn - 1) / t.bn);
    // One workgroup a CU: two read W no faster (one row x 4096 x 4096: 10.5 us
    // with two, 9.2 with one) and leave twice the partials.
    long long s = kCUs / ((long long)p.tiles_m * p.tiles_n);
    const long long most = (k + 4 * kBK - 1) / (4 * kBK);
    s = s < 1 ? 1 : (s > most ? most : s);
    p.k_chunk = (int)(((k + s - 1) / s + kBK - 1) / kBK * kBK);
    p.split = (int)((k + p.k_chunk - 1) / p.k_chunk);
    if (rows <= 64) return p;
    // 7.6 us per 1024 values of K in a tile, 0.9 us per MB of partials, and
    // what the launches cost: T of up to 128 rows takes one more beside a
    // fused product, the sum of the partials none where it goes with the
    // adapters' gradients. As measured over 100 to 1024 rows, K and N 512 to 4096,
    // bf16, rank 16 (512 x 512 x 4096: 17.5 us fused, 31 split; 1024 x 2048 x
    // 2048: 31 and 35; 256 x 4096 x 2048: 45 and 30; 100 x 1024 x 4096: 25 and 21).
    const double fused_us = 14 + (rows <= 128 ? 3 : 0) + 7.6 / 1024 * k;
    const double split_us = (beside ? 9 : 13) + 7.6 / 1024 * p.k_chunk + 0.9e-6 * 4 * p.split * rows * cols;
    return fused_us <= split_us ? best : p;
}

int round8(long long x) { return (int)((x + 7) & ~7ll); }

struct Call {
    int dtype, out, trans_w;
    long long M, N, K, n, r;
    long long ldx, ldw, ldy, lddy, lddx;
    bool back, want_dx, want_ad;
};

struct Layout {
    int rp;
    Product prod;
    int np;                        // 16-bit values that a T in t16 is made of
    int wide, ksplit, slots;       // shrink
    int merged;                    // ... in the split product's own launch
    bool pad_x, pad_w, pad_a, pad_b, pad_dy;
    long long lx, lw, la, lb, ldy; // row strides that the kernels see
    Region x, w, a, b, dy;         // padded copies
    Region t32, t32b, t16, factor, part, order, seg, chunk_first, part_first, chunks, outer;
    int chunk, max_chunks, max_parts;
    unsigned long long total;
};

sam_status check_sizes(const Call& c)
{
    if (c.dtype != SAM_BF16 && c.dtype != SAM_F16)
        return api_fail(SAM_ERR_INVALID_ARG, "adapter projection: operands must be SAM_BF16 or SAM_F16, not dtype %d", c.dtype);
    if (c.out != c.dtype && c.out != SAM_F32)
        return api_fail(SAM_ERR_INVALID_ARG, "result type %d is neither SAM_F32 nor the operands' type", c.out);
    if (c.trans_w != SAM_OP_N && c.trans_w != SAM_OP_T)
        return api_fail(SAM_ERR_INVALID_ARG, "trans_w must be SAM_OP_N or SAM_OP_T");
    if (c.M < 0 || c.N < 1 || c.K < 1 || c.n < 0)
        return api_fail(SAM_ERR_INVALID_ARG, "bad sizes M=%lld N=%lld K=%lld adapters=%lld", c.M, c.N, c.K, c.n);
    if (c.n > 0 && (c.r < 1 || c.r > kMaxRank))
        return api_fail(SAM_ERR_INVALID_ARG, "rank %lld outside 1 .. %d", c.r, kMaxRank);
    const long long most = (1ll << 31) - 1024, row = 0x7FFFFFF0ll / (257 * 4);
    if (c.M > most || c.n > (1 << 20))
        return api_fail(SAM_ERR_INVALID_ARG, "M=%lld or %lld adapters too many", c.M, c.n);
    const long long min_w = c.trans_w ? c.K : c.N;
    if (c.ldx < c.K || c.ldw < min_w || (!c.back && c.ldy < c.N) || (c.back && c.lddy < c.N) ||
        (c.back && c.want_dx && c.lddx < c.K))
        return api_fail(SAM_ERR_INVALID_ARG, "a row stride is smaller than its row");
    if (c.ldx > row || c.ldw > row || c.ldy > row || c.lddy > row || c.lddx > row || c.N > row || c.K > row)
        return api_fail(SAM_ERR_INVALID_ARG, "N, K or a row stride beyond the supported offset range (%lld)", row);
    return SAM_OK;
}

Layout layout(const Call& c)
{
    Layout L{};
    L.rp = c.n == 0 ? 0 : (c.r > 64 ? 128 : (c.r > 32 ? 64 : (c.r > 16 ? 32 : 16)));
    const long long rows = c.M, cols = c.back ? c.K : c.N, k = c.back ? c.N : c.K;
    L.prod = choose(rows, cols, k, c.back && c.want_ad && c.n);
    unsigned long long at = 0;
    auto take = [&](Region& r, unsigned long long bytes) {
        r.off = at;
        r.bytes = bytes;
        at += align256(bytes);
    };
    // Rows that are no whole 16-byte pieces are copied into rows that are.
    const long long wr = c.trans_w ? c.N : c.K, wc = c.trans_w ? c.K : c.N;   // W as stored
    L.pad_x = c.K % 8 || c.ldx % 8;
    // Of W only where its rows run along the product's K: values behind a
    // shorter row then reach columns that are not stored, and they share their
    // 16 aligned bytes with the row's last ones.
    const bool along_k = (c.trans_w != 0) != c.back;
    L.pad_w = (along_k && wc % 8) || c.ldw % 8;
    L.pad_a = c.n && c.K % 8;
    L.pad_b = c.n && c.N % 8;
    L.pad_dy = c.back && (c.N % 8 || c.lddy % 8);
    if (c.back && !c.want_dx) L.pad_w = false;
    if (c.back && !c.want_ad) L.pad_x = false;
    L.lx = L.pad_x ? round8(c.K) : c.ldx;
    L.lw = L.pad_w ? round8(wc) : c.ldw;
    L.la = L.pad_a ? round8(c.K) : c.K;
    L.lb = L.pad_b ? round8(c.N) : c.N;
    L.ldy = L.pad_dy ? round8(c.N) : c.lddy;
    if (L.pad_x) take(L.x, 2ull * c.M * L.lx);
    if (L.pad_w) take(L.w, 2ull * wr * L.lw);
    if (L.pad_a) take(L.a, 2ull * c.n * c.r * L.la);
    if (L.pad_b) take(L.b, 2ull * c.n * c.r * L.lb);
    if (L.pad_dy) take(L.dy, 2ull * c.M * L.ldy);

    // Shrink. Many rows: 64 a workgroup, K cut such that two workgroups a CU
    // share the work (at least 256 values of K each). Up to 128 rows: 16 a
    // workgroup, the distinct adapters of a block (up to 16) and K ranges of
    // what a workgroup loads at once on workgroups of their own. In the first
    // form a block's second adapter has a workgroup too, and the CUs room for
    // 64 of them: few blocks have one in long runs, but two passes of one
    // workgroup, or one that starts when another ends, last as long as two of
    // all (4096 x 11008, rank 64, 4 adapters in runs: 39 us, so 36).
    const int sides = c.back && c.want_ad ? 2 : 1;
    const long long blocks = (c.M + 15) / 16, longest = c.back && c.N > c.K ? c.N : c.K;
    L.wide = blocks > 8;
    L.merged = c.M > 0 && L.prod.split > 0 && L.prod.tile >= 3 && (!c.back || c.want_dx);
    long long s, most;
    if (L.wide) {
        s = (2 * kCUs - 64) / ((c.M + 63) / 64 * sides);
        // One range is rounded where it is made, a launch less; from 1536
        // values on several are sooner there all the same (256 x 2048, N 4096:
        // 34 us and 32; 2049 x 1536: 46 and 47; 4096 x 1024: 46 and 49).
        most = !c.back && c.K <= 1536 ? 1 : (longest + 255) / 256;
    } else {
        s = (longest + 1023) / 1024 * (L.merged && L.prod.tile == 5 ? 2 : 1);   // waves: four, or the narrowest tile's two
        most = 16;
    }
    L.ksplit = (int)(s < 1 ? 1 : (s > most ? most : s));
    s = L.wide ? 4 * kCUs / ((c.M + 63) / 64 * sides * L.ksplit) : 16;
    s = L.wide ? (s < 2 ? 2 : (s > 8 ? 8 : s)) : s;
    L.slots = (int)(s > c.n ? (c.n ? c.n : 1) : s);
    // T inside a tile as two values of the operands' type (16 or 22 bits); an
    // FP32 result of bfloat16 gets three, all 24.
    L.np = c.dtype == SAM_BF16 && c.out == SAM_F32 ? 3 : 2;
    if (c.n) {
        const bool fused = L.prod.split == 0;
        const unsigned long long t = 4ull * c.M * L.rp;
        if (!c.back) {
            take(L.t32, t * L.ksplit);
            if (fused) {
                take(L.t16, t / 2 * L.np);
                take(L.factor, 4ull * c.M);
            }
        } else {
            // T of X (for dB), T of dY (for dA and, rounded, for dX).
            take(L.t32, t * L.ksplit);
            take(L.t32b, t * L.ksplit);
            take(L.t16, t / 2 * L.np);
            take(L.factor, 4ull * c.M);
            take(L.order, 4ull * (c.M + 1));
            take(L.seg, 4ull * (c.n + 1));
        }
    }
    if (L.prod.split > 0 && (!c.back || c.want_dx)) take(L.part, 4ull * L.prod.split * c.M * round8(cols));
    if (c.back && c.want_ad && c.n) {
        // Chunks of rows such that two to four workgroups a CU share the work
        // (4096 rows, 8192 columns: 256 rows 22 us, 128 the same and twice the
        // partials; 1025 rows, 2817 columns: 256 rows 18 us, 64 9 us).
        const long long strips = (c.K + 255) / 256 + (c.N + 255) / 256;
        // Up to 128 rows are one chunk: nothing is left to add.
        long long chunk = c.M <= 128 ? 128 : 64;
        while (chunk < (1 << 20) && (c.M / (2 * chunk)) * strips >= 2 * kCUs) chunk *= 2;
        L.chunk = (int)chunk;
        L.max_chunks = (int)((c.M + chunk - 1) / chunk + c.n);
        // Partials: of adapters with more than `chunk` rows, of which there are
        // no more than M / (chunk + 1); the others' sums are results at once.
        const long long several = c.M / (chunk + 1);
        L.max_parts = (int)(several ? c.M / chunk + (several < c.n ? several : c.n) : 0);
        take(L.outer, 4ull * L.max_parts * c.r * (c.K + c.N));
        take(L.part_first, 4ull * c.n);
        take(L.chunk_first, 4ull * (c.n + 1));
        take(L.chunks, 16ull * (L.max_chunks + 1));
    }
    L.total = at;
    return L;
}

struct Ptrs {
    const void *X, *W, *A, *B, *dY;
    const int* ids;
    const float* scale;
    void* Y;       // forward: Y, backward: dX
    float *dA, *dB;
};

GemmArgs ring_args(const Product& p, const void* X, long long lx, const void* W, long long lw, long long M, long long cols,
                   long long k, float* part)
{
    GemmArgs g{};
    g.A = X;
    g.B = W;
    g.lda = (int)lx;
    g.ldb = (int)lw;
    g.M = (int)M;
    g.N = round8(cols);
    g.K = (int)k;
    g.split = p.split ? p.split : 1;
    g.k_chunk = p.split ? p.k_chunk : (int)((k + kBK - 1) / kBK * kBK);
    g.tiles_m = p.tiles_m;
    g.tiles_n = p.tiles_n;
    g.group_m = 8;
    g.xcd_remap = 1;
    g.raster_n = 1;
    g.out = part;
    g.ldc = g.N;
    g.part_stride = (long long)M * g.N;
    g.alpha = 1.0f;
    return g;
}

sam_status enqueue(const Call& c, const Layout& L, Ptrs p, void* ws, hipStream_t s)
{
    char* wsb = static_cast<char*>(ws);
    auto at = [&](const Region& r) -> void* { return r.bytes ? wsb + r.off : nullptr; };
    // Padded copies, one launch.
    PadCopy pads[kMaxPads];
    int np = 0;
    auto pad = [&](bool on, const void*& src, long long ld, const Region& r, long long ldd, long long rows, long long cols) {
        if (!on || rows == 0) return;
        pads[np++] = {src, ld, at(r), ldd, rows, cols};
        src = at(r);
    };
    const long long wr = c.trans_w ? c.N : c.K, wc = c.trans_w ? c.K : c.N;
    pad(L.pad_x, p.X, c.ldx, L.x, L.lx, c.M, c.K);
    pad(L.pad_w, p.W, c.ldw, L.w, L.lw, wr, wc);
    pad(L.pad_a, p.A, c.K, L.a, L.la, c.n * c.r, c.K);
    pad(L.pad_b, p.B, c.N, L.b, L.lb, c.n * c.r, c.N);
    pad(L.pad_dy, p.dY, c.lddy, L.dy, L.ldy, c.M, c.N);
    hipError_t e = np ? launch_adapter_pad(pads, np, s) : hipSuccess;

    const bool fused = L.prod.split == 0;
    const bool term = c.n > 0;
    const int out16 = c.out != SAM_F32;
    // T's sums are added by the pass that takes them, if that is the finish of
    // the forward pass; otherwise they are added and rounded first.
    ShrinkArgs a{};
    if (term) {
        a.M = (int)c.M;
        a.n = (int)c.n;
        a.r = (int)c.r;
        a.rp = L.rp;
        a.ids = p.ids;
        a.scale = p.scale;
        a.np = L.np;
        a.wide = L.wide;
        a.round = c.back || fused || L.wide;
        a.ksplit = L.ksplit;
        a.slots = L.slots;
        a.sides = 1;
        const ShrinkSide x = {p.X, L.lx, p.A, L.la, (int)c.K, static_cast<float*>(at(L.t32)), c.back || !fused, nullptr, nullptr};
        if (!c.back) {
            a.side[0] = x;
            a.side[0].t16 = at(L.t16);
            a.side[0].factor = static_cast<float*>(at(L.factor));
        } else {
            a.side[0] = {p.dY, L.ldy, p.B, L.lb, (int)c.N, static_cast<float*>(at(L.t32b)), 1, at(L.t16),
                         static_cast<float*>(at(L.factor))};
            if (c.want_ad) {
                a.sides = 2;
                a.side[1] = x;
                a.order = static_cast<int*>(at(L.order));
                a.seg = static_cast<int*>(at(L.seg));
                a.chunk = L.chunk;
                a.max_chunks = L.max_chunks;
                a.chunk_first = static_cast<int*>(at(L.chunk_first));
                a.part_first = static_cast<int*>(at(L.part_first));
                a.chunks = static_cast<int4*>(at(L.chunks));
            }
        }
        if (!L.merged && (c.M > 0 || c.want_ad)) {
            if (e == hipSuccess) e = launch_adapter_shrink(c.dtype, a, s);
            if (e == hipSuccess && a.round) e = launch_adapter_round(c.dtype, a, s);
        }
    }
    FinishArgs f{};
    bool finish = false;   // the split product's partials are still to be added
    if (e == hipSuccess && c.M > 0 && (!c.back || c.want_dx)) {
        const long long cols = c.back ? c.K : c.N, k = c.back ? c.N : c.K;
        const void* X = c.back ? p.dY : p.X;
        const long long lx = c.back ? L.ldy : L.lx;
        const void* B = c.back ? p.A : p.B;
        const long long lb = c.back ? L.la : L.lb;
        const long long ldo = c.back ? c.lddx : c.ldy;
        // Forward reads W as k rows of cols unless it is stored transposed,
        // the backward pass the other way round.
        const int bt = (c.trans_w != 0) != c.back;
        const GemmArgs g = ring_args(L.prod, X, lx, p.W, L.lw, c.M, cols, k, static_cast<float*>(at(L.part)));
        if (fused) {
            AdapterRing x{};
            x.B = B;
            x.ldb = lb;
            x.nb = round8(cols);
            x.n = (int)c.n;
            x.r = (int)c.r;
            x.rp = L.rp;
            x.M = (int)c.M;
            x.N = (int)cols;
            x.ids = p.ids;
            x.t16 = at(L.t16);
            x.np = L.np;
            x.factor = static_cast<const float*>(at(L.factor));
            x.Y = p.Y;
            x.ldy = ldo;
            x.out16 = out16;
            e = launch_adapter_ring(L.prod.tile, c.dtype, bt, g, (int)cols, &x, nullptr, s);
        } else {
            const ShrinkArgs none{};
            e = launch_adapter_ring(L.prod.tile, c.dtype, bt, g, (int)cols, nullptr, L.merged && term ? &a : &none, s);
            if (e == hipSuccess && L.merged && term && a.round) e = launch_adapter_round(c.dtype, a, s);
            finish = true;
            f.part = g.out;
            f.ldp = g.N;
            f.split = L.prod.split;
            f.t32 = static_cast<const float*>(c.back ? at(L.t32b) : at(L.t32));
            f.tsplit = a.round ? 1 : L.ksplit;
            f.B = B;
            f.ldb = lb;
            f.ids = p.ids;
            f.M = (int)c.M;
            f.N = (int)cols;
            f.n = (int)c.n;
            f.r = (int)c.r;
            f.rp = L.rp;
            f.Y = p.Y;
            f.ldy = ldo;
            f.out16 = out16;
        }
    }
    if (e == hipSuccess && c.back && c.want_ad && term) {
        OuterArgs o{};
        o.M = (int)c.M;
        o.n = (int)c.n;
        o.r = (int)c.r;
        o.rp = L.rp;
        o.order = static_cast<const int*>(at(L.order));
        o.chunk = L.chunk;
        o.max_chunks = L.max_chunks;
        o.chunk_first = a.chunk_first;
        o.part_first = a.part_first;
        o.chunks = a.chunks;
        float* part = static_cast<float*>(at(L.outer));
        o.side[0] = {static_cast<const float*>(at(L.t32b)), p.X, L.lx, (int)c.K, p.dA, part};
        o.side[1] = {static_cast<const float*>(at(L.t32)), p.dY, L.ldy, (int)c.N, p.dB,
                     part + (long long)L.max_parts * c.r * c.K};
        e = launch_adapter_outer(c.dtype, o, finish ? &f : nullptr, s);
    } else if (e == hipSuccess && finish) {
        e = launch_adapter_finish(c.dtype, f, s);
    }
    if (e != hipSuccess) return api_fail(SAM_ERR_LAUNCH, "kernel launch failed: %s", hipGetErrorString(e));
    return api_ok();
}

struct Buf {
    const void* p;
    unsigned long long bytes;
    const char* name;
    int align;
    bool written;
};

// Null, alignment and overlap: nothing that is written may overlap anything else.
sam_status check_buffers(const Buf* b, int n)
{
    for (int i = 0; i < n; ++i) {
        if (b[i].bytes && !b[i].p) return api_fail(SAM_ERR_INVALID_ARG, "%s is null", b[i].name);
        if (b[i].bytes && (b[i].align == 16 ? !aligned16(b[i].p) : !aligned4(b[i].p)))
            return api_fail(SAM_ERR_MISALIGNED, "%s must be %d-byte aligned", b[i].name, b[i].align);
    }
    for (int i = 0; i < n; ++i)
        for (int j = 0; j < n; ++j)
            if (i != j && b[i].written && ranges_overlap(b[i].p, b[i].bytes, b[j].p, b[j].bytes))
                return api_fail(SAM_ERR_INVALID_ARG, "%s overlaps %s", b[i].name, b[j].name);
    return SAM_OK;
}

unsigned long long span(long long rows, long long ld, long long cols, int es)
{
    return rows > 0 ? ((unsigned long long)(rows - 1) * ld + cols) * es : 0;
}

// A single row's stride reaches nothing: it is neither a reason to refuse it
// nor one to copy it.
long long stride_of(long long rows, long long ld, long long cols)
{
    return rows <= 1 && cols >= 1 && cols < (1ll << 31) && ld > round8(cols) ? round8(cols) : ld;
}

Call forward_call(int dtype, int trans_w, long long M, long long N, long long K, long long n, long long r, long long ldx,
                  long long ldw, int out, long long ldy)
{
    Call c{};
    c.dtype = dtype;
    c.trans_w = trans_w;
    c.M = M;
    c.N = N;
    c.K = K;
    c.n = n;
    c.r = r;
    c.ldx = stride_of(M, ldx, K);
    c.ldw = stride_of(trans_w ? N : K, ldw, trans_w ? K : N);
    c.out = out;
    c.ldy = stride_of(M, ldy, N);
    return c;
}

}  // namespace

extern "C" {

sam_status sam_adapter_gemm_workspace(sam_dtype dtype, sam_op trans_w, int64_t M, int64_t N, int64_t K, int64_t n_adapters,
                                      int64_t rank, int64_t ldx, int64_t ldw, uint64_t* bytes)
{
    if (!bytes) return api_fail(SAM_ERR_INVALID_ARG, "bytes is null");
    // FP32 results need the most.
    const Call c = forward_call(dtype, trans_w, M, N, K, n_adapters, rank, ldx, ldw, SAM_F32, N);
    const sam_status st = check_sizes(c);
    if (st != SAM_OK) return st;
    *bytes = M == 0 ? 0 : layout(c).total;
    return api_ok();
}

sam_status sam_adapter_gemm(sam_dtype dtype, sam_op trans_w, int64_t M, int64_t N, int64_t K, int64_t n_adapters,
                            int64_t rank, const void* X, int64_t ldx, const void* W, int64_t ldw, const void* A,
                            const void* B, const int32_t* ids, const float* scale, sam_dtype out, void* Y, int64_t ldy,
                            void* workspace, uint64_t workspace_bytes, void* stream)
{
    const Call c = forward_call(dtype, trans_w, M, N, K, n_adapters, rank, ldx, ldw, out, ldy);
    sam_status st = check_sizes(c);
    if (st != SAM_OK) return st;
    if (M == 0) return api_ok();
    const Layout L = layout(c);
    const long long wr = trans_w ? N : K, wc = trans_w ? K : N;
    const Buf bufs[] = {
        {X, span(M, ldx, K, 2), "X", 16, false},
        {W, span(wr, ldw, wc, 2), "W", 16, false},
        {A, 2ull * n_adapters * rank * K, "A", 16, false},
        {B, 2ull * n_adapters * rank * N, "B", 16, false},
        {ids, 4ull * M, "ids", 4, false},
        {scale, scale ? 4ull * n_adapters : 0, "scale", 4, false},
        {Y, span(M, ldy, N, out == SAM_F32 ? 4 : 2), "Y", 16, true},
        {workspace, workspace ? L.total : 0, "workspace", 16, true},
    };
    st = check_buffers(bufs, sizeof(bufs) / sizeof(bufs[0]));
    if (st != SAM_OK) return st;
    if (L.total && (!workspace || workspace_bytes < L.total))
        return api_fail(SAM_ERR_WORKSPACE, "the call needs %llu workspace bytes, got %llu", L.total,
                        (unsigned long long)(workspace ? workspace_bytes : 0));
    st = api_device_check();
    if (st != SAM_OK) return st;
    Ptrs p{};
    p.X = X;
    p.W = W;
    p.A = A;
    p.B = B;
    p.ids = ids;
    p.scale = scale;
    p.Y = Y;
    return enqueue(c, L, p, workspace, static_cast<hipStream_t>(stream));
}

static Call backward_call(sam_dtype dtype, sam_op trans_w, int64_t M, int64_t N, int64_t K, int64_t n, int64_t r,
                          int64_t lddy, int64_t ldx, int64_t ldw, sam_dtype out, bool dx, int64_t lddx, bool ad)
{
    Call c = forward_call(dtype, trans_w, M, N, K, n, r, ldx, ldw, out, N);
    c.back = true;
    c.lddy = stride_of(M, lddy, N);
    c.want_dx = dx;
    c.lddx = dx ? stride_of(M, lddx, K) : K;
    c.want_ad = ad;
    return c;
}

sam_status sam_adapter_backward_workspace(sam_dtype dtype, sam_op trans_w, int64_t M, int64_t N, int64_t K,
                                          int64_t n_adapters, int64_t rank, int64_t lddy, int64_t ldx, int64_t ldw,
                                          int32_t want_dx, int32_t want_dab, uint64_t* bytes)
{
    if (!bytes) return api_fail(SAM_ERR_INVALID_ARG, "bytes is null");
    const Call c = backward_call(dtype, trans_w, M, N, K, n_adapters, rank, lddy, ldx, ldw, SAM_F32, want_dx != 0, K,
                                 want_dab != 0);
    const sam_status st = check_sizes(c);
    if (st != SAM_OK) return st;
    *bytes = layout(c).total;
    return api_ok();
}

sam_status sam_adapter_backward(sam_dtype dtype, sam_op trans_w, int64_t M, int64_t N, int64_t K, int64_t n_adapters,
                                int64_t rank, const void* dY, int64_t lddy, const void* X, int64_t ldx, const void* W,
                                int64_t ldw, const void* A, const void* B, const int32_t* ids, const float* scale,
                                sam_dtype out, void* dX, int64_t lddx, float* dA, float* dB, void* workspace,
                                uint64_t workspace_bytes, void* stream)
{
    if ((dA != nullptr) != (dB != nullptr))
        return api_fail(SAM_ERR_INVALID_ARG, "dA and dB are wanted together or not at all");
    const Call c = backward_call(dtype, trans_w, M, N, K, n_adapters, rank, lddy, ldx, ldw, out, dX != nullptr, lddx,
                                 dA != nullptr);
    sam_status st = check_sizes(c);
    if (st != SAM_OK) return st;
    if (!c.want_dx && !c.want_ad) return api_ok();
    const Layout L = layout(c);
    const long long wr = trans_w ? N : K, wc = trans_w ? K : N;
    const unsigned long long nr = (unsigned long long)n_adapters * (n_adapters ? rank : 0);
    const Buf bufs[] = {
        {dY, span(M, lddy, N, 2), "dY", 16, false},
        {X, c.want_ad ? span(M, ldx, K, 2) : 0, "X", 16, false},
        {W, c.want_dx ? span(wr, ldw, wc, 2) : 0, "W", 16, false},
        {A, 2ull * nr * K, "A", 16, false},
        {B, 2ull * nr * N, "B", 16, false},
        {ids, 4ull * M, "ids", 4, false},
        {scale, scale ? 4ull * n_adapters : 0, "scale", 4, false},
        {dX, dX ? span(M, lddx, K, out == SAM_F32 ? 4 : 2) : 0, "dX", 16, true},
        {dA, dA ? 4ull * nr * K : 0, "dA", 16, true},
        {dB, dB ? 4ull * nr * N : 0, "dB", 16, true},
        {workspace, workspace ? L.total : 0, "workspace", 16, true},
    };
    st = check_buffers(bufs, sizeof(bufs) / sizeof(bufs[0]));
    if (st != SAM_OK) return st;
    if (L.total && (!workspace || workspace_bytes < L.total))
        return api_fail(SAM_ERR_WORKSPACE, "the call needs %llu workspace bytes, got %llu", L.total,
                        (unsigned long long)(workspace ? workspace_bytes : 0));
    st = api_device_check();
    if (st != SAM_OK) return st;
    Ptrs p{};
    p.dY = dY;
    p.X = X;
    p.W = W;
    p.A = A;
    p.B = B;
    p.ids = ids;
    p.scale = scale;
    p.Y = dX;
    p.dA = dA;
    p.dB = dB;
    return enqueue(c, L, p, workspace, static_cast<hipStream_t>(stream));
}

}  // extern "C"
