// Entry points of the MXFP4 tensors and the 4-bit projection (declared in
// include/sam.h): argument checks, workspace layout and launches. Everything
// that can be rejected is rejected before any HIP call.
#include "sam_check.h"
#include "sam_mxfp4.h"

using namespace sam;

namespace {

constexpr long long kMostRow = 0x7FFFFFF0ll / (257 * 4);   // the products' offset range
// Blocks of a tensor, and those of a product's operands in whole 128 values: a
// launch has up to 2^32 threads, two a block (and the copies of the scales).
constexpr long long kMostBlocks = (1ll << 31) - 4096, kMostOperand = (1ll << 31) - (1ll << 28);

int elem(int dtype) { return dtype == SAM_F32 ? 4 : 2; }

bool value_type(int dtype) { return dtype >= SAM_F32 && dtype <= SAM_F16; }

long long blocks_of(long long K) { return (K + 31) / 32; }

// A tensor of `rows` rows of K values beside its codes. lines x line: how the
// values are stored.
sam_status check_tensor(int dtype, long long rows, long long K, long long lines, long long line, long long ldx)
{
    if (!value_type(dtype)) return api_fail(SAM_ERR_INVALID_ARG, "bad dtype %d", dtype);
    if (rows < 0 || K < 1 || rows > (1ll << 30) || K > (1ll << 31) - 64 || rows > kMostBlocks / blocks_of(K))
        return api_fail(SAM_ERR_INVALID_ARG, "bad sizes rows=%lld K=%lld", rows, K);
    if (lines > 1 && (ldx < line || ldx > (1ll << 40)))
        return api_fail(SAM_ERR_INVALID_ARG, "row stride %lld (rows of %lld)", ldx, line);
    return SAM_OK;
}

sam_status done(hipError_t e)
{
    return e == hipSuccess ? api_ok() : api_fail(SAM_ERR_LAUNCH, "kernel launch failed: %s", hipGetErrorString(e));
}

struct Region {
    unsigned long long off = 0, bytes = 0;
};

struct Layout {
    Region codes, scales, wscales, parts;   // forward
    Region w, inner;                        // backward
    unsigned long long total = 0;
    void take(Region& r, unsigned long long bytes)
    {
        r.off = total;
        r.bytes = bytes;
        total += align256(bytes);
    }
};

sam_status check_linear(int dtype, int out, long long M, long long N, long long K)
{
    if (!value_type(dtype)) return api_fail(SAM_ERR_INVALID_ARG, "bad dtype %d", dtype);
    if (out != dtype && out != SAM_F32)
        return api_fail(SAM_ERR_INVALID_ARG, "result type %d is neither SAM_F32 nor the operand's type", out);
    if (M < 0 || N < 1 || K < 1 || N > kMostRow || K > kMostRow)
        return api_fail(SAM_ERR_INVALID_ARG, "bad sizes M=%lld N=%lld K=%lld", M, N, K);
    const long long wide = N > K ? N : K;
    if (M > (1ll << 30) || M > kMostOperand / ((wide + 127) / 128 * 4))
        return api_fail(SAM_ERR_INVALID_ARG, "M=%lld too many rows", M);
    if (N > kMostOperand / ((K + 127) / 128 * 4)) return api_fail(SAM_ERR_INVALID_ARG, "weight N=%lld K=%lld too large", N, K);
    return SAM_OK;
}

sam_status forward_layout(int dtype, int out, long long M, long long N, long long K, Plan* p, Layout* L)
{
    const sam_status st = check_linear(dtype, out, M, N, K);
    if (st != SAM_OK) return st;
    *L = Layout{};
    if (M == 0) return SAM_OK;
    const long long kb = blocks_of(K);
    if (stream4_takes(M, kb)) {
        if (!stream4_rounds(M, kb)) {
            L->take(L->codes, 16ull * M * kb);
            L->take(L->scales, (unsigned long long)M * kb);
        }
        return SAM_OK;
    }
    // The tiles read scales as planes of dwords, X's and a copy of W's; rows
    // that are no whole dwords get zeros behind them. (4096 x 11008 x 4096, the
    // first size N: 107 us, from rows of scales 122. 4096 x 11040 x 4096 with
    // K = 11040 117, with the byte loads that odd rows need there 398.)
    const long long kp = (kb + 3) / 4 * 4;
    if (!plan_auto(M, N, 32 * kp, DT_MX4, p)) return api_fail(SAM_ERR_INTERNAL, "no admissible plan");
    L->take(L->codes, 16ull * M * kp);
    L->take(L->scales, (unsigned long long)scale_rows(M) * kp);
    L->take(L->wscales, (unsigned long long)scale_rows(N) * kp);
    if (p->split > 1) L->take(L->parts, 4ull * p->split * M * N);
    return SAM_OK;
}

// The products copy operands and results whose rows are no whole 16-byte
// pieces, so what they take depends on the strides.
sam_status backward_layout(int dtype, int out, long long M, long long N, long long K, long long lddy, long long lddx, Layout* L)
{
    sam_status st = check_linear(dtype, out, M, N, K);
    if (st != SAM_OK) return st;
    *L = Layout{};
    if (M == 0) return SAM_OK;
    if (lddy < N || lddx < K || lddy > kMostRow || lddx > kMostRow)
        return api_fail(SAM_ERR_INVALID_ARG, "row stride lddy=%lld (rows of %lld) or lddx=%lld (rows of %lld)", lddy, N, lddx, K);
    const long long row = dtype == SAM_F32 ? (K + 3) / 4 * 4 : (K + 7) / 8 * 8;
    L->take(L->w, (unsigned long long)N * row * elem(dtype));
    uint64_t inner = 0;
    if (dtype == SAM_F32) {
        st = sam_gemm_ex_workspace(SAM_F32, SAM_OP_N, SAM_OP_N, M, K, N, lddy, row, lddx, 1.0f, 0.0f, &inner);
    } else {
        st = sam_adapter_gemm_workspace((sam_dtype)dtype, SAM_OP_N, M, K, N, 0, 1, lddy, row, &inner);
    }
    if (st != SAM_OK) return st;
    L->take(L->inner, inner);
    return SAM_OK;
}

// A stride for rows of n values that takes the most: neither n nor whole
// 16-byte pieces.
long long worst_stride(long long n, int es)
{
    const long long ld = (n + 1) * es % 16 ? n + 1 : n + 2;
    return ld > kMostRow ? kMostRow : ld;
}

}  // namespace

extern "C" {

sam_status sam_quantize_mxfp4(sam_dtype dtype, sam_op trans, int64_t rows, int64_t K, const void* X, int64_t ldx,
                              uint8_t* codes, uint8_t* scales, void* stream)
{
    if (trans != SAM_OP_N && trans != SAM_OP_T) return api_fail(SAM_ERR_INVALID_ARG, "trans must be SAM_OP_N or SAM_OP_T");
    const long long lines = trans ? K : rows, line = trans ? rows : K;
    sam_status st = check_tensor(dtype, rows, K, lines, line, ldx);
    if (st != SAM_OK) return st;
    const long long kb = blocks_of(K);
    const int es = elem(dtype);
    const Buf bufs[] = {
        {X, rows ? span(lines, ldx, line, es) : 0, "X", es, false},
        {codes, 16ull * rows * kb, "codes", 16, true},
        {scales, (unsigned long long)rows * kb, "scales", 1, true},
    };
    st = check_buffers(bufs, 3);
    if (st != SAM_OK) return st;
    if (rows == 0) return api_ok();
    st = api_device_check();
    if (st != SAM_OK) return st;
    Quant4Args a{};
    a.x = X;
    a.ldx = lines > 1 ? ldx : line;
    a.rows = rows;
    a.K = (int)K;
    a.kb = (int)kb;
    a.codes = codes;
    a.scales = scales;
    return done(launch_quant4(dtype, trans == SAM_OP_T, a, static_cast<hipStream_t>(stream)));
}

sam_status sam_dequantize_mxfp4(sam_dtype dtype, int64_t rows, int64_t K, const uint8_t* codes, const uint8_t* scales, void* X,
                                int64_t ldx, void* stream)
{
    sam_status st = check_tensor(dtype, rows, K, rows, K, ldx);
    if (st != SAM_OK) return st;
    const long long kb = blocks_of(K);
    const int es = elem(dtype);
    const Buf bufs[] = {
        {codes, 16ull * rows * kb, "codes", 16, false},
        {scales, (unsigned long long)rows * kb, "scales", 1, false},
        {X, span(rows, ldx, K, es), "X", es, true},
    };
    st = check_buffers(bufs, 3);
    if (st != SAM_OK) return st;
    if (rows == 0) return api_ok();
    st = api_device_check();
    if (st != SAM_OK) return st;
    const Dequant4Args a{codes, scales, rows, (int)K, (int)kb, X, rows > 1 ? ldx : K};
    return done(launch_dequant4(dtype, a, static_cast<hipStream_t>(stream)));
}

sam_status sam_linear_mxfp4_workspace(sam_dtype dtype, sam_dtype out, int64_t M, int64_t N, int64_t K, uint64_t* bytes)
{
    if (!bytes) return api_fail(SAM_ERR_INVALID_ARG, "bytes is null");
    Plan p{};
    Layout L;
    const sam_status st = forward_layout(dtype, out, M, N, K, &p, &L);
    if (st != SAM_OK) return st;
    *bytes = L.total;
    return api_ok();
}

sam_status sam_linear_mxfp4(sam_dtype dtype, int64_t M, int64_t N, int64_t K, const void* X, int64_t ldx, const uint8_t* codes,
                            const uint8_t* scales, sam_dtype out, void* Y, int64_t ldy, void* workspace,
                            uint64_t workspace_bytes, void* stream)
{
    Plan p{};
    Layout L;
    sam_status st = forward_layout(dtype, out, M, N, K, &p, &L);
    if (st != SAM_OK) return st;
    if (M == 0) return api_ok();
    if (M > 1 && (ldx < K || ldy < N || ldx > (1ll << 40) || ldy > kMostRow))
        return api_fail(SAM_ERR_INVALID_ARG, "row stride ldx=%lld (rows of %lld) or ldy=%lld (rows of %lld)", (long long)ldx,
                        (long long)K, (long long)ldy, (long long)N);
    const long long kb = blocks_of(K);
    const int es = elem(dtype), eo = elem(out);
    const Buf bufs[] = {
        {X, span(M, ldx, K, es), "X", es, false},
        {codes, 16ull * N * kb, "codes", 16, false},
        {scales, (unsigned long long)N * kb, "scales", 1, false},
        {Y, span(M, ldy, N, eo), "Y", eo, true},
        {workspace, workspace ? L.total : 0, "workspace", 16, true},
    };
    st = check_buffers(bufs, 5);
    if (st != SAM_OK) return st;
    if (L.total && (!workspace || workspace_bytes < L.total))
        return api_fail(SAM_ERR_WORKSPACE, "the call needs %llu workspace bytes, got %llu", L.total,
                        (unsigned long long)(workspace ? workspace_bytes : 0));
    st = api_device_check();
    if (st != SAM_OK) return st;
    char* ws = static_cast<char*>(workspace);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const bool few = stream4_takes(M, kb), rounds = few && L.codes.bytes == 0;
    const long long kp = few ? kb : (kb + 3) / 4 * 4;
    Quant4Args q{};
    q.x = X;
    q.ldx = M > 1 ? ldx : K;
    q.rows = M;
    q.K = (int)K;
    q.kb = (int)kp;
    q.codes = (unsigned char*)ws + L.codes.off;
    q.scales = (unsigned char*)ws + L.scales.off;
    if (!few) {
        q.planes = 1;
        q.from = scales;
        q.to = (unsigned char*)ws + L.wscales.off;
        q.plane_rows = N;
        q.from_kb = (int)kb;
    }
    if (!rounds) {
        const hipError_t e = launch_quant4(dtype, false, q, s);
        if (e != hipSuccess) return done(e);
    }
    if (few) {
        Stream4Args a{};
        a.x = q.x;
        a.ldx = q.ldx;
        if (!rounds) a.xc = q.codes, a.xs = q.scales;
        a.codes = codes;
        a.scales = scales;
        a.M = (int)M;
        a.N = (int)N;
        a.K = (int)K;
        a.kb = (int)kb;
        a.y = Y;
        a.ldy = M > 1 ? ldy : N;
        a.out = out;
        return done(launch_stream4(dtype, a, s));
    }
    GemmArgs g{};
    g.A = q.codes;
    g.sa = q.scales;
    g.B = codes;
    g.sb = q.to;
    g.fmt_a = g.fmt_b = 4;
    g.M = (int)M;
    g.N = (int)N;
    g.K = (int)(32 * kp);
    g.lda = g.K;
    g.ldb = (int)(32 * kb);
    g.k_chunk = p.k_chunk;
    g.split = p.split;
    g.tiles_m = p.tiles_m;
    g.tiles_n = p.tiles_n;
    g.group_m = p.group_m;
    g.xcd_remap = p.xcd_remap;
    g.raster_n = p.raster_n;
    g.part_stride = M * N;
    if (p.split == 1) {
        g.out = static_cast<float*>(Y);
        g.ldc = (int)(M > 1 ? ldy : N);
        return done(launch_tile4(p, g, out, s));
    }
    float* parts = reinterpret_cast<float*>(ws + L.parts.off);
    g.out = parts;
    g.ldc = g.N;
    const hipError_t e = launch_tile4(p, g, SAM_F32, s);
    return done(e != hipSuccess ? e : launch_join4(out, {parts, p.split, Y, M > 1 ? ldy : N, M, (int)N}, s));
}

sam_status sam_linear_mxfp4_backward_workspace(sam_dtype dtype, sam_dtype out, int64_t M, int64_t N, int64_t K, uint64_t* bytes)
{
    if (!bytes) return api_fail(SAM_ERR_INVALID_ARG, "bytes is null");
    sam_status st = check_linear(dtype, out, M, N, K);
    if (st != SAM_OK) return st;
    Layout L;
    st = backward_layout(dtype, out, M, N, K, worst_stride(N, elem(dtype)), worst_stride(K, elem(dtype)), &L);
    if (st != SAM_OK) return st;
    *bytes = L.total;
    return api_ok();
}

sam_status sam_linear_mxfp4_backward_workspace_strided(sam_dtype dtype, sam_dtype out, int64_t M, int64_t N, int64_t K,
                                                       int64_t lddy, int64_t lddx, uint64_t* bytes)
{
    if (!bytes) return api_fail(SAM_ERR_INVALID_ARG, "bytes is null");
    if (M == 1) lddy = N, lddx = K;   // a single row's strides reach nothing
    Layout L;
    const sam_status st = backward_layout(dtype, out, M, N, K, lddy, lddx, &L);
    if (st != SAM_OK) return st;
    *bytes = L.total;
    return api_ok();
}

sam_status sam_linear_mxfp4_backward(sam_dtype dtype, int64_t M, int64_t N, int64_t K, const void* dY, int64_t lddy,
                                     const uint8_t* codes, const uint8_t* scales, sam_dtype out, void* dX, int64_t lddx,
                                     void* workspace, uint64_t workspace_bytes, void* stream)
{
    if (M == 1) lddy = N, lddx = K;
    Layout L;
    sam_status st = backward_layout(dtype, out, M, N, K, lddy, lddx, &L);
    if (st != SAM_OK) return st;
    if (M == 0) return api_ok();
    const long long kb = blocks_of(K);
    const int es = elem(dtype), eo = elem(out);
    const Buf bufs[] = {
        {dY, span(M, lddy, N, es), "dY", 16, false},
        {codes, 16ull * N * kb, "codes", 16, false},
        {scales, (unsigned long long)N * kb, "scales", 1, false},
        {dX, span(M, lddx, K, eo), "dX", 16, true},
        {workspace, workspace ? L.total : 0, "workspace", 16, true},
    };
    st = check_buffers(bufs, 5);
    if (st != SAM_OK) return st;
    if (!workspace || workspace_bytes < L.total)
        return api_fail(SAM_ERR_WORKSPACE, "the call needs %llu workspace bytes, got %llu", L.total,
                        (unsigned long long)(workspace ? workspace_bytes : 0));
    st = api_device_check();
    if (st != SAM_OK) return st;
    char* ws = static_cast<char*>(workspace);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    void* w = ws + L.w.off;
    const long long row = dtype == SAM_F32 ? (K + 3) / 4 * 4 : (K + 7) / 8 * 8;
    const hipError_t e = launch_dequant4(dtype, {codes, scales, N, (int)K, (int)kb, w, row}, s);
    if (e != hipSuccess) return done(e);
    void* inner = L.inner.bytes ? ws + L.inner.off : nullptr;
    if (dtype == SAM_F32)
        return sam_gemm_ex(SAM_F32, SAM_OP_N, SAM_OP_N, M, K, N, 1.0f, dY, lddy, w, row, 0.0f, static_cast<float*>(dX), lddx,
                           inner, L.inner.bytes, stream);
    // The plain projection with results of either type: that of the adapters, of which there are none.
    return sam_adapter_gemm(dtype, SAM_OP_N, M, K, N, 0, 1, dY, lddy, w, row, nullptr, nullptr, nullptr, nullptr, out, dX, lddx,
                            inner, L.inner.bytes, stream);
}

}  // extern "C"
