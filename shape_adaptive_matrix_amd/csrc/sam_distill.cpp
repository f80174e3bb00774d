// Entry points of the distillation loss (declared in include/sam.h): argument
// checks before any HIP call, then one launch each.
#include <math.h>

#include "sam_check.h"
#include "sam_distill.h"

using namespace sam;

namespace {

int elem(int dtype) { return dtype == SAM_F32 ? 4 : 2; }

bool aligned_to(const void* p, int n) { return (unsigned long long)p % (unsigned)n == 0; }

struct Buf {
    const void* p;
    unsigned long long bytes;
    const char* name;
    int align;
    bool written;
};

sam_status check(int dtype, int64_t rows, int64_t V, int64_t top, int64_t ldz, int t_dtype, float T, const Buf* b, int n)
{
    for (int t : {dtype, t_dtype})
        if (t < SAM_F32 || t > SAM_F16) return api_fail(SAM_ERR_INVALID_ARG, "bad dtype %d", t);
    if (rows < 0 || V < 1 || V > (1ll << 31) - 65536 || top < 1 || top > kMaxTop || ldz < V || ldz > (1ll << 40))
        return api_fail(SAM_ERR_INVALID_ARG, "bad sizes rows=%lld V=%lld top=%lld (1 .. %d) ldz=%lld", (long long)rows,
                        (long long)V, (long long)top, kMaxTop, (long long)ldz);
    const long long strips = (V + 16383) / 16384;
    if (rows > ((1ll << 31) - 1) / strips) return api_fail(SAM_ERR_INVALID_ARG, "rows=%lld too many", (long long)rows);
    // Within these 1 / T, T^2 and their products with the other factors are ordinary numbers.
    if (!(T >= 0x1p-40f) || !(T <= 0x1p40f))
        return api_fail(SAM_ERR_INVALID_ARG, "temperature must be positive, between 2^-40 and 2^40");
    for (int i = 0; i < n; ++i) {
        if (b[i].bytes && !b[i].p) return api_fail(SAM_ERR_INVALID_ARG, "%s is null", b[i].name);
        if (b[i].bytes && !aligned_to(b[i].p, b[i].align))
            return api_fail(SAM_ERR_MISALIGNED, "%s must be %d-byte aligned", b[i].name, b[i].align);
    }
    for (int i = 0; i < n; ++i)
        for (int j = 0; j < n; ++j)
            if (i != j && b[i].written && ranges_overlap(b[i].p, b[i].bytes, b[j].p, b[j].bytes))
                return api_fail(SAM_ERR_INVALID_ARG, "%s overlaps %s", b[i].name, b[j].name);
    return SAM_OK;
}

unsigned long long span(int64_t rows, int64_t ld, int64_t cols, int es)
{
    return rows > 0 ? ((unsigned long long)(rows - 1) * ld + cols) * es : 0;
}

DistillArgs arguments(int64_t rows, int64_t V, int64_t top, const void* z, int64_t ldz, int t_dtype, const void* t,
                      const int32_t* index, const float* weight, float T)
{
    DistillArgs a{};
    a.z = z;
    a.ldz = ldz;
    a.t = t;
    a.index = index;
    a.weight = weight;
    a.rows = rows;
    a.V = (int)V;
    a.top = (int)top;
    a.t_dtype = t_dtype;
    a.T = T;
    a.inv_hi = (float)(1.0 / T);
    a.inv_lo = (float)(1.0 / T - a.inv_hi);
    a.scale = (float)(1.4426950408889634074 / T);
    return a;
}

sam_status done(hipError_t e)
{
    return e == hipSuccess ? api_ok() : api_fail(SAM_ERR_LAUNCH, "kernel launch failed: %s", hipGetErrorString(e));
}

// The gradient may take the logits' place, value for value; otherwise the
// two may not overlap.
sam_status check_grad(const void* z, int64_t ldz, const void* grad, int64_t ldg, int64_t rows, int64_t V, int es)
{
    if (ldg < V || ldg > (1ll << 40)) return api_fail(SAM_ERR_INVALID_ARG, "ldg=%lld is smaller than a row", (long long)ldg);
    if (grad == z && ldg == ldz) return SAM_OK;
    if (ranges_overlap(grad, span(rows, ldg, V, es), z, span(rows, ldz, V, es)))
        return api_fail(SAM_ERR_INVALID_ARG, "grad overlaps the logits without being in their place");
    return SAM_OK;
}

}  // namespace

extern "C" {

static sam_status distill(sam_dtype dtype, int64_t rows, int64_t V, int64_t top, const void* logits, int64_t ldz,
                          sam_dtype t_dtype, const void* t, const int32_t* index, const float* weight, float T,
                          float* loss, float* lse, bool want_grad, void* grad, int64_t ldg, void* stream)
{
    const int es = elem(dtype);
    const Buf bufs[] = {
        {logits, span(rows, ldz, V, es), "logits", es, false},
        {t, (unsigned long long)(rows * top) * elem(t_dtype), "teacher", elem(t_dtype), false},
        {index, 4ull * rows * top, "index", 4, false},
        {weight, weight ? 4ull * rows : 0, "weight", 4, false},
        {loss, 4ull * rows, "loss", 4, true},
        {lse, want_grad ? 0 : 4ull * rows, "lse", 4, true},
    };
    sam_status st = check(dtype, rows, V, top, ldz, t_dtype, T, bufs, sizeof(bufs) / sizeof(bufs[0]));
    if (st != SAM_OK) return st;
    if (want_grad) {
        if (rows && !grad) return api_fail(SAM_ERR_INVALID_ARG, "grad is null");
        if (rows && !aligned_to(grad, es)) return api_fail(SAM_ERR_MISALIGNED, "grad must be %d-byte aligned", es);
        st = check_grad(logits, ldz, grad, ldg, rows, V, es);
        if (st != SAM_OK) return st;
        for (const Buf& b : bufs)
            if (b.p != logits && ranges_overlap(grad, span(rows, ldg, V, es), b.p, b.bytes))
                return api_fail(SAM_ERR_INVALID_ARG, "grad overlaps %s", b.name);
    }
    if (rows == 0) return api_ok();
    st = api_device_check();
    if (st != SAM_OK) return st;
    DistillArgs a = arguments(rows, V, top, logits, ldz, t_dtype, t, index, weight, T);
    a.loss = loss;
    a.lse = lse;
    a.grad = grad;
    a.ldg = ldg;
    return done(launch_distill(dtype, a, static_cast<hipStream_t>(stream)));
}

sam_status sam_distill_loss(sam_dtype dtype, int64_t rows, int64_t V, int64_t top, const void* logits, int64_t ldz,
                            sam_dtype t_dtype, const void* teacher, const int32_t* index, const float* weight,
                            float temperature, float* loss, float* lse, void* stream)
{
    return distill(dtype, rows, V, top, logits, ldz, t_dtype, teacher, index, weight, temperature, loss, lse, false,
                   nullptr, 0, stream);
}

sam_status sam_distill(sam_dtype dtype, int64_t rows, int64_t V, int64_t top, const void* logits, int64_t ldz,
                       sam_dtype t_dtype, const void* teacher, const int32_t* index, const float* weight,
                       float temperature, float* loss, void* grad, int64_t ldg, void* stream)
{
    return distill(dtype, rows, V, top, logits, ldz, t_dtype, teacher, index, weight, temperature, loss, nullptr, true,
                   grad, ldg, stream);
}

sam_status sam_distill_grad(sam_dtype dtype, int64_t rows, int64_t V, int64_t top, const void* logits, int64_t ldz,
                            const float* lse, sam_dtype t_dtype, const void* teacher, const int32_t* index,
                            const float* weight, float temperature, void* grad, int64_t ldg, void* stream)
{
    const int es = elem(dtype);
    const Buf bufs[] = {
        {logits, span(rows, ldz, V, es), "logits", es, false},
        {teacher, (unsigned long long)(rows * top) * elem(t_dtype), "teacher", elem(t_dtype), false},
        {index, 4ull * rows * top, "index", 4, false},
        {weight, weight ? 4ull * rows : 0, "weight", 4, false},
        {lse, 4ull * rows, "lse", 4, false},
        {grad, span(rows, ldg, V, es), "grad", es, false},
    };
    sam_status st = check(dtype, rows, V, top, ldz, t_dtype, temperature, bufs, sizeof(bufs) / sizeof(bufs[0]));
    if (st != SAM_OK) return st;
    st = check_grad(logits, ldz, grad, ldg, rows, V, es);
    if (st != SAM_OK) return st;
    for (int i = 1; i < 5; ++i)
        if (ranges_overlap(grad, span(rows, ldg, V, es), bufs[i].p, bufs[i].bytes))
            return api_fail(SAM_ERR_INVALID_ARG, "grad overlaps %s", bufs[i].name);
    if (rows == 0) return api_ok();
    st = api_device_check();
    if (st != SAM_OK) return st;
    DistillArgs a = arguments(rows, V, top, logits, ldz, t_dtype, teacher, index, weight, temperature);
    a.lse = const_cast<float*>(lse);
    a.grad = grad;
    a.ldg = ldg;
    return done(launch_distill_grad(dtype, a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
