// Entry points of the token log probabilities (declared in include/sam.h):
// argument checks before any HIP call, then the launches.
#include "sam_check.h"
#include "sam_tokens.h"

using namespace sam;

namespace {

int elem(int dtype) { return dtype == SAM_F32 ? 4 : 2; }

sam_status check_sizes(int dtype, int64_t rows, int64_t V, int64_t ldz, float T)
{
    if (dtype < SAM_F32 || dtype > SAM_F16) return api_fail(SAM_ERR_INVALID_ARG, "bad dtype %d", dtype);
    if (rows < 0 || V < 1 || V > (1ll << 31) - 65536 || (rows > 1 && (ldz < V || ldz > (1ll << 40))))
        return api_fail(SAM_ERR_INVALID_ARG, "bad sizes rows=%lld V=%lld ldz=%lld", (long long)rows, (long long)V, (long long)ldz);
    // A launch has up to 2^32 threads: workgroups of a row or a strip of one.
    const long long strips = (V + 16383) / 16384;
    if (rows > ((1ll << 22) - 1) / strips) return api_fail(SAM_ERR_INVALID_ARG, "rows=%lld too many", (long long)rows);
    if (!(T >= 0x1p-40f) || !(T <= 0x1p40f))
        return api_fail(SAM_ERR_INVALID_ARG, "temperature must be positive, between 2^-40 and 2^40");
    return SAM_OK;
}

sam_status done(hipError_t e)
{
    return e == hipSuccess ? api_ok() : api_fail(SAM_ERR_LAUNCH, "kernel launch failed: %s", hipGetErrorString(e));
}

}  // namespace

extern "C" {

sam_status sam_token_logprobs_workspace(sam_dtype dtype, int64_t rows, int64_t V, int64_t top, uint64_t* bytes)
{
    if (!bytes) return api_fail(SAM_ERR_INVALID_ARG, "bytes is null");
    const sam_status st = check_sizes(dtype, rows, V, V, 1.0f);
    if (st != SAM_OK) return st;
    if (top < 0 || top > kMaxAlternatives || top > V)
        return api_fail(SAM_ERR_INVALID_ARG, "top=%lld outside 0 .. %d or over V", (long long)top, kMaxAlternatives);
    const int parts = rows > 0 ? tokens_parts(dtype, rows, V, top) : 1;
    *bytes = parts > 1 ? align256(16ull * rows * parts) + align256(4ull * rows) + 8ull * rows * parts * top : 0;
    return api_ok();
}

sam_status sam_token_logprobs(sam_dtype dtype, int64_t rows, int64_t V, int64_t top, const void* logits, int64_t ldz,
                              const int32_t* tokens, float temperature, float* logprob, float* entropy, float* norm,
                              float* top_logprob, int32_t* top_index, void* workspace, uint64_t workspace_bytes, void* stream)
{
    sam_status st = check_sizes(dtype, rows, V, ldz, temperature);
    if (st != SAM_OK) return st;
    uint64_t need = 0;
    st = sam_token_logprobs_workspace(dtype, rows, V, top, &need);
    if (st != SAM_OK) return st;
    const int es = elem(dtype);
    const unsigned long long n = rows > 0 ? rows : 0;
    const Buf bufs[] = {
        {logits, span(rows, ldz, V, es), "logits", es, false},
        {tokens, 4 * n, "tokens", 4, false},
        {logprob, 4 * n, "logprob", 4, true},
        {entropy, 4 * n, "entropy", 4, true},
        {norm, 8 * n, "norm", 4, true},
        {top_logprob, 4 * n * top, "top_logprob", 4, true},
        {top_index, 4 * n * top, "top_index", 4, true},
        {workspace, workspace ? need : 0, "workspace", 16, true},
    };
    st = check_buffers(bufs, sizeof(bufs) / sizeof(bufs[0]));
    if (st != SAM_OK) return st;
    if (need && (!workspace || workspace_bytes < need))
        return api_fail(SAM_ERR_WORKSPACE, "the call needs %llu workspace bytes, got %llu", (unsigned long long)need,
                        (unsigned long long)(workspace ? workspace_bytes : 0));
    if (rows == 0) return api_ok();
    st = api_device_check();
    if (st != SAM_OK) return st;
    TokenArgs a{};
    a.z = logits;
    a.ldz = rows > 1 ? ldz : V;
    a.token = tokens;
    a.rows = rows;
    a.V = (int)V;
    a.top = (int)top;
    a.T = temperature;
    a.inv_hi = (float)(1.0 / temperature);
    a.inv_lo = (float)(1.0 / temperature - a.inv_hi);
    a.scale = (float)(1.4426950408889634074 / temperature);
    a.logprob = logprob;
    a.entropy = entropy;
    a.norm = norm;
    a.top_logprob = top_logprob;
    a.top_index = top_index;
    a.parts = tokens_parts(dtype, rows, V, top);
    if (a.parts > 1) {
        char* ws = static_cast<char*>(workspace);
        a.part = reinterpret_cast<float4*>(ws);
        ws += align256(16ull * rows * a.parts);
        a.z_token = reinterpret_cast<float*>(ws);
        a.list = reinterpret_cast<unsigned long long*>(ws + align256(4ull * rows));
    }
    return done(launch_tokens(dtype, a, static_cast<hipStream_t>(stream)));
}

sam_status sam_token_logprobs_grad(sam_dtype dtype, int64_t rows, int64_t V, const void* logits, int64_t ldz,
                                   const int32_t* tokens, float temperature, const float* norm, const float* entropy,
                                   const float* dlogprob, const float* dentropy, void* grad, int64_t ldg, void* stream)
{
    sam_status st = check_sizes(dtype, rows, V, ldz, temperature);
    if (st != SAM_OK) return st;
    if (rows > 1 && (ldg < V || ldg > (1ll << 40)))
        return api_fail(SAM_ERR_INVALID_ARG, "ldg=%lld is smaller than a row", (long long)ldg);
    if (rows <= 1) ldz = ldg = V;
    const int es = elem(dtype);
    const unsigned long long n = rows > 0 ? rows : 0;
    const bool in_place = grad == logits && ldg == ldz;
    const Buf bufs[] = {
        {logits, span(rows, ldz, V, es), "logits", es, false},
        {tokens, 4 * n, "tokens", 4, false},
        {norm, 8 * n, "norm", 4, false},
        {entropy, dentropy ? 4 * n : 0, "entropy", 4, false},
        {dlogprob, dlogprob ? 4 * n : 0, "dlogprob", 4, false},
        {dentropy, dentropy ? 4 * n : 0, "dentropy", 4, false},
        {grad, span(rows, ldg, V, es), "grad", es, false},
    };
    constexpr int kGrad = 6;
    st = check_buffers(bufs, kGrad + 1);
    if (st != SAM_OK) return st;
    // The gradient may take the logits' place, value for value.
    for (int i = in_place ? 1 : 0; i < kGrad; ++i)
        if (ranges_overlap(grad, bufs[kGrad].bytes, bufs[i].p, bufs[i].bytes))
            return api_fail(SAM_ERR_INVALID_ARG, "grad overlaps %s", bufs[i].name);
    if (rows == 0) return api_ok();
    st = api_device_check();
    if (st != SAM_OK) return st;
    TokenGradArgs a{};
    a.z = logits;
    a.ldz = ldz;
    a.token = tokens;
    a.rows = rows;
    a.V = (int)V;
    a.T = temperature;
    a.inv = (float)(1.0 / temperature);
    a.scale = (float)(1.4426950408889634074 / temperature);
    a.norm = norm;
    a.entropy = entropy;
    a.u = dlogprob;
    a.v = dentropy;
    a.grad = grad;
    a.ldg = ldg;
    return done(launch_tokens_grad(dtype, a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
