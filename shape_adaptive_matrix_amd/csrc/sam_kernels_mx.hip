// Block-scaled variants (sam_mx8.h) with FP32 results, and their launch.
#include "sam_mx8.h"
#include "sam_variants.h"

namespace sam {

namespace {

using namespace mx8;

typedef void (*KernelFn)(GemmArgs);

struct Mx8Kernels {
    int id;
    KernelFn fn[2][2][2];   // 8-bit: [scales through LDS][format of A][format of B]: 0 E4M3, 1 E5M2
    KernelFn fn4[2];        // E2M1: [scales through LDS]
    int threads;
};

#define SAM_MX8_FORMS(BM, BN, WM, WN, BK, SD)                                                                   \
    {{gemm_mx8_kernel<0, 0, BM, BN, WM, WN, BK, SD, 8>, gemm_mx8_kernel<0, 1, BM, BN, WM, WN, BK, SD, 8>},      \
     {gemm_mx8_kernel<1, 0, BM, BN, WM, WN, BK, SD, 8>, gemm_mx8_kernel<1, 1, BM, BN, WM, WN, BK, SD, 8>}}
// The E2M1 form runs twice the values of K per stage (same 128-byte rows).
#define SAM_MX8_ENTRY(id, name, BM, BN, WM, WN, BK, SD, gm, xr, ms, e8, e4)                                  \
    {id, {SAM_MX8_FORMS(BM, BN, WM, WN, BK, false), SAM_MX8_FORMS(BM, BN, WM, WN, BK, SD != 0)},               \
     {gemm_mx8_kernel<4, 4, BM, BN, WM, WN, 2 * BK, false, 4>, gemm_mx8_kernel<4, 4, BM, BN, WM, WN, 2 * BK, SD != 0, 4>}, \
     WM * WN * 64},

const Mx8Kernels kMx8Table[] = {SAM_MX8_VARIANTS(SAM_MX8_ENTRY)};

}  // namespace

hipError_t launch_mx8(const Plan& p, const GemmArgs& a, hipStream_t s)
{
    const bool fp4 = p.dtype == DT_MX4;
    if (!fp4 && (a.fmt_a < 0 || a.fmt_a > 1 || a.fmt_b < 0 || a.fmt_b > 1)) return hipErrorInvalidValue;
    for (const Mx8Kernels& d : kMx8Table) {
        if (d.id != p.variant_id) continue;
        // The scale dwords are 4-byte aligned when K % 128 == 0.
        const int sd = a.K % 128 == 0;
        KernelFn fn = fp4 ? d.fn4[sd] : d.fn[sd][a.fmt_a][a.fmt_b];
        hipLaunchKernelGGL(fn, dim3((unsigned)p.grid), dim3(d.threads), 0, s, a);
        return hipGetLastError();
    }
    return hipErrorInvalidDeviceFunction;
}

}  // namespace sam
