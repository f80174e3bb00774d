// The 4-bit projection of many rows: the E2M1 form of the block-scaled
// variants (sam_mx8.h), with results stored in their own type and stride.
#include "sam_mx8.h"
#include "sam_mxfp4.h"
#include "sam_variants.h"

namespace sam {

namespace {

using namespace mx8;

typedef void (*KernelFn)(GemmArgs);

struct Form {
    int id, threads;
    KernelFn fn[3];   // by the type of the result
};

#define SAM_TILE4(BM, BN, WM, WN, BK, SD)                                                                           \
    {gemm_mx8_kernel<4, 4, BM, BN, WM, WN, 2 * BK, SD, 4, DT_F32>, gemm_mx8_kernel<4, 4, BM, BN, WM, WN, 2 * BK, SD, 4, DT_BF16>, \
     gemm_mx8_kernel<4, 4, BM, BN, WM, WN, 2 * BK, SD, 4, DT_F16>}
#define SAM_TILE4_ENTRY(id, name, BM, BN, WM, WN, BK, SD, gm, xr, ms, e8, e4)                                       \
    {id, WM * WN * 64, SAM_TILE4(BM, BN, WM, WN, BK, SD != 0)},

const Form kForms[] = {SAM_MX8_VARIANTS(SAM_TILE4_ENTRY)};

}  // namespace

// K is a multiple of 128: scales come as planes of dwords.
hipError_t launch_tile4(const Plan& p, const GemmArgs& a, int out, hipStream_t s)
{
    for (const Form& f : kForms) {
        if (f.id != p.variant_id) continue;
        hipLaunchKernelGGL(f.fn[out], dim3((unsigned)p.grid), dim3(f.threads), 0, s, a);
        return hipGetLastError();
    }
    return hipErrorInvalidDeviceFunction;
}

}  // namespace sam
