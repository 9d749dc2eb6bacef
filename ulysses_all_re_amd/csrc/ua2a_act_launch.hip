// The HIP launches of the activation operators.
#include <hip/hip_runtime.h>

#include "ua2a_act_internal.h"

namespace ua2a {

// The kernel of a launch; null where none is built for it.
const void* norm_kernel(const ActLaunch& L);
const void* norm_grad_kernel(const ActLaunch& L);
const void* columns_kernel();
const void* cache_kernel(const ActLaunch& L);

int act_launch(const ActLaunch& L, void* stream)
{
    const void* fn = nullptr;
    void* args[1] = {nullptr};
    switch (L.kernel) {
    case ActKernel::Norm:
        fn = norm_kernel(L);
        args[0] = const_cast<NormArgs*>(&L.norm);
        break;
    case ActKernel::NormGrad:
        fn = norm_grad_kernel(L);
        args[0] = const_cast<NormGradArgs*>(&L.grad);
        break;
    case ActKernel::Columns:
        fn = columns_kernel();
        args[0] = const_cast<ColumnArgs*>(&L.columns);
        break;
    case ActKernel::CacheWrite:
    case ActKernel::CacheRead:
        fn = cache_kernel(L);
        args[0] = const_cast<CacheArgs*>(&L.cache);
        break;
    }
    if (fn == nullptr) return static_cast<int>(hipErrorInvalidValue);
    const hipError_t e = hipLaunchKernel(fn, dim3(L.grid_x, L.grid_y, 1), dim3(L.block), args, 0,
                                         static_cast<hipStream_t>(stream));
    return e == hipSuccess ? 0 : static_cast<int>(e);
}

}  // namespace ua2a
