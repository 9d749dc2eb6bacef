// The HIP launches of the attention block's operators.
#include <hip/hip_runtime.h>

#include "ua2a_attn_internal.h"

namespace ua2a {

// The kernel of a launch; null where none is built for it.
const void* attention_kernel(const AttnLaunch& L);
const void* decode_kernel(const AttnLaunch& L);
const void* attention_grad_kernel(const AttnLaunch& L);
const void* rope_kernel(const AttnLaunch& L);

int attn_launch(const AttnLaunch& L, void* stream)
{
    const void* fn = nullptr;
    void* args[1] = {nullptr};
    switch (L.kernel) {
    case AttnKernel::Rope:
        fn = rope_kernel(L);
        args[0] = const_cast<RopeArgs*>(&L.rope);
        break;
    case AttnKernel::Decode:
        fn = decode_kernel(L);
        args[0] = const_cast<AttnArgs*>(&L.attn);
        break;
    case AttnKernel::Forward:
    case AttnKernel::Join:
        fn = attention_kernel(L);
        args[0] = const_cast<AttnArgs*>(&L.attn);
        break;
    case AttnKernel::GradRows:
    case AttnKernel::GradKeys:
    case AttnKernel::GradJoin:
        fn = attention_grad_kernel(L);
        args[0] = const_cast<AttnGradArgs*>(&L.grad);
        break;
    }
    if (fn == nullptr) return static_cast<int>(hipErrorInvalidValue);
    const hipError_t e = hipLaunchKernel(fn, dim3(L.grid_x, L.grid_y, 1), dim3(L.block), args, 0,
                                         static_cast<hipStream_t>(stream));
    return e == hipSuccess ? 0 : static_cast<int>(e);
}

}  // namespace ua2a
