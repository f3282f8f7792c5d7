// dgq_attn_window.cu -- instances of the decode kernel (dgq_attn_kernel.cuh) for 8-bit caches with a scale
// per block and head, and for attention that sees a window of the last tokens and a few first ones
// (sm_103a).
#include "dgq_attn_kernel.cuh"

namespace dgq {

AttnKernel attn_window_kernel(int dec, bool win)
{
    switch (dec) {
    case kDecBlockI8: return win ? attn_kernel<kDecBlockI8, true> : attn_kernel<kDecBlockI8, false>;
    case kDecBlockE4: return win ? attn_kernel<kDecBlockE4, true> : attn_kernel<kDecBlockE4, false>;
    case kDecBf16: return win ? attn_kernel<kDecBf16, true> : nullptr;
    case kDecAffine: return win ? attn_kernel<kDecAffine, true> : nullptr;
    }
    return nullptr;
}

}  // namespace dgq
