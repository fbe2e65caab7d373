// attend_mx8_kernels.hip -- the attention kernels of a cache of 8-bit codes (gfx950).
#include "attend_items.h"

namespace moe {

#define ATTEND_KERNELS(D)                                                                \
    template __global__ void moe_attend_kernel<false, D, 1, 1, MX_E4M3, true>(AttendParams); \
    template __global__ void moe_attend_kernel<false, D, 2, 1, MX_E4M3, true>(AttendParams); \
    template __global__ void moe_attend_kernel<false, D, 2, 2, MX_E4M3, true>(AttendParams); \
    template __global__ void moe_attend_kernel<false, D, 2, 4, MX_E4M3, true>(AttendParams); \
    template __global__ void moe_attend_kernel<true, D, 1, 1, MX_E4M3, true>(AttendParams);  \
    template __global__ void moe_attend_kernel<true, D, 2, 1, MX_E4M3, true>(AttendParams);  \
    template __global__ void moe_attend_kernel<true, D, 2, 2, MX_E4M3, true>(AttendParams);  \
    template __global__ void moe_attend_kernel<true, D, 2, 4, MX_E4M3, true>(AttendParams)
ATTEND_KERNELS(32);
ATTEND_KERNELS(64);
ATTEND_KERNELS(96);
ATTEND_KERNELS(128);
ATTEND_KERNELS(192);
ATTEND_KERNELS(256);

}  // namespace moe
