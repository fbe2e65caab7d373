// attend_kernels.hip -- the attention kernels of a cache in the queries' own 16-bit type (gfx950), and the launches that join
// parts, which are the same for every format.
#include "attend_items.h"

namespace moe {

#define ATTEND_KERNELS(D)                                                                 \
    template __global__ void moe_attend_kernel<false, D, 1, 1, MX_NONE, false>(AttendParams); \
    template __global__ void moe_attend_kernel<false, D, 2, 1, MX_NONE, false>(AttendParams); \
    template __global__ void moe_attend_kernel<false, D, 2, 2, MX_NONE, false>(AttendParams); \
    template __global__ void moe_attend_kernel<false, D, 2, 4, MX_NONE, false>(AttendParams); \
    template __global__ void moe_attend_kernel<true, D, 1, 1, MX_NONE, false>(AttendParams);  \
    template __global__ void moe_attend_kernel<true, D, 2, 1, MX_NONE, false>(AttendParams);  \
    template __global__ void moe_attend_kernel<true, D, 2, 2, MX_NONE, false>(AttendParams);  \
    template __global__ void moe_attend_kernel<true, D, 2, 4, MX_NONE, false>(AttendParams);  \
    template __global__ void moe_attend_join_kernel<false, D>(AttendParams);              \
    template __global__ void moe_attend_join_kernel<true, D>(AttendParams);               \
    template __global__ void moe_shared_join_kernel<false, D>(SharedJoinParams);          \
    template __global__ void moe_shared_join_kernel<true, D>(SharedJoinParams)
ATTEND_KERNELS(32);
ATTEND_KERNELS(64);
ATTEND_KERNELS(80);
ATTEND_KERNELS(96);
ATTEND_KERNELS(112);
ATTEND_KERNELS(128);
ATTEND_KERNELS(192);
ATTEND_KERNELS(256);

}  // namespace moe
