// pd_prefix_d256.cu -- the shared-prefix pass for head dims padded to 256 columns.
#include "pd_prefix_launch.cuh"

PD_INSTANTIATE_PREFIX(256, false)
PD_INSTANTIATE_PREFIX(256, true)
