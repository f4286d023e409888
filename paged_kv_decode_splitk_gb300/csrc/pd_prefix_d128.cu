// pd_prefix_d128.cu -- the shared-prefix pass for head dims padded to 128 columns.
#include "pd_prefix_launch.cuh"

PD_INSTANTIATE_PREFIX(128, false)
PD_INSTANTIATE_PREFIX(128, true)
