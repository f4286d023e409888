// pd_prefix_d64.cu -- the shared-prefix pass for head dims padded to 64 columns.
#include "pd_prefix_launch.cuh"

PD_INSTANTIATE_PREFIX(64, false)
PD_INSTANTIATE_PREFIX(64, true)
