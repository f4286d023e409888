// pd_unit_own_d256.cu -- unit kernels of pd_decode_attn_prefix's own-token pass,
// head dims padded to 256 columns, over BF16 and FP8 caches.
#include "pd_unit_launch.cuh"

PD_INSTANTIATE_UNIT(256, 1, true, pd::kModeOwn, false, false)
PD_INSTANTIATE_UNIT(256, 1, false, pd::kModeOwn, false, false)
PD_INSTANTIATE_UNIT(256, 2, false, pd::kModeOwn, false, false)
PD_INSTANTIATE_UNIT(256, 1, true, pd::kModeOwn, false, true)
PD_INSTANTIATE_UNIT(256, 1, false, pd::kModeOwn, false, true)
PD_INSTANTIATE_UNIT(256, 2, false, pd::kModeOwn, false, true)
