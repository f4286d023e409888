// pd_chunk_d128.cu -- attention of new tokens for head dims padded to 128 columns.
#include "pd_chunk_launch.cuh"

PD_INSTANTIATE_CHUNK(128, false)
PD_INSTANTIATE_CHUNK(128, true)
