// pd_chunk_d256.cu -- attention of new tokens for head dims padded to 256 columns.
#include "pd_chunk_launch.cuh"

PD_INSTANTIATE_CHUNK(256, false)
PD_INSTANTIATE_CHUNK(256, true)
