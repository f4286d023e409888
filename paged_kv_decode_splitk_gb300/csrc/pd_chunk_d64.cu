// pd_chunk_d64.cu -- attention of new tokens for head dims padded to 64 columns.
#include "pd_chunk_launch.cuh"

PD_INSTANTIATE_CHUNK(64, false)
PD_INSTANTIATE_CHUNK(64, true)
