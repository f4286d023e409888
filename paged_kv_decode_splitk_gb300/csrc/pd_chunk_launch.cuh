// pd_chunk_launch.cuh -- host launcher of the kernel of pd_chunk_attn, included by
// the translation units that instantiate it.
#pragma once

#include <mutex>

#include "pd_chunk.cuh"

namespace pd {
namespace chunk {

template <int DPAD, bool KV8>
cudaError_t launch_chunk(const CUtensorMap *tk, const CUtensorMap *tv, const CUtensorMap *tq, const ChunkParams &p, int ctas,
                         cudaStream_t stream) {
    auto kern = chunk_kernel<DPAD, KV8>;
    static std::mutex mu;
    static bool configured[64] = {false};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    constexpr int smem = Plan<DPAD, KV8>::total;
    static_assert(smem <= 227 * 1024, "shared memory of a CTA");
    {
        std::lock_guard<std::mutex> lock(mu);
        if (!configured[dev]) {
            e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
            if (e != cudaSuccess) return e;
            configured[dev] = true;
        }
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(Plan<DPAD, KV8>::kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    ChunkMaps maps;
    maps.k = *tk;
    maps.v = *tv;
    maps.q = *tq;
    return cudaLaunchKernelEx(&cfg, kern, maps, p);
}

}  // namespace chunk
}  // namespace pd

#define PD_INSTANTIATE_CHUNK(DPAD, KV8)                                                                             \
    template cudaError_t pd::chunk::launch_chunk<DPAD, KV8>(const CUtensorMap *, const CUtensorMap *, const CUtensorMap *, \
                                                            const pd::chunk::ChunkParams &, int, cudaStream_t);
