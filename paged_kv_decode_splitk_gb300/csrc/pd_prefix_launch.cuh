// pd_prefix_launch.cuh -- host launcher of the shared-prefix pass, included by
// the translation units that instantiate it.
#pragma once

#include <cstring>
#include <mutex>

#include "pd_prefix.cuh"

namespace pd {
namespace prefix {

template <int DPAD, bool KV8, bool MULTI>
cudaError_t launch_prefix_as(const CUtensorMap *tk, const CUtensorMap *tv, const PrefixParams &p, int teams,
                             cudaStream_t stream) {
    auto kern = prefix_kernel<DPAD, KV8, MULTI>;
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
    cfg.gridDim = dim3(static_cast<unsigned>(2 * teams));
    cfg.blockDim = dim3(Plan<DPAD, KV8>::kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    // A cluster only puts a team's two CTAs on neighbouring SMs (they exchange nothing),
    // which leaves whole neighbours to the own-token pass: 256 sequences behind 32768
    // tokens with own ones 127 us, 145 without.
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    KvMaps<1> maps;
    maps.k[0] = *tk;
    maps.v[0] = *tv;
    return cudaLaunchKernelEx(&cfg, kern, maps, p);
}

template <int DPAD, bool KV8>
cudaError_t launch_prefix(const CUtensorMap *tk, const CUtensorMap *tv, const PrefixParams &p, int teams,
                          cudaStream_t stream) {
    return p.num_groups > 1 ? launch_prefix_as<DPAD, KV8, true>(tk, tv, p, teams, stream)
                            : launch_prefix_as<DPAD, KV8, false>(tk, tv, p, teams, stream);
}

}  // namespace prefix
}  // namespace pd

#define PD_INSTANTIATE_PREFIX(DPAD, KV8)                                                                     \
    template cudaError_t pd::prefix::launch_prefix<DPAD, KV8>(const CUtensorMap *, const CUtensorMap *,      \
                                                              const pd::prefix::PrefixParams &, int, cudaStream_t);
