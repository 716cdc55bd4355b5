// ds_host.cuh -- host-side helpers shared by the library's translation units.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "ds_topk.h"

namespace dsk {

struct DevInfo {
    int sms = 0;
    int smem_optin = 0;
    int smem_per_sm = 0;
    bool ok = false;
};

// Properties of device `dev`, looked up once per device (defined in ds_topk.cu).
bool dev_info(int dev, DevInfo& out);

// The library-owned workspace of (device, stream, kind), zeroed when allocated and grown to
// at least `bytes` (defined in ds_topk.cu).  Calls on one stream are ordered and share it.
// Kinds are kept apart because the top-k's threshold words are told from stale ones by a call
// number, which another operator's data could imitate.
enum WsKind : int { kWsTopk = 0, kWsAttend = 1 };
ds_status library_workspace(int dev, WsKind kind, size_t bytes, cudaStream_t stream, void** out);

// The current device's status word, for kernels that record a wait that ran out (defined in
// ds_topk.cu); null on a CUDA error.
uint32_t* status_word();

// Launches `kern` so that it may begin while the stream's previous kernel ends
// (programmatic dependent launch): the kernel waits for its predecessor (pdl_wait) before
// it touches global memory.  `cluster` > 1 sets the thread-block cluster's size.
template <typename Kern, typename... Args>
inline ds_status launch_pdl(Kern kern, dim3 grid, int threads, size_t smem, int cluster, cudaStream_t stream,
                            Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    int na = 0;
    attr[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[na].val.programmaticStreamSerializationAllowed = 1;
    ++na;
    if (cluster > 1) {
        attr[na].id = cudaLaunchAttributeClusterDimension;
        attr[na].val.clusterDim.x = cluster;
        attr[na].val.clusterDim.y = 1;
        attr[na].val.clusterDim.z = 1;
        ++na;
    }
    cfg.attrs = attr;
    cfg.numAttrs = na;
    return cudaLaunchKernelEx(&cfg, kern, args...) == cudaSuccess ? DS_OK : DS_ERR_CUDA;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace dsk
