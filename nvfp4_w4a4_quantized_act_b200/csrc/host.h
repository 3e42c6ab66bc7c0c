// host.h -- host-side services shared by the library's translation units:
// kernel launches, launch accounting and the per-device state.
#pragma once

#include <cstdint>
#include <cstring>

#include <cuda.h>
#include <cuda_runtime.h>

namespace nvfp4 {
namespace host {

inline bool &launch_failed_flag()
{
    static thread_local bool failed = false;
    return failed;
}

// Launches a kernel with programmatic stream serialization: the kernel may
// be scheduled while the previous kernel on the stream is still running and
// waits for it (griddepcontrol.wait) before touching global memory.  Every
// kernel of this library does that wait first, so stream order holds.
template <typename... KArgs, typename... Args>
void launch(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, Args... args)
{
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kernel, args...) != cudaSuccess)
        launch_failed_flag() = true;
}

// Whether a launch of this thread failed since the last call.
inline bool launch_failed()
{
    const bool failed = launch_failed_flag();
    launch_failed_flag() = false;
    return (cudaGetLastError() != cudaSuccess) || failed;
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

struct Device {
    int index;
    int sm_count;
    uint32_t *status;  // device address of the status word
    EncodeTiledFn encode_tiled;
};

// The current device (NVFP4_OK, NVFP4_ERR_CUDA or NVFP4_ERR_NO_DEVICE).
int device(Device *out);

// Counts one launch for nvfp4_launch_count().
void count_launch();

// Clears `n` words on the stream (one counted launch).
int clear_words(uint32_t *words, int n, cudaStream_t stream);

}  // namespace host
}  // namespace nvfp4
