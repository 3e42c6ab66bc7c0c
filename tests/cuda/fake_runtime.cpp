// fake_runtime.cpp -- the CUDA runtime functions and library services that the
// attention layer's entry points call, as recorders: no GPU is needed, no
// pointer is followed, and a chosen launch can be refused.
#include <cstdint>
#include <cstring>
#include <map>
#include <string>
#include <vector>

#include <cuda.h>
#include <cuda_runtime.h>

#include "host.h"
#include "nvfp4.h"

namespace {

std::map<const void *, std::string> &names()
{
    static std::map<const void *, std::string> m;
    return m;
}

std::vector<std::string> launched;
int refuse = -1;  // launch that fails, counted from the last reset
int counted = 0;
cudaError_t last_error = cudaSuccess;

CUresult encode(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill)
{
    return CUDA_SUCCESS;
}

cudaError_t record(const void *fn)
{
    const int k = static_cast<int>(launched.size());
    launched.push_back(names().count(fn) ? names()[fn] : "?");
    last_error = k == refuse ? cudaErrorLaunchOutOfResources : cudaSuccess;
    return last_error;
}

}  // namespace

extern "C" {

void fake_reset(int refuse_launch)
{
    launched.clear();
    refuse = refuse_launch;
    counted = 0;
    last_error = cudaSuccess;
}
int fake_launches() { return static_cast<int>(launched.size()); }
int fake_counted() { return counted; }
const char *fake_name(int i) { return launched[i].c_str(); }

void **__cudaRegisterFatBinary(void *)
{
    static void *handle;
    return &handle;
}
void __cudaRegisterFatBinaryEnd(void **) {}
void __cudaUnregisterFatBinary(void **) {}
char __cudaInitModule(void **) { return 0; }
void __cudaRegisterFunction(void **, const char *host, char *, const char *name, int, uint3 *, uint3 *, dim3 *, dim3 *, int *)
{
    names()[host] = name;
}
unsigned __cudaPopCallConfiguration(dim3 *, dim3 *, size_t *, void *) { return 0; }
cudaError_t cudaFuncSetAttribute(const void *, cudaFuncAttribute, int) { return cudaSuccess; }
cudaError_t cudaGetLastError()
{
    const cudaError_t e = last_error;
    last_error = cudaSuccess;
    return e;
}
cudaError_t cudaLaunchKernel(const void *fn, dim3, dim3, void **, size_t, cudaStream_t) { return record(fn); }
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t *, const void *fn, void **) { return record(fn); }

}  // extern "C"

namespace nvfp4 {
namespace host {

int device(Device *out)
{
    static uint32_t status;
    out->index = 0;
    out->sm_count = 148;
    out->status = &status;
    out->encode_tiled = encode;
    return NVFP4_OK;
}
void count_launch() { ++counted; }
int clear_words(uint32_t *, int, cudaStream_t) { return NVFP4_OK; }

}  // namespace host
}  // namespace nvfp4
