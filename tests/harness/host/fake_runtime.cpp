// fake_runtime.cpp -- a CUDA runtime without a device for host tests of the entry points
// (linked with --cudart none): launches succeed or fail as told, the last error behaves as
// the runtime's, attributes and launches are recorded.

#include <cuda_runtime.h>

#include <cstring>
#include <map>
#include <mutex>
#include <set>

namespace {

std::mutex mu;
std::map<const void *, std::set<int>> limits;  // dynamic shared memory limits each kernel was given
std::map<const void *, int> limit;             // the present one
int launches = 0;
thread_local cudaError_t last = cudaSuccess;
thread_local int fail_in = 0;  // the launch that will fail, counted from 1; 0: none
thread_local struct {
    dim3 grid, block;
    size_t smem;
    cudaStream_t stream;
} config;

cudaError_t launched(const void *kernel, size_t smem)
{
    std::lock_guard<std::mutex> lock(mu);
    const auto at = limit.find(kernel);
    const size_t most = at == limit.end() ? 48 * 1024 : (size_t)at->second;
    if ((fail_in > 0 && --fail_in == 0) || smem > most) return last = cudaErrorInvalidValue;
    ++launches;
    return cudaSuccess;
}

}  // namespace

extern "C" {

// what the tests ask
void fake_fail_in(int n) { fail_in = n; }
int fake_last_error() { return (int)last; }
int fake_launches() { return launches; }
int fake_most_limits()  // the most different limits that one kernel was given
{
    std::lock_guard<std::mutex> lock(mu);
    size_t most = 0;
    for (const auto &k : limits)
        if (k.second.size() > most) most = k.second.size();
    return (int)most;
}

// the runtime
cudaError_t cudaGetLastError()
{
    const cudaError_t e = last;
    last = cudaSuccess;
    return e;
}
cudaError_t cudaPeekAtLastError() { return last; }
const char *cudaGetErrorString(cudaError_t) { return "fake"; }
cudaError_t cudaFuncSetAttribute(const void *f, cudaFuncAttribute, int value)
{
    std::lock_guard<std::mutex> lock(mu);
    limits[f].insert(value);
    limit[f] = value;
    return cudaSuccess;
}
cudaError_t __cudaGetKernel(cudaKernel_t *kernel, const void *f)  // a kernel's handle: its host function
{
    *kernel = (cudaKernel_t)f;
    return cudaSuccess;
}
cudaError_t __cudaLaunchKernel(cudaKernel_t f, dim3, dim3, void **, size_t smem, cudaStream_t)
{
    return launched((const void *)f, smem);
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t *c, const void *f, void **)
{
    return launched(f, c->dynamicSmemBytes);
}
cudaError_t cudaGetDevice(int *d)
{
    *d = 0;
    return cudaSuccess;
}
cudaError_t cudaDeviceGetAttribute(int *v, cudaDeviceAttr, int)
{
    *v = 152;
    return cudaSuccess;
}
cudaError_t cudaDeviceSynchronize() { return cudaSuccess; }
cudaError_t cudaStreamSynchronize(cudaStream_t) { return cudaSuccess; }
cudaError_t cudaMemcpyFromSymbol(void *dst, const void *, size_t n, size_t, cudaMemcpyKind)
{
    memset(dst, 0, n);
    return cudaSuccess;
}
cudaError_t cudaMemcpyToSymbol(const void *, const void *, size_t, size_t, cudaMemcpyKind) { return cudaSuccess; }

// what compiled kernels register themselves with
void **__cudaRegisterFatBinary(void *)
{
    static void *handle;
    return &handle;
}
void __cudaRegisterFatBinaryEnd(void **) {}
void __cudaUnregisterFatBinary(void **) {}
void __cudaRegisterFunction(void **, const char *, char *, const char *, int, void *, void *, void *, void *, int *) {}
void __cudaRegisterVar(void **, char *, char *, const char *, int, size_t, int, int) {}
char __cudaInitModule(void **) { return 0; }
unsigned __cudaPushCallConfiguration(dim3 grid, dim3 block, size_t smem, void *stream)
{
    config = {grid, block, smem, (cudaStream_t)stream};
    return 0;
}
cudaError_t __cudaPopCallConfiguration(dim3 *grid, dim3 *block, size_t *smem, void *stream)
{
    *grid = config.grid;
    *block = config.block;
    *smem = config.smem;
    *(cudaStream_t *)stream = config.stream;
    return cudaSuccess;
}
}
