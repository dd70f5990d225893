"""The library over a CUDA runtime of our own, for host-side tests without a GPU: its object files linked with one that counts
launches and copies, lets a launch fail, and says what device there is.  No kernel runs."""
import ctypes
import os
import subprocess

from kda_gated_delta_gb300 import build

SOURCE = r"""
#include <cuda_runtime_api.h>
#include <cstring>

static int launches = 0, copies = 0, fail_at = -1, sms = 152, device = 0, silent = 0;
static cudaError_t last = cudaSuccess;

static cudaError_t launch()
{
    if (launches++ != fail_at) return cudaSuccess;
    return last = cudaErrorLaunchOutOfResources;
}
static int encode(...) { return 0; }

extern "C" {
// the test's side
void fake_reset(int fail) { launches = copies = 0; fail_at = fail; last = cudaSuccess; }
int fake_copies() { return copies; }
int fake_launches() { return launches; }
void fake_device(int dev, int count) { device = dev; sms = count; }
void fake_silent(int queries) { silent = queries; }        // so many attribute queries fail

// the library's side
void** __cudaRegisterFatBinary(void*) { static void* handle; return &handle; }
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
void __cudaRegisterFunction(void**, const char*, char*, const char*, int, void*, void*, void*, void*, int*) {}
void __cudaRegisterVar(void**, char*, char*, const char*, int, size_t, int, int) {}
unsigned __cudaPushCallConfiguration(dim3, dim3, size_t, struct CUstream_st*) { return 0; }
cudaError_t __cudaPopCallConfiguration(dim3* grid, dim3* block, size_t* smem, void* stream)
{
    *grid = *block = dim3{1, 1, 1};
    *smem = 0;
    *(void**)stream = nullptr;
    return cudaSuccess;
}
cudaError_t __cudaGetKernel(cudaKernel_t* kernel, const void*) { *kernel = nullptr; return cudaSuccess; }
cudaError_t __cudaLaunchKernel(cudaKernel_t, dim3, dim3, void**, size_t, cudaStream_t) { return launch(); }
cudaError_t cudaLaunchKernel(const void*, dim3, dim3, void**, size_t, cudaStream_t) { return launch(); }
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t*, const void*, void**) { return launch(); }
cudaError_t cudaGetLastError() { const cudaError_t e = last; last = cudaSuccess; return e; }
cudaError_t cudaGetDevice(int* d) { *d = device; return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int* v, enum cudaDeviceAttr, int)
{
    if (silent > 0) { --silent; return cudaErrorUnknown; }
    *v = sms;
    return cudaSuccess;
}
cudaError_t cudaFuncGetAttributes(cudaFuncAttributes* f, const void*) { memset(f, 0, sizeof(*f)); f->numRegs = 96; return cudaSuccess; }
cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int) { return cudaSuccess; }
cudaError_t cudaOccupancyMaxActiveBlocksPerMultiprocessorWithFlags(int* n, const void*, int, size_t, unsigned) { *n = 2; return cudaSuccess; }
cudaError_t cudaGetDriverEntryPointByVersion(const char*, void** f, unsigned, unsigned long long, enum cudaDriverEntryPointQueryResult* r)
{
    *f = (void*)&encode;
    *r = cudaDriverEntryPointSuccess;
    return cudaSuccess;
}
cudaError_t cudaMemcpyFromSymbol(void* to, const void*, size_t n, size_t, enum cudaMemcpyKind) { ++copies; memset(to, 0, n); return cudaSuccess; }
cudaError_t cudaMemcpyToSymbol(const void*, const void*, size_t, size_t, enum cudaMemcpyKind) { ++copies; return cudaSuccess; }
cudaError_t cudaMemcpyFromSymbolAsync(void* to, const void*, size_t n, size_t, enum cudaMemcpyKind, cudaStream_t)
{
    ++copies;
    memset(to, 0, n);
    return cudaSuccess;
}
cudaError_t cudaGetSymbolAddress(void** p, const void*) { *p = (void*)(size_t)(1 << 20); return cudaSuccess; }
cudaError_t cudaStreamSynchronize(cudaStream_t) { return cudaSuccess; }
cudaError_t cudaEventRecord(cudaEvent_t, cudaStream_t) { return cudaSuccess; }
}
"""
OBJECTS = [os.path.splitext(f)[0] + ".o" for f in build.SOURCES]


def load(folder) -> ctypes.CDLL:
    """A fresh copy of the library, with none of another test's device properties."""
    build.build()
    objects = [os.path.join(build.BUILD, o) for o in OBJECTS]
    if not all(map(os.path.exists, objects)):
        build.build(force=True)
    src, lib = os.path.join(str(folder), "runtime.cpp"), os.path.join(str(folder), "libfake.so")
    with open(src, "w") as f:
        f.write(SOURCE)
    cuda = os.path.join(os.path.dirname(os.path.dirname(build.nvcc())), "include")
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-Wl,-Bsymbolic,--no-undefined", "-I", cuda, src, *objects, "-o", lib], check=True)
    return ctypes.CDLL(lib, mode=os.RTLD_LOCAL | os.RTLD_NOW)
