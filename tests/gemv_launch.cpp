// The host side of mx_gemv.cu on a CUDA runtime that is a fake: which launches
// it makes for given sizes, and what it does when a query fails.  Linked with
// mx_gemv.o by test_gemv_launch.py.
//
// Arguments, one call each: tokens,n,k,f32,nvfp4,fail with fail = 1 for calls
// whose cluster queries fail.  Prints for each call: the error, the kernels
// launched, and for the last one its grid, block, cluster and shared memory;
// then the kernel that the queries were made of (0: none, -1: several).
#include <cstdio>
#include <cstdlib>
#include <set>

#include <cuda_runtime.h>

#include "mx.h"
#include "mx_internal.h"

namespace {
bool failing = false;
int launches = 0;
cudaLaunchConfig_t last = {};
unsigned last_cluster = 1;
std::set<const void *> allowed, asked;

unsigned cluster_of(const cudaLaunchConfig_t *c) {
    for (unsigned i = 0; i < c->numAttrs; ++i)
        if (c->attrs[i].id == cudaLaunchAttributeClusterDimension) return c->attrs[i].val.clusterDim.x;
    return 1;
}
}  // namespace

extern "C" {
void **__cudaRegisterFatBinary(void *) { static void *p; return &p; }
void __cudaRegisterFatBinaryEnd(void **) {}
void __cudaUnregisterFatBinary(void **) {}
void __cudaRegisterFunction(void **, const char *, char *, const char *, int, uint3 *, uint3 *, dim3 *, dim3 *, int *) {}
void __cudaRegisterVar(void **, char *, char *, const char *, int, size_t, int, int) {}
unsigned __cudaPopCallConfiguration(dim3 *, dim3 *, size_t *, void *) { return 1; }
cudaError_t cudaLaunchKernel(const void *, dim3, dim3, void **, size_t, cudaStream_t) { return cudaErrorNotSupported; }
cudaError_t cudaGetDevice(int *d) { *d = 0; return cudaSuccess; }
cudaError_t cudaFuncSetAttribute(const void *f, cudaFuncAttribute, int) { allowed.insert(f); return cudaSuccess; }
cudaError_t cudaOccupancyMaxActiveClusters(int *n, const void *f, const cudaLaunchConfig_t *c) {
    asked.insert(f);
    if (failing || !allowed.count(f)) return cudaErrorUnknown;
    const unsigned size = cluster_of(c);
    *n = size == 2 ? 74 : size == 4 ? 34 : 16;
    return cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t *c, const void *f, void **) {
    ++launches;
    last = *c;
    last_cluster = cluster_of(c);
    return allowed.count(f) ? cudaSuccess : cudaErrorInvalidValue;
}
}

int main(int argc, char **argv) {
    for (int i = 1; i < argc; ++i) {
        long long m, n, k;
        int f32, nv, fail;
        if (std::sscanf(argv[i], "%lld,%lld,%lld,%d,%d,%d", &m, &n, &k, &f32, &nv, &fail) != 6) return 2;
        static float enc = 1.0f;
        MxGemvArgs a = {};
        a.codes = a.scales = a.x = a.y = &enc;
        a.enc = nv ? &enc : nullptr;
        a.lines = n;
        a.sl = MX_SCALES_MMA;
        a.xdt = a.ydt = f32 ? MX_F32 : MX_BF16;
        a.ldx = k; a.ldy = n; a.M = m; a.N = n; a.K = k; a.alpha = 1.0f; a.num_sms = 148;
        failing = fail;
        launches = 0;
        const int rc = mx_launch_gemv(a, nullptr);
        std::printf("%d %d", rc, launches);
        if (launches)
            std::printf(" %u,%u %u %u %zu", last.gridDim.x, last.gridDim.y, last.blockDim.x, last_cluster, last.dynamicSmemBytes);
        std::printf("\n");
    }
    const long who = asked.empty() ? 0 : asked.size() > 1 ? -1 : reinterpret_cast<long>(*asked.begin());
    std::printf("%ld\n", who);
    return 0;
}
