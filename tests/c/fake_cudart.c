/* A CUDA runtime without a device, linked under the library's own objects: every
 * call succeeds and launches nothing, except the one that fake_fail names.  Like
 * the real one it remembers the last error until cudaGetLastError is called. */
#include <cuda.h>
#include <cuda_runtime_api.h>
#include <string.h>

static cudaError_t g_last;
static char g_name[64];
static int g_nth, g_seen, g_launches;

/* The nth call (from 1) of `name` from now on fails, once; nth 0: none. */
void fake_fail(const char* name, int nth) {
    strncpy(g_name, name, sizeof g_name - 1);
    g_nth = nth;
    g_seen = 0;
}
int fake_seen(void) { return g_seen; }         /* calls of that name since */
int fake_launches(void) { return g_launches; }

static cudaError_t answer(const char* name) {
    if (strcmp(name, g_name) == 0 && ++g_seen == g_nth) return g_last = cudaErrorInvalidValue;
    return cudaSuccess;
}

cudaError_t cudaGetLastError(void) {
    const cudaError_t e = g_last;
    g_last = cudaSuccess;
    return e;
}
const char* cudaGetErrorName(cudaError_t e) { return e == cudaSuccess ? "cudaSuccess" : "cudaErrorInvalidValue"; }
cudaError_t cudaGetDevice(int* d) { return *d = 0, answer("cudaGetDevice"); }
cudaError_t cudaDeviceGetAttribute(int* v, enum cudaDeviceAttr a, int d) {
    (void)a, (void)d;
    const cudaError_t e = answer("cudaDeviceGetAttribute");
    if (e == cudaSuccess) *v = 152;
    return e;
}
cudaError_t cudaPointerGetAttributes(struct cudaPointerAttributes* a, const void* p) {
    memset(a, 0, sizeof *a);
    a->type = cudaMemoryTypeDevice;
    a->devicePointer = (void*)p;
    return answer("cudaPointerGetAttributes");
}
cudaError_t cudaFuncSetAttribute(const void* f, enum cudaFuncAttribute a, int v) {
    (void)f, (void)a, (void)v;
    return answer("cudaFuncSetAttribute");
}
cudaError_t cudaOccupancyMaxActiveBlocksPerMultiprocessor(int* n, const void* f, int t, size_t s) {
    (void)f, (void)t, (void)s;
    return *n = 3, answer("cudaOccupancyMaxActiveBlocksPerMultiprocessor");
}
cudaError_t cudaOccupancyMaxActiveClusters(int* n, const void* f, const cudaLaunchConfig_t* c) {
    (void)f;
    return *n = 128 / (int)c->gridDim.x, answer("cudaOccupancyMaxActiveClusters");
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void** args) {
    (void)c, (void)f, (void)args;
    ++g_launches;
    return answer("cudaLaunchKernelExC");
}
static CUresult fake_encode(CUtensorMap* m) { return memset(m, 0, sizeof *m), CUDA_SUCCESS; }
cudaError_t cudaGetDriverEntryPointByVersion(const char* s, void** p, unsigned v, unsigned long long f, enum cudaDriverEntryPointQueryResult* r) {
    (void)s, (void)v, (void)f;
    *p = (void*)fake_encode;
    *r = cudaDriverEntryPointSuccess;
    return answer("cudaGetDriverEntryPointByVersion");
}
cudaError_t cudaStreamSynchronize(cudaStream_t s) { return (void)s, answer("cudaStreamSynchronize"); }
cudaError_t cudaGetSymbolAddress(void** p, const void* s) { return *p = (void*)s, answer("cudaGetSymbolAddress"); }
cudaError_t cudaMemcpyFromSymbol(void* d, const void* s, size_t n, size_t o, enum cudaMemcpyKind k) {
    (void)s, (void)o, (void)k;
    return memset(d, 0, n), answer("cudaMemcpyFromSymbol");
}
cudaError_t cudaMemcpyToSymbol(const void* s, const void* p, size_t n, size_t o, enum cudaMemcpyKind k) {
    (void)s, (void)p, (void)n, (void)o, (void)k;
    return answer("cudaMemcpyToSymbol");
}

/* what the compiler's host code calls around them */
void** __cudaRegisterFatBinary(void* f) { static void* h; return (void)f, &h; }
void __cudaRegisterFatBinaryEnd(void** h) { (void)h; }
void __cudaUnregisterFatBinary(void** h) { (void)h; }
void __cudaRegisterFunction(void** h, const char* f, char* d, const char* n, int t, void* a, void* b, void* c, void* e, int* w) {
    (void)h, (void)f, (void)d, (void)n, (void)t, (void)a, (void)b, (void)c, (void)e, (void)w;
}
void __cudaRegisterVar(void** h, char* v, char* d, const char* n, int e, size_t s, int c, int g) {
    (void)h, (void)v, (void)d, (void)n, (void)e, (void)s, (void)c, (void)g;
}
unsigned __cudaPushCallConfiguration(struct dim3 g, struct dim3 b, size_t s, void* t) { return (void)g, (void)b, (void)s, (void)t, 0; }
cudaError_t __cudaPopCallConfiguration(struct dim3* g, struct dim3* b, size_t* s, void* t) { return (void)g, (void)b, (void)s, (void)t, cudaSuccess; }
cudaError_t __cudaGetKernel(void** k, const void* f) { return *k = (void*)f, cudaSuccess; }
cudaError_t __cudaLaunchKernel(void* k, struct dim3 g, struct dim3 b, void** a, size_t s, void* t) {
    (void)k, (void)g, (void)b, (void)a, (void)s, (void)t;
    ++g_launches;
    return answer("__cudaLaunchKernel");
}
