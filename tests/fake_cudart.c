/* A stand-in for the CUDA runtime that launches nothing: the host code of the
 * library runs against it on a machine without a GPU.  It reports a device of
 * 152 SMs, and logs one line for each kernel that is prepared ("attribute
 * NAME", "query NAME") or launched ("launch NAME x y z"). */
#include <cuda_runtime_api.h>
#include <stdio.h>
#include <string.h>

static char g_log[1 << 20];
static size_t g_used;
static int g_registers = 255;
static const void* g_fn[4096];
static const char* g_name[4096];
static int g_fns;

static void put(const char* what, const void* fn, const dim3* grid) {
  const char* name = "?";
  for (int i = 0; i < g_fns; ++i)
    if (g_fn[i] == fn) name = g_name[i];
  const size_t left = sizeof(g_log) - g_used;
  const int n = grid ? snprintf(g_log + g_used, left, "%s %s %u %u %u\n", what, name, grid->x, grid->y, grid->z)
                     : snprintf(g_log + g_used, left, "%s %s\n", what, name);
  if (n > 0 && (size_t)n < left) g_used += (size_t)n;
}

const char* fake_log(void) { return g_log; }
void fake_clear(void) { g_used = 0, g_log[0] = 0; }
void fake_registers(int n) { g_registers = n; }   /* what a kernel's attributes report */

void** __cudaRegisterFatBinary(void* p) {
  static void* handle;
  (void)p;
  return &handle;
}
void __cudaRegisterFatBinaryEnd(void** h) { (void)h; }
void __cudaUnregisterFatBinary(void** h) { (void)h; }
void __cudaRegisterVar(void** h, char* v, char* a, const char* n, int e, size_t s, int c, int g) {
  (void)h, (void)v, (void)a, (void)n, (void)e, (void)s, (void)c, (void)g;
}
void __cudaRegisterFunction(void** h, const char* fn, char* dev, const char* name, int t, void* a, void* b, void* c, void* d,
                            int* w) {
  (void)h, (void)dev, (void)t, (void)a, (void)b, (void)c, (void)d, (void)w;
  if (g_fns < 4096) g_fn[g_fns] = fn, g_name[g_fns++] = name;
}
cudaError_t __cudaGetKernel(cudaKernel_t* k, const void* fn) {
  *k = (cudaKernel_t)fn;
  return cudaSuccess;
}
unsigned __cudaPushCallConfiguration(dim3 g, dim3 b, size_t s, struct CUstream_st* st) {
  (void)g, (void)b, (void)s, (void)st;
  return 0;
}
cudaError_t __cudaPopCallConfiguration(dim3* g, dim3* b, size_t* s, void* st) {
  (void)g, (void)b, (void)s, (void)st;
  return cudaSuccess;
}
cudaError_t __cudaLaunchKernel(cudaKernel_t k, dim3 g, dim3 b, void** a, size_t s, cudaStream_t st) {
  (void)b, (void)a, (void)s, (void)st;
  put("launch", (const void*)k, &g);
  return cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* fn, void** a) {
  (void)a;
  put("launch", fn, &c->gridDim);
  return cudaSuccess;
}
cudaError_t cudaFuncSetAttribute(const void* fn, enum cudaFuncAttribute a, int v) {
  (void)a, (void)v;
  put("attribute", fn, NULL);
  return cudaSuccess;
}
cudaError_t cudaFuncGetAttributes(struct cudaFuncAttributes* a, const void* fn) {
  memset(a, 0, sizeof(*a));
  a->numRegs = g_registers;
  put("query", fn, NULL);
  return cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveBlocksPerMultiprocessorWithFlags(int* n, const void* fn, int b, size_t s, unsigned f) {
  (void)b, (void)s, (void)f;
  *n = 1;
  put("query", fn, NULL);
  return cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveClusters(int* n, const void* fn, const cudaLaunchConfig_t* c) {
  (void)c;
  *n = 1;
  put("query", fn, NULL);
  return cudaSuccess;
}
cudaError_t cudaGetDevice(int* d) {
  *d = 0;
  return cudaSuccess;
}
cudaError_t cudaDeviceGetAttribute(int* v, enum cudaDeviceAttr a, int d) {
  (void)a, (void)d;
  *v = 152;
  return cudaSuccess;
}
cudaError_t cudaGetLastError(void) { return cudaSuccess; }
cudaError_t cudaGetSymbolAddress(void** p, const void* s) {
  *p = (void*)s;
  return cudaSuccess;
}
cudaError_t cudaMemcpyAsync(void* d, const void* s, size_t n, enum cudaMemcpyKind k, cudaStream_t st) {
  (void)d, (void)s, (void)n, (void)k, (void)st;
  return cudaSuccess;
}
cudaError_t cudaMemsetAsync(void* d, int v, size_t n, cudaStream_t st) {
  (void)d, (void)v, (void)n, (void)st;
  return cudaSuccess;
}
cudaError_t cudaStreamSynchronize(cudaStream_t st) {
  (void)st;
  return cudaSuccess;
}
