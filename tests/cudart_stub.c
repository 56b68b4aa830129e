/* The CUDA runtime calls of ac_layer.cu on a machine without a GPU: device
 * memory is host memory, every call succeeds.  And the registration hooks of a
 * module without kernels. */
#include <stdlib.h>
#include <string.h>

static int device, entry;
static void *handle;

void stub_device(int d) { device = d; }

int cudaGetDevice(int *d) { return *d = device, 0; }
int cudaGetLastError(void) { return 0; }
int cudaDeviceGetAttribute(int *v, int a, int d) { return (void)a, (void)d, *v = 148, 0; }
int cudaMalloc(void **p, size_t n) { return *p = calloc(1, n), 0; }
int cudaFree(void *p) { return free(p), 0; }
int cudaMemset(void *p, int v, size_t n) { return memset(p, v, n), 0; }
int cudaMemsetAsync(void *p, int v, size_t n, void *s) { return (void)s, memset(p, v, n), 0; }
int cudaMemcpyAsync(void *d, const void *s, size_t n, int k, void *st) { return (void)k, (void)st, memcpy(d, s, n), 0; }
int cudaStreamSynchronize(void *s) { return (void)s, 0; }
int cudaGetDriverEntryPoint(const char *n, void **f, unsigned long long g, int *q) {
    return (void)n, (void)g, *f = &entry, *q = 0, 0;
}

void **__cudaRegisterFatBinary(void *p) { return (void)p, &handle; }
void __cudaRegisterFatBinaryEnd(void **p) { (void)p; }
void __cudaUnregisterFatBinary(void **p) { (void)p; }
