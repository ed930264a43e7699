/* A CUDA runtime with two devices and no GPU, preloaded under libtide.so so
 * that its host side can be tested: device 1 has fewer SMs and holds fewer
 * clusters than device 0.  Launches do nothing but leave their shape. */
#include <cuda_runtime_api.h>
#include <stdlib.h>
#include <string.h>

static int current = 0;
static int syncs[2] = {0, 0};
static int launches = 0;
static unsigned last_grid[3] = {0, 0, 0};
static unsigned last_cluster = 0;
static int* error_word = NULL;
static int error_at_sync[2] = {0, 0};

/* For the tests. */
int fake_syncs(int device) { return syncs[device]; }
int fake_launches(void) { return launches; }
unsigned fake_grid(int i) { return last_grid[i]; }
unsigned fake_cluster(void) { return last_cluster; }
/* The kernels of `device` write `value` to the error word by the time it is synchronised. */
void fake_error_at_sync(int device, int value) { error_at_sync[device] = value; }

cudaError_t cudaGetDevice(int* d) { return *d = current, cudaSuccess; }
cudaError_t cudaSetDevice(int d) { return current = d, cudaSuccess; }
cudaError_t cudaGetDeviceCount(int* n) { return *n = 2, cudaSuccess; }
cudaError_t cudaGetLastError(void) { return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int* v, enum cudaDeviceAttr attr, int d) {
  *v = attr == cudaDevAttrMultiProcessorCount ? (d ? 16 : 152) : 0;
  return cudaSuccess;
}
cudaError_t cudaDeviceSynchronize(void) {
  ++syncs[current];
  if (error_word && error_at_sync[current]) *error_word = error_at_sync[current];
  return cudaSuccess;
}
cudaError_t cudaStreamIsCapturing(cudaStream_t s, enum cudaStreamCaptureStatus* st) {
  (void)s;
  *st = cudaStreamCaptureStatusNone;
  return cudaSuccess;
}
cudaError_t cudaHostAlloc(void** p, size_t n, unsigned flags) {
  (void)flags;
  *p = calloc(1, n);
  if (!error_word) error_word = (int*)*p;
  return *p ? cudaSuccess : cudaErrorMemoryAllocation;
}
cudaError_t cudaHostGetDevicePointer(void** d, void* h, unsigned flags) {
  (void)flags;
  return *d = h, cudaSuccess;
}
cudaError_t cudaFreeHost(void* p) {
  if (p == error_word) error_word = NULL;
  free(p);
  return cudaSuccess;
}
cudaError_t cudaFuncSetAttribute(const void* f, enum cudaFuncAttribute a, int v) {
  (void)f, (void)a, (void)v;
  return cudaSuccess;
}
static unsigned cluster_of(const cudaLaunchConfig_t* c) {
  for (unsigned i = 0; i < c->numAttrs; ++i)
    if (c->attrs[i].id == cudaLaunchAttributeClusterDimension) return c->attrs[i].val.clusterDim.x;
  return 1;
}
cudaError_t cudaOccupancyMaxActiveClusters(int* n, const void* f, const cudaLaunchConfig_t* c) {
  (void)f;
  *n = (int)((current ? 16 : 144) / cluster_of(c));
  return cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void** args) {
  (void)f, (void)args;
  ++launches;
  last_grid[0] = c->gridDim.x, last_grid[1] = c->gridDim.y, last_grid[2] = c->gridDim.z;
  last_cluster = cluster_of(c);
  return cudaSuccess;
}
static int encode_nothing() { return 0; } /* cuTensorMapEncodeTiled */
cudaError_t cudaGetDriverEntryPointByVersion(const char* name, void** fn, unsigned version, unsigned long long flags,
                                             enum cudaDriverEntryPointQueryResult* found) {
  (void)name, (void)version, (void)flags;
  *fn = (void*)encode_nothing;
  *found = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}
