/* Stand-in for the part of the HIP runtime that allocations and launches go through, with two
 * GPUs that run nothing: it keeps the current device of the thread, gives host memory and
 * writes down each launch's device, stream and grid.  Loaded with RTLD_GLOBAL before PyTorch
 * and the library, whose references to these names it then takes (host-only tests). */
#define __HIP_PLATFORM_AMD__ 1
#include <hip/hip_runtime_api.h>
#include <stdlib.h>
#include <string.h>

typedef struct {
  int device;
  void* stream;
  unsigned grid[3], block[3];
} launch_t;

enum { MOST = 256 };
static launch_t launches[MOST];
static int count;
static __thread int current;
static __thread struct {
  dim3 grid, block;
  size_t lds;
  hipStream_t stream;
} pushed;
static const size_t memory = (size_t)1 << 28;

int fake_count(void) { return count; }
const launch_t* fake_launches(void) { return launches; }
void fake_clear(void) { count = 0; }

hipError_t hipGetDeviceCount(int* n) {
  *n = 2;
  return hipSuccess;
}
hipError_t hipGetDevice(int* d) {
  *d = current;
  return hipSuccess;
}
hipError_t hipSetDevice(int d) {
  if (d < 0 || d > 1) return hipErrorInvalidDevice;
  current = d;
  return hipSuccess;
}
hipError_t hipGetDeviceProperties(hipDeviceProp_t* p, int d) {
  (void)d;
  memset(p, 0, sizeof *p);
  strcpy(p->name, "none");
  strcpy(p->gcnArchName, "gfx950");
  p->totalGlobalMem = memory;
  p->warpSize = 64;
  p->major = 9;
  p->minor = 5;
  p->multiProcessorCount = 256;
  p->maxThreadsPerBlock = 1024;
  return hipSuccess;
}
hipError_t hipDeviceGetAttribute(int* v, hipDeviceAttribute_t attribute, int d) {
  (void)attribute;
  (void)d;
  *v = 256;
  return hipSuccess;
}
hipError_t hipDeviceCanAccessPeer(int* can, int d, int peer) {
  (void)d;
  (void)peer;
  *can = 0;
  return hipSuccess;
}
hipError_t hipDevicePrimaryCtxGetState(hipDevice_t d, unsigned* flags, int* active) {
  (void)d;
  *flags = 0;
  *active = 1;
  return hipSuccess;
}
hipError_t hipGetLastError(void) { return hipSuccess; }
hipError_t hipPeekAtLastError(void) { return hipSuccess; }
hipError_t hipDeviceGetStreamPriorityRange(int* least, int* greatest) {
  *least = *greatest = 0;
  return hipSuccess;
}
hipError_t hipStreamIsCapturing(hipStream_t s, hipStreamCaptureStatus* status) {
  (void)s;
  *status = hipStreamCaptureStatusNone;
  return hipSuccess;
}
hipError_t hipDeviceSynchronize(void) { return hipSuccess; }
hipError_t hipStreamSynchronize(hipStream_t s) {
  (void)s;
  return hipSuccess;
}
hipError_t hipGetSymbolAddress(void** p, const void* symbol) {
  *p = (void*)symbol;
  return hipSuccess;
}
hipError_t hipMalloc(void** p, size_t n) {
  *p = n > memory ? NULL : aligned_alloc(512, (n + 511) / 512 * 512);
  return *p == NULL ? hipErrorOutOfMemory : hipSuccess;
}
hipError_t hipFree(void* p) {
  free(p);
  return hipSuccess;
}
hipError_t hipMemGetInfo(size_t* available, size_t* total) {
  *available = *total = memory;
  return hipSuccess;
}
hipError_t __hipPushCallConfiguration(dim3 grid, dim3 block, size_t lds, hipStream_t stream) {
  pushed.grid = grid;
  pushed.block = block;
  pushed.lds = lds;
  pushed.stream = stream;
  return hipSuccess;
}
hipError_t __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* lds, hipStream_t* stream) {
  *grid = pushed.grid;
  *block = pushed.block;
  *lds = pushed.lds;
  *stream = pushed.stream;
  return hipSuccess;
}
hipError_t hipLaunchKernel(const void* f, dim3 grid, dim3 block, void** args, size_t lds, hipStream_t stream) {
  (void)f;
  (void)args;
  (void)lds;
  if (count < MOST) {
    launch_t l = {current, stream, {grid.x, grid.y, grid.z}, {block.x, block.y, block.z}};
    launches[count++] = l;
  }
  return hipSuccess;
}
