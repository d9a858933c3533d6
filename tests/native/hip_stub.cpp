// A stand-in for the HIP runtime's launch and device calls, for tests without
// a GPU: loaded with RTLD_GLOBAL before the library, its definitions come
// first.  A launch is written down with the host thread and the current
// device, and takes a while, so that threads that may interleave do.
#include <hip/hip_runtime_api.h>

#include <pthread.h>
#include <stddef.h>
#include <stdlib.h>
#include <unistd.h>

#include <mutex>
#include <vector>

namespace {
struct Launch {
  uint64_t thread;
  int device;
  hipStream_t stream;
};
std::mutex lock;
std::vector<Launch> launches;
int devices = 2;
thread_local int current = 0;
thread_local struct {
  dim3 grid, block;
  size_t lds;
  hipStream_t stream;
} configuration;
}  // namespace

extern "C" {

// What the compiler makes of a kernel's call, around hipLaunchKernel.
hipError_t __hipPushCallConfiguration(dim3 grid, dim3 block, size_t lds, hipStream_t stream) {
  configuration = {grid, block, lds, stream};
  return hipSuccess;
}
hipError_t __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* lds, hipStream_t* stream) {
  *grid = configuration.grid;
  *block = configuration.block;
  *lds = configuration.lds;
  *stream = configuration.stream;
  return hipSuccess;
}
hipError_t hipLaunchKernel(const void*, dim3, dim3, void**, size_t, hipStream_t stream) {
  {
    std::lock_guard<std::mutex> hold(lock);
    launches.push_back({static_cast<uint64_t>(pthread_self()), current, stream});
  }
  usleep(500);
  return hipSuccess;
}
hipError_t hipGetLastError(void) { return hipSuccess; }
hipError_t hipFuncSetAttribute(const void*, hipFuncAttribute, int) { return hipSuccess; }
hipError_t hipGetDeviceCount(int* n) {
  *n = devices;
  return hipSuccess;
}
hipError_t hipGetDevice(int* d) {
  *d = current;
  return hipSuccess;
}
hipError_t hipSetDevice(int d) {
  if (d < 0 || d >= devices) return hipErrorInvalidDevice;
  current = d;
  return hipSuccess;
}
hipError_t hipGetSymbolAddress(void** p, const void*) {
  *p = reinterpret_cast<void*>(uintptr_t{1} << 20);
  return hipSuccess;
}
hipError_t hipDeviceGetStreamPriorityRange(int* least, int* greatest) {
  *least = *greatest = 0;
  return hipSuccess;
}
// The allocator of torch's tensors, from host memory.
void* stub_alloc(ptrdiff_t bytes, int, hipStream_t) {
  return aligned_alloc(512, (bytes + 511) / 512 * 512);
}
void stub_free(void* p, ptrdiff_t, int, hipStream_t) { free(p); }

int stub_launches(void) {
  std::lock_guard<std::mutex> hold(lock);
  return static_cast<int>(launches.size());
}
uint64_t stub_thread(int i) { return launches[i].thread; }
int stub_device(int i) { return launches[i].device; }
void stub_clear(void) {
  std::lock_guard<std::mutex> hold(lock);
  launches.clear();
}

}  // extern "C"
