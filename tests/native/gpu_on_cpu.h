// What a simple kernel needs of the GPU's language, on the CPU: a work-group
// is as many host threads, lane shuffles and __syncthreads are barriers.  It
// runs a kernel's own source under AddressSanitizer and UBSan, with operands
// that end where they end, so an access outside them is reported.  All lanes
// of a wave have to take part in a shuffle.  Shared arrays are static; dynamic
// ones are gpu_on_cpu::lds.
#pragma once

#include <pthread.h>
#include <stddef.h>
#include <stdint.h>

#include <algorithm>
#include <thread>
#include <vector>

struct dim3 {
  unsigned x, y, z;
  dim3(unsigned x_ = 1, unsigned y_ = 1, unsigned z_ = 1) : x(x_), y(y_), z(z_) {}
};
typedef int hipError_t;
typedef void* hipStream_t;
enum { hipSuccess = 0, hipFuncAttributeMaxDynamicSharedMemorySize = 8 };
inline hipError_t hipGetLastError() { return hipSuccess; }
inline hipError_t hipFuncSetAttribute(const void*, int, int) { return hipSuccess; }

inline thread_local dim3 threadIdx, blockIdx, blockDim, gridDim;

namespace gpu_on_cpu {

struct Barrier {
  pthread_barrier_t b;
  explicit Barrier(unsigned n) { pthread_barrier_init(&b, nullptr, n); }
  ~Barrier() { pthread_barrier_destroy(&b); }
  void wait() { pthread_barrier_wait(&b); }
};
struct Wave {
  Barrier barrier{64};
  int64_t lane[64];
};
inline Barrier* group;                   // of the work-group that runs
inline std::vector<Wave*> waves;
inline std::vector<int32_t> lds;

template <class T>
T from_lane(T v, int from) {
  Wave& w = *waves[threadIdx.x / 64];
  const int lane = threadIdx.x % 64;
  w.lane[lane] = v;
  w.barrier.wait();
  const T r = static_cast<T>(w.lane[from < 0 || from > 63 ? lane : from]);
  w.barrier.wait();
  return r;
}

template <class K, class A>
void launch(K kernel, dim3 grid, dim3 block, size_t lds_bytes, const A& a) {
  const unsigned n = block.x;
  for (unsigned wg = 0; wg < grid.x; ++wg) {
    Barrier all(n);
    group = &all;
    waves.clear();
    for (unsigned w = 0; w < n / 64; ++w) waves.push_back(new Wave);
    lds.assign(lds_bytes / 4, 0x5A5A5A5A);
    std::vector<std::thread> threads;
    for (unsigned t = 0; t < n; ++t)
      threads.emplace_back([=, &a] {
        threadIdx = dim3(t);
        blockIdx = dim3(wg);
        blockDim = block;
        gridDim = grid;
        kernel(a);
      });
    for (auto& t : threads) t.join();
    for (Wave* w : waves) delete w;
  }
}

}  // namespace gpu_on_cpu

template <class T>
T __shfl_up(T v, int d) { return gpu_on_cpu::from_lane(v, static_cast<int>(threadIdx.x % 64) - d); }
template <class T>
T __shfl_xor(T v, int d) { return gpu_on_cpu::from_lane(v, static_cast<int>(threadIdx.x % 64) ^ d); }
inline void __syncthreads() { gpu_on_cpu::group->wait(); }

#define __global__
#define __device__
#define __forceinline__ inline
#define __launch_bounds__(...)
#define __shared__ static
#define hipLaunchKernelGGL(kernel, grid, block, lds, stream, ...) \
  gpu_on_cpu::launch(kernel, grid, block, lds, __VA_ARGS__)

using std::max;
using std::min;
