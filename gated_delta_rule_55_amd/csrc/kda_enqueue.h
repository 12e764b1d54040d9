// kda_enqueue.h -- a kernel launch with its own status.
#pragma once

#include <hip/hip_runtime.h>

#include <tuple>
#include <utility>

namespace kda {

// Enqueues `kernel` with these arguments and returns this launch's status.
// (hipGetLastError would answer with, and clear, an error that any earlier call
// of the thread left behind: a good launch then looks failed.)  A launch's own
// failure is not left behind for later callers.
template <typename... P, typename... A>
hipError_t enqueue(void (*kernel)(P...), unsigned blocks, unsigned threads, hipStream_t stream, A&&... args) {
  std::tuple<P...> values(std::forward<A>(args)...);
  return std::apply(
      [&](P&... v) {
        void* ptrs[] = {static_cast<void*>(&v)...};
        const hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(kernel), dim3(blocks), dim3(threads),
                                             ptrs, 0, stream);
        if (e != hipSuccess) (void)hipGetLastError();
        return e;
      },
      values);
}

}  // namespace kda
