// What holds for one device only and is set once for each: shared by the
// libnys translation units.  Not part of the ABI.
#pragma once

#include <atomic>
#include <cstddef>

namespace nys {

// The largest value that was set so far on each device.  Threads that meet set
// it twice, which is harmless; a failure is not remembered.
class PerDevice {
 public:
  // set() returns 0 on success; it is called where `value` is above what the device
  // has (from `first` on), and its answer returned.
  template <typename F>
  auto raise(int device, size_t value, size_t first, F set) -> decltype(set()) {
    const bool known = device >= 0 && device < kMost;
    const size_t have = known ? most_[device].load(std::memory_order_relaxed) : 0;
    if (known && value <= (have > first ? have : first)) return decltype(set())(0);
    const auto rc = set();
    if (known && rc == decltype(set())(0)) {
      size_t was = have;
      while (was < value && !most_[device].compare_exchange_weak(was, value)) {
      }
    }
    return rc;
  }

 private:
  static constexpr int kMost = 64;
  std::atomic<size_t> most_[kMost] = {};
};

#ifdef __CUDACC__
// Raise a kernel's dynamic shared-memory limit on the current device, only when a
// launch needs more than any earlier one there (one driver call per kernel, device
// and size, none during later launches -- e.g. inside CUDA graph capture after a
// warm-up launch).
template <auto Kernel>
inline cudaError_t ensure_smem(size_t bytes) {
  static PerDevice limits;  // one record per kernel
  int device = 0;
  const cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  return limits.raise(device, bytes, 48 * 1024, [bytes] {
    return cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  });
}
#endif

}  // namespace nys
