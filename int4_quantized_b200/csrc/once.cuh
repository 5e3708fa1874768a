// once.cuh -- what a launch sets up once on each device (host side).
#pragma once

#include <atomic>
#include <cstdint>

#include <cuda_runtime.h>

namespace q4 {

// Runs set() the first time on each device (a bit of `ready` each; every time beyond the 64th).
// Two threads may both run it, with the same result. A kernel's attributes belong to the device and
// not to the calling thread: set() gives them the largest value that any call needs, never this
// call's own, which another thread's launch might find too small.
template <typename F>
cudaError_t once_per_device(std::atomic<uint64_t> &ready, F set) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
    if (ready.load(std::memory_order_acquire) & bit) return cudaSuccess;
    e = set();
    if (e == cudaSuccess) ready.fetch_or(bit, std::memory_order_release);
    return e;
}

}  // namespace q4
