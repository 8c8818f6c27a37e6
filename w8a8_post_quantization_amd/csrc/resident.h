// How many blocks of a kernel a GPU holds at once, asked of the runtime once
// for each kernel and GPU.
#pragma once

#include <atomic>
#include <cstdint>

namespace sq {

// ask() for this kernel on GPU `gpu`, remembered.  The kernel itself is the
// key: kernels of one type (the instances of a template) have values of their
// own.  GPUs past the array are asked every time.
template <auto Kernel, class Ask>
int64_t once_per_gpu(int gpu, Ask ask) {
    constexpr int kGpus = 64;
    static std::atomic<int64_t> known[kGpus];  // 0: not asked yet
    if (gpu < 0 || gpu >= kGpus) return ask();
    int64_t n = known[gpu].load(std::memory_order_relaxed);
    if (n == 0) known[gpu].store(n = ask(), std::memory_order_relaxed);
    return n;
}

}  // namespace sq
