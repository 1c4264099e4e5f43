// Two threads that make a kernel's first calls with different sizes: the limit
// must end at the larger, whichever comes first.  The CUDA calls are stand-ins:
// the one that sets the smaller limit waits (at most a moment) for the larger.
#include <cuda_runtime.h>

#include <atomic>
#include <chrono>
#include <cstdio>
#include <thread>

static std::atomic<int> limit_now{0}, smaller_started{0};
constexpr int kSmall = 100000, kLarge = 200000;

static cudaError_t fake_device(int *dev)
{
    *dev = 3;
    return cudaSuccess;
}
template <typename Kernel>
static cudaError_t fake_set(Kernel, cudaFuncAttribute, int bytes)
{
    if (bytes == kSmall) {
        smaller_started = 1;
        const auto until = std::chrono::steady_clock::now() + std::chrono::milliseconds(300);
        while (limit_now != kLarge && std::chrono::steady_clock::now() < until) std::this_thread::yield();
    }
    limit_now = bytes;
    return cudaSuccess;
}
#define cudaGetDevice fake_device
#define cudaFuncSetAttribute fake_set
#include "moira_launch.h"

static __global__ void kernel() {}

int main()
{
    static std::atomic<int> seen[64];
    cudaError_t small = cudaErrorUnknown, large = cudaErrorUnknown;
    std::thread a([&] { small = moira::raise_smem_limit(kernel, kSmall, seen); });
    while (!smaller_started) std::this_thread::yield();
    std::thread b([&] { large = moira::raise_smem_limit(kernel, kLarge, seen); });
    a.join();
    b.join();
    if (small != cudaSuccess || large != cudaSuccess || limit_now != kLarge || seen[3] != kLarge) {
        std::printf("limit %d, record %d\n", limit_now.load(), seen[3].load());
        return 1;
    }
    moira::raise_smem_limit(kernel, kSmall, seen);
    if (limit_now != kLarge) {
        std::printf("lowered to %d\n", limit_now.load());
        return 1;
    }
    std::printf("ok\n");
    return 0;
}
