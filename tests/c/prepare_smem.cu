// Two threads that allow one kernel different amounts of shared memory for the
// first time, against stand-ins for the runtime's calls: the larger amount has to
// be what the kernel is left with.
#include <atomic>
#include <chrono>
#include <cstdio>
#include <thread>

static std::atomic<int> g_left{0};
static cudaError_t fake_device(int* dev) {
    *dev = 0;
    return cudaSuccess;
}
template <class K>
static cudaError_t fake_set(K, cudaFuncAttribute, int bytes) {
    // the smaller amount takes its time
    if (bytes < 2048) std::this_thread::sleep_for(std::chrono::milliseconds(300));
    g_left = bytes;
    return cudaSuccess;
}
#define cudaGetDevice fake_device
#define cudaFuncSetAttribute fake_set
#include "kvw_device.cuh"

__global__ void kernel() {}

int main() {
    std::thread small([] { kvw::prepare_smem<&kernel>(1024); });
    std::this_thread::sleep_for(std::chrono::milliseconds(100));
    std::thread large([] { kvw::prepare_smem<&kernel>(98308); });
    small.join();
    large.join();
    kvw::prepare_smem<&kernel>(98308);  // a later call finds it allowed
    std::printf("left with %d bytes\n", g_left.load());
    return g_left.load() == 98308 ? 0 : 1;
}
