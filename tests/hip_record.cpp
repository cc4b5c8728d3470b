// hip_record.cpp -- the HIP runtime calls of libfp8gemm.so's host code without a GPU: memory is a
// made-up address, and a kernel launch is a line of a log (thread, stream, blocks, threads) followed
// by a short sleep, so that calls of other threads get their chance between two launches.  Loaded
// before the library with its symbols global, so that the library finds these first.
#include <hip/hip_runtime_api.h>

#include <unistd.h>

#include <atomic>
#include <cstring>
#include <mutex>
#include <vector>

namespace {

struct Launch {
    int64_t thread, stream, blocks, threads;
};
std::mutex mu;
std::vector<Launch> launches;
std::atomic<uint64_t> next_address{uint64_t(1) << 40};
std::atomic<int> allocations{0};
std::atomic<int> frees{0};
std::atomic<int> fail_after{-1};                 // allocations that still succeed, or -1: all do
std::atomic<int> pause_us{500};
thread_local hipError_t last_error = hipSuccess; // as the runtime keeps it: until it is asked for

struct Config {
    dim3 grid, block;
    size_t shared;
    hipStream_t stream;
};
thread_local Config config;

}  // namespace

extern "C" {

// Lines of the log from `first` on, 4 numbers each; returns how many there are in all.
int64_t record_launches(int64_t first, int64_t* out, int64_t room) {
    std::lock_guard<std::mutex> lock(mu);
    for (int64_t i = 0; i < room && first + i < (int64_t)launches.size(); ++i)
        std::memcpy(out + 4 * i, &launches[first + i], sizeof(Launch));
    return (int64_t)launches.size();
}
void record_pause(int us) { pause_us = us; }
int record_allocations() { return allocations; }
int record_frees() { return frees; }
void record_fail_after(int n) { fail_after = n; }

hipError_t __hipPushCallConfiguration(dim3 grid, dim3 block, size_t shared, hipStream_t stream) {
    config = {grid, block, shared, stream};
    return hipSuccess;
}
hipError_t __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* shared, hipStream_t* stream) {
    *grid = config.grid;
    *block = config.block;
    *shared = config.shared;
    *stream = config.stream;
    return hipSuccess;
}
hipError_t hipLaunchKernel(const void*, dim3 grid, dim3 block, void**, size_t, hipStream_t stream) {
    {
        std::lock_guard<std::mutex> lock(mu);
        launches.push_back({(int64_t)gettid(), (int64_t)(uintptr_t)stream, (int64_t)grid.x * grid.y * grid.z,
                            (int64_t)block.x * block.y * block.z});
    }
    if (pause_us > 0) usleep(pause_us);
    return hipSuccess;
}
hipError_t hipGetLastError() {
    const hipError_t e = last_error;
    last_error = hipSuccess;
    return e;
}
hipError_t hipGetDevice(int* device) {
    *device = 0;
    return hipSuccess;
}
hipError_t hipGetDevicePropertiesR0600(hipDeviceProp_tR0600* prop, int) {
    std::memset(prop, 0, sizeof *prop);
    prop->multiProcessorCount = 256;
    return hipSuccess;
}
hipError_t hipOccupancyMaxActiveBlocksPerMultiprocessor(int* blocks, const void*, int, size_t) {
    *blocks = 1;
    return hipSuccess;
}
hipError_t hipGetSymbolAddress(void** address, const void*) {
    *address = reinterpret_cast<void*>(next_address.fetch_add(uint64_t(1) << 32));
    return hipSuccess;
}
hipError_t hipMalloc(void** p, size_t) {
    if (fail_after >= 0 && fail_after-- == 0) return last_error = hipErrorOutOfMemory;
    ++allocations;
    *p = reinterpret_cast<void*>(next_address.fetch_add(uint64_t(1) << 32));
    return hipSuccess;
}
hipError_t hipFree(void* p) {
    if (p) ++frees;
    return hipSuccess;
}
hipError_t hipMemset(void*, int, size_t) { return hipSuccess; }
hipError_t hipStreamIsCapturing(hipStream_t, hipStreamCaptureStatus* status) {
    *status = hipStreamCaptureStatusNone;
    return hipSuccess;
}

}  // extern "C"
