// cache_api.cu -- status word and test hook of libhstu_cache_b200.
#include <atomic>

#include "../ptx.cuh"
#include "cache_internal.h"

namespace hstu {

namespace {
std::atomic<long long> g_wait_limit{0};
std::atomic<int> g_withhold{0};
}  // namespace

DebugWait cache_debug_wait() {
    DebugWait w;
    const long long l = g_wait_limit.load();
    w.limit = l > 0 ? l : ptx::kWaitLimitCycles;
    w.withhold_first_load = g_withhold.load();
    return w;
}

}  // namespace hstu

using namespace hstu;

int hstu_cache_debug_set_wait_fault(int64_t wait_limit_cycles, int32_t withhold_first_load) {
    if (wait_limit_cycles < 0 || (withhold_first_load != 0 && withhold_first_load != 1)) return HSTU_ERR_INVALID_ARG;
    g_wait_limit.store(wait_limit_cycles);
    g_withhold.store(withhold_first_load);
    return HSTU_OK;
}

int hstu_cache_check_device_error(void* workspace, void* stream) {
    if (!aligned(workspace, 256)) return HSTU_ERR_WORKSPACE;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int status = 0;
    cudaError_t e = cudaMemcpyAsync(&status, workspace, sizeof(int), cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e == cudaSuccess && status != 0) {
        e = cudaMemsetAsync(workspace, 0, sizeof(int), s);
        if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    }
    if (e != cudaSuccess) return cuda_status(e);
    if (status & kStatusTimeout) return HSTU_ERR_DEVICE_TIMEOUT;
    if (status & kStatusBounds) return HSTU_ERR_DEVICE_BOUNDS;
    if (status & kStatusFull) return HSTU_ERR_CACHE_FULL;
    return HSTU_OK;
}
