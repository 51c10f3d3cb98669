// The host side of every call that takes a workspace, with a recorder in the place of
// the HIP runtime and of the kernels: which call each launch belongs to, in the order of
// the launches.  Built together with gemm_relu_api.hip, groups_api.hip and blocks_api.hip
// as they are.  Pointers are never followed.
#include <hip/hip_runtime.h>

#include <chrono>
#include <condition_variable>
#include <cstring>
#include <mutex>
#include <thread>
#include <vector>

#include "../tiled_dense_gemm_relu_amd/csrc/blocks_table.hpp"
#include "../tiled_dense_gemm_relu_amd/csrc/groups_table.hpp"
#include "../tiled_dense_gemm_relu_amd/csrc/kernel_table.hpp"

namespace {

char g_kernel;
std::mutex g_mutex;
std::condition_variable g_changed;
std::vector<int> g_log;
int g_held = -1;
thread_local int t_call = -1;

template <class Table>
Table all_kernels()
{
    Table t;
    const void** p = reinterpret_cast<const void**>(&t);
    for (size_t i = 0; i < sizeof(Table) / sizeof(void*); ++i) p[i] = &g_kernel;
    return t;
}
template <class Table>
const Table& table()
{
    static const Table t = all_kernels<Table>();
    return t;
}

}  // namespace

namespace gemm_relu_hip {
const DtypeKernels& kernels_f16() { return table<DtypeKernels>(); }
const DtypeKernels& kernels_bf16() { return table<DtypeKernels>(); }
const GroupKernels& group_kernels_f16() { return table<GroupKernels>(); }
const GroupKernels& group_kernels_bf16() { return table<GroupKernels>(); }
const StagedKernels& staged_kernels_f16_even() { return table<StagedKernels>(); }
const StagedKernels& staged_kernels_f16_odd() { return table<StagedKernels>(); }
const StagedKernels& staged_kernels_bf16_even() { return table<StagedKernels>(); }
const StagedKernels& staged_kernels_bf16_odd() { return table<StagedKernels>(); }
const BlocksKernels& blocks_kernels_e4m3_e4m3() { return table<BlocksKernels>(); }
const BlocksKernels& blocks_kernels_e4m3_e5m2() { return table<BlocksKernels>(); }
const BlocksKernels& blocks_kernels_e5m2_e4m3() { return table<BlocksKernels>(); }
const BlocksKernels& blocks_kernels_e5m2_e5m2() { return table<BlocksKernels>(); }
const ExpertsKernels& experts_kernels_f16() { return table<ExpertsKernels>(); }
const ExpertsKernels& experts_kernels_bf16() { return table<ExpertsKernels>(); }
const void* quantize_kernel(int, int, int, int) { return &g_kernel; }
const void* zero_fill_kernel() { return &g_kernel; }
}  // namespace gemm_relu_hip

extern "C" {

hipError_t hipGetDevice(int* dev)
{
    *dev = 0;
    return hipSuccess;
}

hipError_t hipGetDeviceProperties(hipDeviceProp_t* prop, int)
{
    std::memset(prop, 0, sizeof(*prop));
    std::strcpy(prop->gcnArchName, "gfx950");
    prop->multiProcessorCount = 256;
    return hipSuccess;
}

hipError_t hipGetSymbolAddress(void**, const void*) { return hipErrorInvalidSymbol; }

hipError_t hipLaunchKernel(const void*, dim3, dim3, void**, size_t, hipStream_t)
{
    std::unique_lock<std::mutex> lock(g_mutex);
    g_log.push_back(t_call);
    g_changed.notify_all();
    // A queue that is full: held calls wait here until they are let go (or 20 s have passed).
    g_changed.wait_for(lock, std::chrono::seconds(20), [] { return g_held != t_call; });
    lock.unlock();
    std::this_thread::sleep_for(std::chrono::microseconds(30));     // others' turn
    return hipSuccess;
}

// Whose launches follow on this thread.
void begin(int call) { t_call = call; }

// The launches of `call` (-1: of none) wait.
void hold(int call)
{
    std::lock_guard<std::mutex> lock(g_mutex);
    g_held = call;
    g_changed.notify_all();
}

// Whether `call` has launched `count` times, within so many seconds.
int launched(int call, int count, double seconds)
{
    std::unique_lock<std::mutex> lock(g_mutex);
    return g_changed.wait_for(lock, std::chrono::duration<double>(seconds), [&] {
        int n = 0;
        for (int c : g_log) n += c == call;
        return n >= count;
    });
}

// The calls of all launches since the last time, in order; returns their number.
int taken(int* calls, int room)
{
    std::lock_guard<std::mutex> lock(g_mutex);
    const int n = (int)g_log.size();
    for (int i = 0; i < n && i < room; ++i) calls[i] = g_log[i];
    g_log.clear();
    return n;
}

}  // extern "C"
