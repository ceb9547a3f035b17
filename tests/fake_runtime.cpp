// A stand-in for the CUDA runtime, linked with the row operators' host code: it runs nothing, keeps a list of what was
// asked of it, and fails the call that a test names.
#include <cuda_runtime.h>

#include <map>
#include <mutex>
#include <string>
#include <vector>

namespace prism {
void note_launches(int) {}
}  // namespace prism

namespace {
struct Event {
    int kind;                 // 0: a launch, 1: a kernel's shared-memory limit, 2: a memset
    std::string kernel;
    size_t bytes;             // shared memory of the launch, the limit, the bytes cleared
    unsigned grid[3], block[3];
};
std::vector<Event> g_events;
std::map<const void*, std::string> g_names;
std::mutex g_names_lock;
int g_fail = -1;              // calls until one fails; -1: none does
cudaError_t g_last = cudaSuccess;
struct Config {
    dim3 grid, block;
    size_t shared;
    void* stream;
} g_config;

cudaError_t done(Event e) {
    g_events.push_back(std::move(e));
    if (g_fail < 0 || g_fail-- != 0) return cudaSuccess;
    return g_last = cudaErrorInvalidValue;
}
}  // namespace

extern "C" {
void** __cudaRegisterFatBinary(void*) {
    static void* handle[8];
    return handle;
}
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
void __cudaRegisterFunction(void**, const char* host, char*, const char* name, int, uint3*, uint3*, dim3*, dim3*, int*) {
    std::lock_guard<std::mutex> l(g_names_lock);
    g_names[host] = name;
}
unsigned __cudaPushCallConfiguration(dim3 grid, dim3 block, size_t shared, void* stream) {
    g_config = {grid, block, shared, stream};
    return 0;
}
cudaError_t __cudaPopCallConfiguration(dim3* grid, dim3* block, size_t* shared, void* stream) {
    *grid = g_config.grid;
    *block = g_config.block;
    *shared = g_config.shared;
    *(void**)stream = g_config.stream;
    return cudaSuccess;
}
cudaError_t cudaLaunchKernel(const void* f, dim3 g, dim3 b, void**, size_t shared, cudaStream_t) {
    return done({0, g_names[f], shared, {g.x, g.y, g.z}, {b.x, b.y, b.z}});
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void**) {
    return done({0, g_names[f], c->dynamicSmemBytes, {c->gridDim.x, c->gridDim.y, c->gridDim.z},
                 {c->blockDim.x, c->blockDim.y, c->blockDim.z}});
}
cudaError_t cudaFuncSetAttribute(const void* f, cudaFuncAttribute, int value) {
    return done({1, g_names[f], (size_t)value, {0, 0, 0}, {0, 0, 0}});
}
cudaError_t cudaMemsetAsync(void*, int, size_t n, cudaStream_t) { return done({2, "", n, {0, 0, 0}, {0, 0, 0}}); }
cudaError_t cudaGetLastError(void) {
    const cudaError_t e = g_last;
    g_last = cudaSuccess;
    return e;
}

// what a test asks
void fake_reset(int fail) {
    g_events.clear();
    g_fail = fail;
    g_last = cudaSuccess;
}
int fake_count(void) { return (int)g_events.size(); }
int fake_last_error(void) { return (int)g_last; }
int fake_event(int i, const char** kernel, unsigned long long* bytes, unsigned* dims) {
    const Event& e = g_events[i];
    *kernel = e.kernel.c_str();
    *bytes = e.bytes;
    for (int k = 0; k < 3; ++k) {
        dims[k] = e.grid[k];
        dims[3 + k] = e.block[k];
    }
    return e.kind;
}
}
