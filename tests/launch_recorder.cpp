// Stand-ins for the CUDA runtime calls that the state-space layer's host code
// makes, linked in front of the real ones (ld --wrap): nothing is launched,
// what would have been is recorded.  Test infrastructure.
#include <stddef.h>
#include <stdint.h>

#include <mutex>
#include <vector>

struct Dim3 {
    unsigned x, y, z;
};
struct Event {
    const void *kernel;
    long limit;                // cudaFuncSetAttribute's value, or -1 for a launch
    unsigned grid, block;
    size_t shared;
};

static std::vector<Event> events;
static std::mutex lock;

static void add(const Event &e) {
    std::lock_guard<std::mutex> hold(lock);
    events.push_back(e);
}

namespace mdn {
int current_device_status(int **status) {
    static int word;
    *status = &word;
    return 0;
}
}  // namespace mdn

extern "C" {

int __wrap_cudaGetDevice(int *dev) {
    *dev = 0;
    return 0;
}
int __wrap_cudaGetLastError() { return 0; }
int __wrap_cudaMemsetAsync(void *, int, size_t, void *) { return 0; }
int __wrap_cudaFuncSetAttribute(const void *kernel, int, int value) {
    add(Event{kernel, value, 0, 0, 0});
    return 0;
}
int __wrap___cudaGetKernel(const void **kernel, const void *host) {
    *kernel = host;
    return 0;
}
int __wrap___cudaLaunchKernel(const void *kernel, Dim3 grid, Dim3 block, void **, size_t shared, void *) {
    add(Event{kernel, -1, grid.x, block.x, shared});
    return 0;
}

void recorder_clear() { events.clear(); }
int recorder_count() { return (int)events.size(); }
void recorder_event(int i, uint64_t *kernel, long *limit, unsigned *grid, unsigned *block, long *shared) {
    const Event &e = events[i];
    *kernel = (uint64_t)(uintptr_t)e.kernel;
    *limit = e.limit;
    *grid = e.grid;
    *block = e.block;
    *shared = (long)e.shared;
}

}  // extern "C"
