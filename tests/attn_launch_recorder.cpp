// Stand-ins, beside launch_recorder.cpp's, for what the host code of linear
// attention and the group norm calls: nothing is launched or copied, what would
// have been is recorded.  Test infrastructure.
#define __wrap_cudaMemsetAsync __wrap_unrecorded_cudaMemsetAsync
#include "launch_recorder.cpp"
#undef __wrap_cudaMemsetAsync

#include <cuda.h>

struct Config {                    // cudaLaunchConfig_t's first members
    Dim3 grid, block;
    size_t shared;
};

struct Copy {
    const void *to, *from;         // from: nullptr for zeros
    size_t bytes;
};
static std::vector<Copy> copies;

namespace mdn {
bool make_map_3d(CUtensorMap *, CUtensorMapDataType, const void *, const uint64_t *, const uint64_t *, const uint32_t *) {
    return true;
}
}  // namespace mdn

extern "C" {

int __wrap_cudaLaunchKernelExC(const Config *c, const void *kernel, void **) {
    add(Event{kernel, -1, c->grid.x, c->block.x, c->shared});
    return 0;
}
int __wrap_cudaOccupancyMaxActiveBlocksPerMultiprocessorWithFlags(int *blocks, const void *, int, size_t, unsigned) {
    *blocks = 2;
    return 0;
}
int __wrap_cudaMemcpyAsync(void *to, const void *from, size_t bytes, int, void *) {
    copies.push_back(Copy{to, from, bytes});
    return 0;
}
int __wrap_cudaMemsetAsync(void *to, int, size_t bytes, void *) {
    copies.push_back(Copy{to, nullptr, bytes});
    return 0;
}

void recorder_clear_copies() { copies.clear(); }
int recorder_copies() { return (int)copies.size(); }
void recorder_copy(int i, uint64_t *to, uint64_t *from, uint64_t *bytes) {
    *to = (uint64_t)(uintptr_t)copies[i].to;
    *from = (uint64_t)(uintptr_t)copies[i].from;
    *bytes = copies[i].bytes;
}

}  // extern "C"
