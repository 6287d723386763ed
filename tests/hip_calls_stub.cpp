// Stands in for the HIP calls that a launch makes, on a machine without a GPU: a current device
// that the test sets, the dynamic LDS allowed for each kernel on each device, and a count of
// launches that ask for more than their device allows them (64 KB unless raised).
#include <hip/hip_runtime.h>

#include <map>
#include <string.h>
#include <utility>

namespace {
int device = 0;
std::map<std::pair<int, const void*>, size_t> allowed;
int launches = 0, large = 0, refused = 0;
dim3 g, b;
size_t lds;
hipStream_t on;
}  // namespace

extern "C" {

void stub_set_device(int d) { device = d; }
// launches, those of more than 64 KB, those past what their device allows
void stub_counts(int* out) {
    out[0] = launches;
    out[1] = large;
    out[2] = refused;
}

hipError_t hipGetDevice(int* d) {
    *d = device;
    return hipSuccess;
}
hipError_t hipGetDeviceProperties(hipDeviceProp_t* p, int) {
    memset(p, 0, sizeof(*p));
    strcpy(p->gcnArchName, "gfx950");
    return hipSuccess;
}
hipError_t hipFuncSetAttribute(const void* f, hipFuncAttribute attr, int value) {
    if (attr == hipFuncAttributeMaxDynamicSharedMemorySize) allowed[{device, f}] = static_cast<size_t>(value);
    return hipSuccess;
}
hipError_t hipGetLastError(void) { return hipSuccess; }
hipError_t __hipPushCallConfiguration(dim3 grid, dim3 block, size_t shared, hipStream_t stream) {
    g = grid;
    b = block;
    lds = shared;
    on = stream;
    return hipSuccess;
}
hipError_t __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* shared, hipStream_t* stream) {
    *grid = g;
    *block = b;
    *shared = lds;
    *stream = on;
    return hipSuccess;
}
hipError_t hipLaunchKernel(const void* f, dim3, dim3, void**, size_t shared, hipStream_t) {
    ++launches;
    if (shared > 64 * 1024) {
        ++large;
        const auto it = allowed.find({device, f});
        if (it == allowed.end() || it->second < shared) ++refused;
    }
    return hipSuccess;
}
}
