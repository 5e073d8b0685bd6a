// Stands in for the HIP calls that a launch makes, so that a host without a GPU
// can look at the launches themselves: which device was current, which grid,
// how much dynamic LDS, and what limit its kernel had been given on that device.
// Nothing runs; pointers handed to kernels are never followed.
#include <cstddef>
#include <cstdint>
#include <map>
#include <utility>
#include <vector>

namespace {

struct Dim {
  uint32_t x, y, z;
};
struct Launch {
  int device;
  uint64_t threads_x;   // gridDim.x * blockDim.x
  uint64_t blocks_yz;   // the larger of gridDim.y and gridDim.z
  uint64_t lds;         // dynamic, bytes
  uint64_t allowed;     // the kernel's limit on the device, 0 when never set
};

struct Config {   // of the launch being made
  Dim grid, block;
  size_t lds;
  void* stream;
};

int current = 0;
Config pending;
std::map<std::pair<int, const void*>, uint64_t> limits;
std::vector<Launch> launches;

}  // namespace

extern "C" {

int hipGetDevice(int* d) {
  *d = current;
  return 0;
}
int hipGetLastError() { return 0; }
int hipFuncSetAttribute(const void* f, int, int value) {
  limits[{current, f}] = static_cast<uint64_t>(value);
  return 0;
}
int __hipPushCallConfiguration(Dim grid, Dim block, size_t lds, void* stream) {
  pending = {grid, block, lds, stream};
  return 0;
}
int __hipPopCallConfiguration(Dim* grid, Dim* block, size_t* lds, void** stream) {
  *grid = pending.grid;
  *block = pending.block;
  *lds = pending.lds;
  *stream = pending.stream;
  return 0;
}
int hipLaunchKernel(const void* f, Dim grid, Dim block, void**, size_t lds, void*) {
  const auto it = limits.find({current, f});
  launches.push_back({current, uint64_t(grid.x) * block.x, grid.y > grid.z ? grid.y : grid.z, lds,
                      it == limits.end() ? 0 : it->second});
  return 0;
}

void recorder_device(int d) { current = d; }
int recorder_count() { return static_cast<int>(launches.size()); }
void recorder_clear() { launches.clear(); }
uint64_t recorder_threads_x(int i) { return launches[i].threads_x; }
uint64_t recorder_blocks_yz(int i) { return launches[i].blocks_yz; }
uint64_t recorder_lds(int i) { return launches[i].lds; }
uint64_t recorder_allowed(int i) { return launches[i].allowed; }
}
