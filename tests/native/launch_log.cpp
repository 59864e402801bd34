// The HIP runtime calls that libpe.so makes on its way to a kernel, recorded
// instead of made (no GPU): loaded before libpe.so with its symbols global, it
// is what the library's references bind to.  Every kernel of the library is
// registered by name when it loads; a launch is the name of its kernel and its
// sizes.
#include <cstddef>
#include <cstdint>
#include <cstdio>
#include <map>
#include <string>
#include <vector>

namespace {
struct Dim3 { uint32_t x, y, z; };
struct Config { Dim3 grid, block; size_t lds; void* stream; };

std::map<const void*, std::string>& kernels() {
  static std::map<const void*, std::string> m;
  return m;
}
std::vector<std::string>& launches() {
  static std::vector<std::string> v;
  return v;
}
Config g_config;
std::string g_text;
void* g_module;
}  // namespace

extern "C" {

void** __hipRegisterFatBinary(const void*) { return &g_module; }
void __hipUnregisterFatBinary(void**) {}
void __hipRegisterVar(void**, void*, char*, char*, int, size_t, int, int) {}
void __hipRegisterFunction(void**, const void* host, char*, const char* name, unsigned, void*, void*, void*, void*, int*) {
  kernels()[host] = name;
}
int __hipPushCallConfiguration(Dim3 grid, Dim3 block, size_t lds, void* stream) {
  g_config = Config{grid, block, lds, stream};
  return 0;
}
int __hipPopCallConfiguration(Dim3* grid, Dim3* block, size_t* lds, void** stream) {
  *grid = g_config.grid;
  *block = g_config.block;
  *lds = g_config.lds;
  *stream = g_config.stream;
  return 0;
}
int hipLaunchKernel(const void* f, Dim3 grid, Dim3 block, void**, size_t lds, void*) {
  char sizes[128];
  std::snprintf(sizes, sizeof sizes, " %u %u %u %u %zu", grid.x, grid.y, grid.z, block.x * block.y * block.z, lds);
  launches().push_back(kernels()[f] + sizes);
  return 0;
}
int hipGetDevice(int* d) { *d = 0; return 0; }
int hipSetDevice(int) { return 0; }
int hipGetLastError() { return 0; }

// One line per registered kernel, or per launch since the last call.
const char* launch_log_kernels() {
  g_text.clear();
  for (const auto& k : kernels()) g_text += k.second + "\n";
  return g_text.c_str();
}
const char* launch_log_take() {
  g_text.clear();
  for (const auto& l : launches()) g_text += l + "\n";
  launches().clear();
  return g_text.c_str();
}

}  // extern "C"
