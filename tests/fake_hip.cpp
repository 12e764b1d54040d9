// Stand-ins for the HIP runtime's launch calls, preloaded over it: launches are
// counted and kept by kernel name, their status and an older error of the
// thread are set by a test.  No device is touched.
#include <cstddef>
#include <cstring>
#include <map>
#include <string>

struct Dim3 {
  unsigned x, y, z;
};

static std::map<const void*, std::string>& names() {
  static std::map<const void*, std::string> m;
  return m;
}
static std::string g_log;
static int g_launch = 0, g_older = 0, g_fails_from = 1 << 30, g_count = 0;

extern "C" {
void** __hipRegisterFatBinary(const void*) {
  static void* handle[1];
  return handle;
}
void __hipUnregisterFatBinary(void**) {}
void __hipRegisterVar(void*, void*, char*, char*, int, size_t, int, int) {}
void __hipRegisterFunction(void**, const void* host, char*, const char* name, unsigned, void*, void*, void*, void*,
                           int*) {
  names()[host] = name;
}
static Dim3 g_grid, g_block;
static void* g_stream;
int __hipPushCallConfiguration(Dim3 grid, Dim3 block, size_t, void* stream) {
  g_grid = grid, g_block = block, g_stream = stream;
  return 0;
}
int __hipPopCallConfiguration(Dim3* grid, Dim3* block, size_t* shared, void** stream) {
  *grid = g_grid, *block = g_block, *shared = 0, *stream = g_stream;
  return 0;
}
int hipLaunchKernel(const void* f, Dim3 grid, Dim3 block, void**, size_t, void*) {
  const int status = g_count++ >= g_fails_from ? g_launch : 0;
  if (status) g_older = status;
  g_log += names()[f] + " " + std::to_string(grid.x) + " " + std::to_string(block.x) + "\n";
  return status;
}
int hipGetLastError() {
  const int e = g_older;
  g_older = 0;
  return e;
}

// Launches fail with `status` from the fails_from-th on; `older` is what the
// thread's earlier calls left.
void fake_reset(int older, int status, int fails_from) {
  g_log.clear();
  g_older = older, g_launch = status, g_fails_from = fails_from, g_count = 0;
}
int fake_older() { return g_older; }
const char* fake_log() { return g_log.c_str(); }
}
