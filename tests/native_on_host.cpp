// The module _fast (csrc/kda_torch.cpp) built for tests without a GPU: it takes
// CPU tensors, and the library's entry points are stand-ins that count their
// calls, keep what they saw and answer the status set by a test.
#include <Python.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ops/empty.h>

#include <utility>

#include "kda_linear.h"
#include "kda_norm.h"

namespace c10::hip {
struct HostStream {
  void* stream() const { return nullptr; }
};
inline DeviceIndex host_device() { return -1; }
inline HostStream host_stream(DeviceIndex) { return {}; }
}  // namespace c10::hip

#define is_cuda is_cpu
#define kCUDA kCPU
#define current_device host_device
#define getCurrentHIPStream host_stream
#include "kda_torch.cpp"

static int g_calls = 0, g_status = 0, g_gil = 0;

static int answer() {
  ++g_calls;
  g_gil += PyGILState_Check();
  return g_status;
}

extern "C" {
int kda_linear_decode(const kda_linear_decode_desc*, void*) { return answer(); }
int kda_linear_prefill(const kda_linear_prefill_desc*, void*, size_t, void*) { return answer(); }
size_t kda_linear_workspace_bytes(const kda_linear_prefill_desc*, int* status) {
  *status = KDA_OK;
  return 64;
}
int kda_gated_norm(const kda_gated_norm_desc*, void*) { return answer(); }
int kda_block_norm(const kda_block_norm_desc*, void*) { return answer(); }

void host_reset(int status) { g_calls = g_gil = 0, g_status = status; }
int host_calls() { return g_calls; }
int host_calls_with_gil() { return g_gil; }
}
