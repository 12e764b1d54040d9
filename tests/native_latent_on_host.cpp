// The module _fast_latent (csrc/kda_latent_torch.cpp) built for tests without a GPU: it
// takes CPU tensors, and the library's entry points are stand-ins that count their
// calls, keep the descriptors they saw and answer the status set by a test.
#include <Python.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ops/empty.h>

#include <cstring>
#include <utility>

#include "kda_latent.h"
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
#include "kda_latent_torch.cpp"

static int g_calls = 0, g_status = 0, g_gil = 0;
static size_t g_workspace = 0;
static unsigned char g_seen[512];

template <typename Desc>
static int answer(const Desc* d) {
  static_assert(sizeof(Desc) <= sizeof(g_seen), "");
  ++g_calls;
  g_gil += PyGILState_Check();
  std::memcpy(g_seen, d, sizeof(Desc));
  return g_status;
}

extern "C" {
int kda_latent_attend(const kda_latent_attend_desc* d, void*, size_t bytes, void*) {
  g_workspace = bytes;
  return answer(d);
}
size_t kda_latent_workspace_bytes(const kda_latent_attend_desc*, int* status) {
  *status = KDA_OK;
  return 64;
}
int kda_latent_prefill(const kda_latent_prefill_desc* d, void*, size_t bytes, void*) {
  g_workspace = bytes;
  return answer(d);
}
size_t kda_latent_prefill_workspace_bytes(const kda_latent_prefill_desc* d, int* status) {
  *status = d->dn == 8 ? KDA_ERR_UNSUPPORTED : KDA_OK;
  return d->k_total == d->q_total ? 0 : 32;
}
int kda_latent_append(const kda_latent_append_desc* d, void*) { return answer(d); }
int kda_rotary(const kda_rotary_desc* d, void*) { return answer(d); }

void host_reset(int status) { g_calls = g_gil = 0, g_status = status, g_workspace = 0; }
int host_calls() { return g_calls; }
int host_calls_with_gil() { return g_gil; }
size_t host_workspace() { return g_workspace; }
const void* host_seen() { return g_seen; }
}
