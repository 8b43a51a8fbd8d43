// Stand-ins for the CUDA runtime and for the library's launchers, for host
// code that is compiled with them and tested without a GPU: device memory is
// host memory, and what matters of each call is written to a log.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <string>

#include "../cross_model_attention_gb300/csrc/mf_handle.h"

static int g_device = 0, g_launches = 0;
static cudaError_t g_sync = cudaSuccess;
static std::string g_log, g_error;

static void say(const char* what) { g_log += std::string(what) + std::to_string(g_device) + " "; }

#define FAKE extern "C" __attribute__((visibility("default")))
FAKE void fake_device(int dev) { g_device = dev; }
FAKE int fake_current() { return g_device; }
FAKE void fake_sync_returns(int e) { g_sync = static_cast<cudaError_t>(e); }
FAKE int fake_launches() { return g_launches; }
FAKE const char* fake_log() {
  static std::string last;
  last.swap(g_log);
  g_log.clear();
  return last.c_str();
}

extern "C" {
cudaError_t cudaGetDevice(int* d) { return *d = g_device, cudaSuccess; }
cudaError_t cudaSetDevice(int d) { return g_device = d, cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr, int) { return *v = 152, cudaSuccess; }
cudaError_t cudaMallocAsync(void** p, size_t n, cudaStream_t) { return say("alloc"), *p = std::malloc(n), cudaSuccess; }
cudaError_t cudaFreeAsync(void* p, cudaStream_t) { return say("free"), std::free(p), cudaSuccess; }
cudaError_t cudaMallocHost(void** p, size_t n) { return say("pin"), *p = std::malloc(n), cudaSuccess; }
cudaError_t cudaFreeHost(void* p) { return say("unpin"), std::free(p), cudaSuccess; }
cudaError_t cudaMemcpy(void* d, const void* s, size_t n, cudaMemcpyKind) { return __builtin_memcpy(d, s, n), cudaSuccess; }
cudaError_t cudaMemcpyAsync(void* d, const void* s, size_t n, cudaMemcpyKind, cudaStream_t) { return __builtin_memcpy(d, s, n), cudaSuccess; }
cudaError_t cudaMemset(void* d, int v, size_t n) { return __builtin_memset(d, v, n), cudaSuccess; }
cudaError_t cudaMemsetAsync(void* d, int v, size_t n, cudaStream_t) { return __builtin_memset(d, v, n), cudaSuccess; }
cudaError_t cudaDeviceSynchronize() { return say("sync"), g_sync; }
cudaError_t cudaStreamSynchronize(cudaStream_t) { return cudaSuccess; }
cudaError_t cudaEventDestroy(cudaEvent_t) { return cudaSuccess; }
cudaError_t cudaGetLastError() { return cudaSuccess; }
const char* cudaGetErrorString(cudaError_t) { return "fake"; }
}

#ifndef FAKE_RUNTIME_ONLY
extern "C" const char* mf_last_error(void) { return g_error.c_str(); }
namespace mf {
int fail(int code, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  std::vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  g_error = buf;
  return code;
}
int cuda_fail(cudaError_t, const char* what) { return fail(MF_ERR_CUDA, "%s", what); }
int make_map(CUtensorMap*, const void*, uint64_t, uint64_t, uint64_t, uint32_t, uint32_t, CUtensorMapSwizzle) { return MF_OK; }
int make_map4(CUtensorMap*, const void*, const uint64_t*, const uint64_t*, const uint32_t*) { return MF_OK; }
static cudaError_t launched() { return ++g_launches, cudaSuccess; }
cudaError_t launch_rope(const RopeParams&, long long, int, int, cudaStream_t) { return launched(); }
cudaError_t launch_attn_packed(const AttnParams&, int, int, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&, cudaStream_t) { return launched(); }
cudaError_t launch_attn_join(const AttnParams&, int, const AttnJoin*, int, cudaStream_t) { return launched(); }
cudaError_t launch_attn_cache(const AttnParams&, int, int, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&,
                              const CUtensorMap&, const CUtensorMap&, const CUtensorMap&, cudaStream_t) { return launched(); }
}  // namespace mf
#endif
