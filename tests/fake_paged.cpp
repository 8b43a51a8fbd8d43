// Stand-ins for the paged cache's launchers, for its host code on the fake CUDA
// runtime of fake_cuda.cpp.
#include <cstdarg>

#include "../cross_model_attention_gb300/csrc/mf_internal.cuh"

static int g_calls = 0;
extern "C" __attribute__((visibility("default"))) int fake_paged_launches() { return g_calls; }

namespace mf {
static cudaError_t called() { return ++g_calls, cudaSuccess; }
cudaError_t launch_cache_append(const CacheParams&, long long, int, cudaStream_t) { return called(); }
cudaError_t launch_cache_read(const CacheParams&, long long, int, cudaStream_t) { return called(); }
cudaError_t launch_paged(const PagedParams&, int, cudaStream_t) { return called(); }
void paged_shape(int Lq, int G, int sms, int* grid, int* parts, int* rows) {
  *grid = sms;
  *parts = sms * 16;
  *rows = Lq * G < 16 ? Lq * G : 16;
}
}  // namespace mf
