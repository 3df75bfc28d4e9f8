// The C entry points of the paged K/V cache over launches and a CUDA runtime that only
// record: what a call enqueues, and in which order calls of several threads do.
//   paged_calls_host threads   two threads, one workspace and stream
//   paged_calls_host apart     two threads, a workspace each
// Prints "whole" when the launches of each call follow one another, "mixed" if not.
#include <unistd.h>

#include <atomic>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <mutex>
#include <thread>
#include <vector>

#include "ibp_paged.cuh"
#include "ibp_tma.cuh"

namespace {

struct Launch {
  const void* workspace;
  const void* out;  // tells the call
  int stage;
};
std::mutex g_mu;
std::vector<Launch> g_log;

cudaError_t note(const ibp::PagedAttnArgs& a, int stage) {
  {
    std::lock_guard<std::mutex> lock(g_mu);
    g_log.push_back({a.ws, a.out, stage});
  }
  usleep(200);  // the time of a launch, and room for the other thread
  return cudaSuccess;
}

CUresult encode(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill) {
  return CUDA_SUCCESS;
}

}  // namespace

namespace ibp {
EncodeTiledFn encode_tiled() { return &encode; }
cudaError_t launch_paged_chunk(const PagedAttnArgs& a, const PagedMaps&, int, cudaStream_t) {
  return note(a, 0);
}
cudaError_t launch_paged_step(const PagedAttnArgs& a, const PagedMaps&, int, bool, cudaStream_t) {
  note(a, 1);
  return note(a, 2);  // and its join
}
cudaError_t launch_paged_chunk_join(const PagedAttnArgs& a, int, cudaStream_t) {
  return note(a, 3);
}
cudaError_t launch_paged_append(const PagedAppendArgs&, int, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_paged_bounds(const PagedGeom&, const PagedBatchView&, uint8_t*, cudaStream_t) {
  return cudaSuccess;
}
cudaError_t launch_paged_scores(const PagedGeom&, const PagedBatchView&, const uint8_t*, uint64_t,
                                uint32_t, const uint8_t*, float*, int, cudaStream_t) {
  return cudaSuccess;
}
cudaError_t launch_paged_select(const PagedGeom&, const PagedBatchView&, const float*, uint32_t,
                                int32_t*, int, cudaStream_t) {
  return cudaSuccess;
}
}  // namespace ibp

// the runtime, on host memory
extern "C" {
cudaError_t cudaMalloc(void** p, size_t n) { return (*p = malloc(n)) ? cudaSuccess : cudaErrorMemoryAllocation; }
cudaError_t cudaFree(void* p) { return free(p), cudaSuccess; }
cudaError_t cudaMemset(void* p, int v, size_t n) { return memset(p, v, n), cudaSuccess; }
cudaError_t cudaMemsetAsync(void* p, int v, size_t n, cudaStream_t) { return memset(p, v, n), cudaSuccess; }
cudaError_t cudaMemcpyAsync(void* d, const void* s, size_t n, cudaMemcpyKind, cudaStream_t) {
  return memcpy(d, s, n), cudaSuccess;
}
cudaError_t cudaStreamSynchronize(cudaStream_t) { return cudaSuccess; }
cudaError_t cudaGetLastError(void) { return cudaSuccess; }
cudaError_t cudaGetDevice(int* d) { return *d = 0, cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr, int) { return *v = 152, cudaSuccess; }
}

int main(int argc, char** argv) {
  const bool shared = argc > 1 && !strcmp(argv[1], "threads");
  alignas(16) static uint8_t pages[2][64], q[64], out[2][64], ws[2][16];
  static int32_t array[8];
  ibp_paged_desc d = {pages[0], pages[1], 16 * 2 * 64 * 2, 128, 256, 4, 16, 2, 64, 0};
  ibp_paged* cache = nullptr;
  if (ibp_paged_create(&cache, &d) != IBP_OK) return 1;
  // a batch that needs every kernel
  ibp_paged_batch b = {array, array, array, 4, 2, 4, 40, 39};
  std::atomic<int> failed{0}, ready{0};
  auto calls = [&](int i) {
    ++ready;
    while (ready < 2) {}
    for (int k = 0; k < 20; ++k)
      if (ibp_paged_attention(cache, &b, q, 4 * 128, 4, out[i], nullptr, 1.f, 1, 0, nullptr, 0,
                              ws[shared ? 0 : i], IBP_PAGED_WORKSPACE_BYTES, nullptr) != IBP_OK)
        ++failed;
  };
  std::thread t0(calls, 0), t1(calls, 1);
  t0.join();
  t1.join();
  if (failed || g_log.size() != 2 * 20 * 4) return 1;
  bool whole = true;
  for (size_t i = 0; i < g_log.size(); ++i) {
    if (g_log[i].stage != (int)(i % 4)) whole = false;
    if (g_log[i].out != g_log[i / 4 * 4].out) whole = false;
  }
  puts(whole ? "whole" : "mixed");
  return ibp_paged_destroy(cache) == IBP_OK ? 0 : 1;
}
