// The C entry point of the page tables over a launch and a CUDA runtime that only record: in
// which order calls of several threads are enqueued.
//   paged_tables_host threads   two threads, the same tables
//   paged_tables_host apart     two threads, tables each
// Prints "whole" when a call's launches follow one another, "mixed" if not.
#include <unistd.h>

#include <atomic>
#include <cstdio>
#include <cstring>
#include <mutex>
#include <thread>
#include <vector>

#include "paged_fakes_host.h"

namespace {

std::mutex g_mu;
std::vector<const void*> g_log;  // a call's q_starts, for each of its two launches

void note(const void* call) {
  {
    std::lock_guard<std::mutex> lock(g_mu);
    g_log.push_back(call);
  }
  usleep(200);  // the time of a launch, and room for the other thread
}

}  // namespace

namespace ibp {
cudaError_t launch_paged_resize(const PagedTablesArgs& a, int, cudaStream_t) {
  note(a.q_starts);
  note(a.q_starts);
  return cudaSuccess;
}
#define NOTHING(name, ...) \
  cudaError_t name(__VA_ARGS__) { return cudaSuccess; }
NOTHING(launch_paged_append, const PagedAppendArgs&, int, cudaStream_t)
NOTHING(launch_paged8_append, const PagedAppendArgs&, int, cudaStream_t)
NOTHING(launch_paged_bounds, const PagedGeom&, const PagedBatchView&, uint8_t*, cudaStream_t)
NOTHING(launch_paged8_bounds, const PagedGeom&, const PagedBatchView&, uint8_t*, cudaStream_t)
NOTHING(launch_paged_scores, const PagedGeom&, const PagedBatchView&, const uint8_t*, uint64_t,
        uint32_t, const uint8_t*, float*, int, cudaStream_t)
NOTHING(launch_paged_select, const PagedGeom&, const PagedBatchView&, const float*, uint32_t,
        int32_t*, int, cudaStream_t)
NOTHING(launch_paged_step, const PagedAttnArgs&, const PagedMaps&, int, bool, cudaStream_t)
NOTHING(launch_paged8_step, const PagedAttnArgs&, const PagedMaps&, int, bool, cudaStream_t)
NOTHING(launch_paged_chunk, const PagedAttnArgs&, const PagedMaps&, int, cudaStream_t)
NOTHING(launch_paged8_chunk, const PagedAttnArgs&, const PagedMaps&, int, cudaStream_t)
NOTHING(launch_paged_chunk_join, const PagedAttnArgs&, int, cudaStream_t)
NOTHING(launch_paged8_chunk_join, const PagedAttnArgs&, int, cudaStream_t)
NOTHING(launch_paged8_stage, const PagedAttnArgs&, const PagedAttnArgs&, int, cudaStream_t)
}  // namespace ibp

int main(int argc, char** argv) {
  const bool shared = argc > 1 && !strcmp(argv[1], "threads");
  alignas(16) static uint8_t pages[2][64], scales[2][8];
  alignas(16) static int32_t table[8], lens[2], free_pages[4], state[2][64], target[2], starts[2][4];
  alignas(16) static int64_t slots[8];
  ibp_paged_desc d = {pages[0], pages[1], 16 * 2 * 64, 64, 128, 4, 16, 2, 64, 0};
  ibp_paged* cache = nullptr;
  if (ibp_paged_create_8bit(&cache, &d, scales[0], scales[1]) != IBP_OK) return 1;
  std::atomic<int> failed{0}, ready{0};
  auto calls = [&](int i) {
    ibp_paged_tables t = {table, lens, free_pages, state[shared ? 0 : i], 4, 2, 4};
    ++ready;
    while (ready < 2) {}
    for (int k = 0; k < 40; ++k)
      if (ibp_paged_resize(cache, &t, target, starts[i], slots, 8, nullptr) != IBP_OK) ++failed;
  };
  std::thread t0(calls, 0), t1(calls, 1);
  t0.join();
  t1.join();
  if (failed || g_log.size() != 2 * 40 * 2) return 1;
  bool whole = true;
  for (size_t i = 0; i < g_log.size(); ++i) whole = whole && g_log[i] == g_log[i / 2 * 2];
  puts(whole ? "whole" : "mixed");
  return ibp_paged_destroy(cache) == IBP_OK ? 0 : 1;
}
