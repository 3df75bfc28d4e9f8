// What a call of attention over 8-bit pages enqueues, over launches that only record:
//   paged_stage_host bf16 head_dim kv_heads q_heads n_seqs max_pages n_tokens max_q_tokens room
// for pages of 16 tokens.  Prints the bytes of workspace that the batch makes use of, beyond the
// ordinary ones, and the launches of a call that has `room` bytes beyond them (-1: what it
// makes use of, -2: one less).
#include <cstdio>
#include <string>

#include "paged_fakes_host.h"

namespace {

std::string g_log;

cudaError_t note(const char* what) {
  g_log += std::string(" ") + what;
  return cudaSuccess;
}

}  // namespace

namespace ibp {
cudaError_t launch_paged_resize(const PagedTablesArgs&, int, cudaStream_t) { return note("resize"); }
cudaError_t launch_paged_append(const PagedAppendArgs&, int, cudaStream_t) { return note("append"); }
cudaError_t launch_paged8_append(const PagedAppendArgs&, int, cudaStream_t) { return note("append8"); }
cudaError_t launch_paged_bounds(const PagedGeom&, const PagedBatchView&, uint8_t*, cudaStream_t) {
  return note("bounds");
}
cudaError_t launch_paged8_bounds(const PagedGeom&, const PagedBatchView&, uint8_t*, cudaStream_t) {
  return note("bounds8");
}
cudaError_t launch_paged_scores(const PagedGeom&, const PagedBatchView&, const uint8_t*, uint64_t,
                                uint32_t, const uint8_t*, float*, int, cudaStream_t) {
  return note("scores");
}
cudaError_t launch_paged_select(const PagedGeom&, const PagedBatchView&, const float*, uint32_t,
                                int32_t*, int, cudaStream_t) {
  return note("select");
}
cudaError_t launch_paged_step(const PagedAttnArgs&, const PagedMaps&, int, bool, cudaStream_t) {
  return note("step");
}
cudaError_t launch_paged8_step(const PagedAttnArgs& a, const PagedMaps&, int, bool behind,
                               cudaStream_t) {
  return note(!a.g.k_scales || a.b.table_heads ? "step8?" : behind ? "behind8" : "step8");
}
// (the 16-bit kernel is given the pages that were made, the 8-bit ones the cache's)
cudaError_t launch_paged_chunk(const PagedAttnArgs& a, const PagedMaps&, int, cudaStream_t) {
  const bool made = a.g.k > a.ws && !a.g.k_scales && a.b.table_heads == a.b.max_pages;
  return note(made ? "chunk16" : "chunk16?");
}
cudaError_t launch_paged8_chunk(const PagedAttnArgs& a, const PagedMaps&, int, cudaStream_t) {
  return note(a.g.k_scales && !a.b.table_heads ? "chunk8" : "chunk8?");
}
cudaError_t launch_paged_chunk_join(const PagedAttnArgs&, int, cudaStream_t) { return note("join16"); }
cudaError_t launch_paged8_chunk_join(const PagedAttnArgs&, int, cudaStream_t) { return note("join8"); }
cudaError_t launch_paged8_stage(const PagedAttnArgs& a, const PagedAttnArgs& to, int, cudaStream_t) {
  const uint64_t pages = (uint64_t)a.b.n_seqs * a.b.max_pages;
  const uint64_t kv = pages * a.g.H * a.g.D * 2u << a.g.page_lg;
  const uint8_t* table = reinterpret_cast<const uint8_t*>(to.b.table);
  const bool fits = table == a.ws + IBP_PAGED_WORKSPACE_BYTES && to.g.n_pages == pages &&
                    to.g.k >= table + pages * a.g.H * 4u && to.g.v == to.g.k + kv &&
                    a.g.k_scales && !to.g.k_scales;
  return note(fits ? "stage" : "stage?");
}
}  // namespace ibp

int main(int argc, char** argv) {
  if (argc != 10) return 2;
  const uint32_t bf16 = atoi(argv[1]), D = atoi(argv[2]), H = atoi(argv[3]), Hq = atoi(argv[4]);
  alignas(16) static uint8_t pages[2][64], scales[2][64], q[64], out[64], ws[16];
  static int32_t array[8];
  ibp_paged_desc d = {pages[0], pages[1], 16ull * H * D, D, (uint64_t)H * D, 4, 16, H, D, bf16};
  ibp_paged* cache = nullptr;
  if (ibp_paged_create_8bit(&cache, &d, scales[0], scales[1]) != IBP_OK) return 1;
  const uint32_t max_pages = atoi(argv[6]);
  ibp_paged_batch b = {array,     array, array, max_pages, (uint32_t)atoi(argv[5]),
                       max_pages, (uint32_t)atoi(argv[7]), (uint32_t)atoi(argv[8])};
  uint64_t bytes = 0;
  if (ibp_paged_workspace(cache, &b, Hq, &bytes) != IBP_OK) return 1;
  const uint64_t more = bytes - IBP_PAGED_WORKSPACE_BYTES;
  const long long room = atoll(argv[9]);
  const uint64_t has = room == -1 ? more : room == -2 ? more - 1 : (uint64_t)room;
  if (ibp_paged_attention(cache, &b, q, (uint64_t)Hq * D * 2u, Hq, out, nullptr, 1.f, 1, 0, nullptr,
                          0, ws, IBP_PAGED_WORKSPACE_BYTES + has, nullptr) != IBP_OK)
    return 1;
  printf("%llu%s\n", (unsigned long long)more, g_log.c_str());
  return ibp_paged_destroy(cache) == IBP_OK ? 0 : 1;
}
