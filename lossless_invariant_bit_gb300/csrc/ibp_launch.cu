// Host-side launch helpers shared by the tensor-core kernels: the tensor-map
// encoder and the kernels' shared-memory limits.
#include <mutex>

#include "ibp_tma.cuh"

namespace ibp {

namespace {
std::mutex g_enc_mu;
EncodeTiledFn g_encode = nullptr;
}  // namespace

EncodeTiledFn encode_tiled() {
  std::lock_guard<std::mutex> lock(g_enc_mu);
  if (!g_encode) {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess || fn == nullptr) {
      cudaGetLastError();
      return nullptr;
    }
    g_encode = reinterpret_cast<EncodeTiledFn>(fn);
  }
  return g_encode;
}

cudaError_t smem_limit(const void* fn, size_t smem) {
  struct Seen {
    const void* fn;
    int dev;
    size_t smem;
  };
  static std::mutex mu;
  static Seen seen[64];
  static int n_seen = 0;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(mu);
  for (int i = 0; i < n_seen; ++i)
    if (seen[i].fn == fn && seen[i].dev == dev && seen[i].smem >= smem) return cudaSuccess;
  const cudaError_t e =
      cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  for (int i = 0; i < n_seen; ++i)
    if (seen[i].fn == fn && seen[i].dev == dev) {
      seen[i].smem = smem;
      return cudaSuccess;
    }
  if (n_seen < 64) seen[n_seen++] = Seen{fn, dev, smem};
  return cudaSuccess;
}

}  // namespace ibp
