// Per-device state of the transformer-block operators and the call that
// reads its error word.
#include <mutex>

#include "blocks.cuh"

namespace prm {
namespace {
std::mutex g_mutex;
BlockDevice g_devices[64];
}  // namespace

int block_device(const BlockDevice** out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return PRM_ERR_CUDA;
  std::lock_guard<std::mutex> lock(g_mutex);
  BlockDevice& d = g_devices[dev];
  if (!d.ready) {
    int major = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&d.num_sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return PRM_ERR_CUDA;
    if (major != 10) return PRM_ERR_UNSUPPORTED;
    if (d.d_err == nullptr && cudaMalloc(reinterpret_cast<void**>(&d.d_err), sizeof(int)) != cudaSuccess)
      return PRM_ERR_CUDA;
    if (cudaMemset(d.d_err, 0, sizeof(int)) != cudaSuccess) return PRM_ERR_CUDA;
    d.ready = true;
  }
  *out = &d;
  return PRM_OK;
}

}  // namespace prm

extern "C" int prm_blocks_sync_status(void* stream) {
  using namespace prm;
  const BlockDevice* d;
  const int rc = block_device(&d);
  if (rc != PRM_OK) return rc;
  if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return PRM_ERR_CUDA;
  int word = 0;
  if (cudaMemcpy(&word, d->d_err, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess) return PRM_ERR_CUDA;
  if (word == 0) return PRM_OK;
  cudaMemset(d->d_err, 0, sizeof(int));
  return PRM_ERR_TIMEOUT;
}
