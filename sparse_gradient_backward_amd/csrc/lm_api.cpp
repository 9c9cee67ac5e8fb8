// lm_api.cpp -- the parts of libsgb_lm.so that no operator owns: call epochs,
// device facts, the status read-back.
#include <atomic>

#include "lm_internal.h"

namespace sgb_lm {

// 24 bits, never 0 (a fresh workspace's likeliest content).
uint32_t next_epoch() {
  static std::atomic<uint32_t> n{0};
  uint32_t e;
  do e = (n.fetch_add(1, std::memory_order_relaxed) + 1) & 0xFFFFFFu;
  while (e == 0);
  return e;
}

int current_device() {
  int d = -1;
  return hipGetDevice(&d) == hipSuccess ? d : -1;
}

int compute_units(int device) {
  int n = 0;
  return hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, device) == hipSuccess &&
                 n > 0
             ? n
             : 256;
}

}  // namespace sgb_lm

extern "C" sgb_status sgb_lm_device_status(const void* workspace, void* stream_, int32_t* out) {
  if (!sgb_lm::workspace_ok(workspace) || !out) return SGB_ERR_INVALID_ARGUMENT;
  hipStream_t stream = reinterpret_cast<hipStream_t>(stream_);
  sgb_lm::Header h{};
  if (hipMemcpyAsync(&h, workspace, sizeof h, hipMemcpyDeviceToHost, stream) != hipSuccess)
    return SGB_ERR_HIP;
  if (hipStreamSynchronize(stream) != hipSuccess) return SGB_ERR_HIP;
  *out = (h.status >> 8) == h.epoch ? (int32_t)(h.status & 0xFFu) : (int32_t)SGB_OK;
  return SGB_OK;
}
