// Host-only stand-ins for the launchers of the gated product, the gated block
// and rotary positions, beside stubs.cpp and stubs_mx.cpp: a launcher that is
// reached counts the call and fails.
#include "../../bit_nf4_quantized_03_amd/csrc/block.h"

extern "C" int qlora_stub_launches;

namespace {
hipError_t reached() {
  ++qlora_stub_launches;
  return hipErrorNotSupported;
}
}  // namespace

namespace qnf4 {
hipError_t launch_mx_pair(const MxPair &, hipStream_t) { return reached(); }
hipError_t launch_mx_gated(const MxLinear &, uint8_t *, uint8_t *, int, bool, hipStream_t) { return reached(); }
hipError_t launch_rope(const Rope &, hipStream_t) { return reached(); }
size_t gated_ws_bytes(int64_t M, int64_t N, int64_t K, int r, bool backward) {
  return static_cast<size_t>((M + N + K) / 64 + r) * (backward ? 32 : 16);
}
hipError_t launch_gated_fwd(const GatedArgs &, const void *, void *, void *, void *, void *, void *, hipStream_t) { return reached(); }
hipError_t launch_gated_bwd(const GatedArgs &, const void *, const void *, const void *, const void *, const void *, void *,
                            void *const (&)[2], void *const (&)[2], void *, hipStream_t) {
  return reached();
}
}  // namespace qnf4
