// Host-only stand-ins for the launchers of the microscaled kernels and of
// RMSNorm, beside stubs.cpp: a launcher that is reached counts the call and
// fails.
#include "../../bit_nf4_quantized_03_amd/csrc/mx.h"

extern "C" int qlora_stub_launches;

namespace {
hipError_t reached() {
  ++qlora_stub_launches;
  return hipErrorNotSupported;
}
}  // namespace

namespace qnf4 {
hipError_t launch_mx_quantize(const void *, bool, int64_t, int64_t, int, uint8_t *, uint8_t *, hipStream_t) { return reached(); }
hipError_t launch_mx_dequantize(const uint8_t *, const uint8_t *, int64_t, int64_t, int, void *, bool, hipStream_t) { return reached(); }
hipError_t launch_rms_fwd(const RmsFwd &, hipStream_t) { return reached(); }
size_t rms_bwd_ws_bytes(int64_t rows, int64_t cols) { return rows > 4 ? static_cast<size_t>(rows + cols) * 4 : 0; }
hipError_t launch_rms_bwd(const void *, const void *, const void *, bool, const float *, const void *, int64_t, int64_t, void *, float *,
                          void *, hipStream_t) {
  return reached();
}
hipError_t launch_mx_linear(const MxLinear &, hipStream_t) { return reached(); }
}  // namespace qnf4
