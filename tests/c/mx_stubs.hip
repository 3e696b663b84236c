// Stand-ins for the launchers of routing by a rule and of the microscaled products, linked with
// their ABI file alone for the host sanitizer build: they count the calls that get through.
#include "qmoe_mx_internal.h"

extern "C" int launches;
int launches = 0;

namespace qmoe {

static hipError_t reached() {
  ++launches;
  return hipSuccess;
}

hipError_t launch_route_scored(const void*, int, int, int, int, const moe_route_rule&, const moe_routing*,
                               void*, hipStream_t) {
  return reached();
}
hipError_t launch_mx_quantize(const MxQuantArgs& a, hipStream_t) {
  return a.rows > 0 && a.row_stride * mx_type_size(a.dtype) >= 0 ? reached() : hipErrorUnknown;
}
hipError_t launch_mx_dequantize(const uint8_t*, const uint8_t*, int64_t, void*, int, hipStream_t) {
  return reached();
}
hipError_t launch_mx_linear(const MxLinearArgs& a, hipStream_t) {
  const int64_t last = (a.n - 1) * a.out_stride, from = a.x ? (a.n - 1) * a.row_stride * mx_type_size(a.dtype) : 0;
  return last >= 0 && from >= 0 ? reached() : hipErrorUnknown;
}
hipError_t launch_mx_ffn(const MxFfnArgs& a, hipStream_t) {
  return (a.n - 1) * a.row_stride * mx_type_size(a.dtype) >= 0 ? reached() : hipErrorUnknown;
}

}  // namespace qmoe
