#include "group_norm_launch.h"

namespace e3b {
e3_status gn_launch_dbl(NormArgs& a, const GnConfig& c, bool f64, int vec, bool drop, void* ws, cudaStream_t s) {
  return gn_launch<GN_DBL>(a, c, f64, vec, drop, ws, s);
}
}  // namespace e3b
