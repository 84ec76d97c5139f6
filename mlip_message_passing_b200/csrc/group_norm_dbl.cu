#include "group_norm_launch.h"

namespace e3b {
e3_status gn_launch_dbl(const NormArgs& a, const GnConfig& c, bool f64, bool drop, cudaStream_t s) {
  return gn_launch<GN_DBL>(a, c, f64, drop, s);
}
}  // namespace e3b
