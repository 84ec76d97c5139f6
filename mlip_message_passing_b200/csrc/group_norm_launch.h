// Launch configuration of the group norm and its per-form launchers (one translation unit each).
#pragma once

#include "group_norm.cuh"

namespace e3b {

struct GnConfig {
  bool local = false;
  int vec = 1;
  int64_t col_parts = 0;  // slots of colpart
  dim3 grid;              // local kernel, or both passes of split
  // workspace layout (bytes)
  size_t part = 0, coef = 0, colpart = 0, total = 0;
};
// rows of a segment that a thread of the local kernel keeps in registers
__host__ __device__ constexpr int gn_reg_rows(int op) { return op == GN_DBL ? 4 : 8; }

e3_status gn_launch_fwd(const NormArgs& a, const GnConfig& c, bool f64, bool drop, cudaStream_t s);
e3_status gn_launch_bwd(const NormArgs& a, const GnConfig& c, bool f64, bool drop, cudaStream_t s);
e3_status gn_launch_dbl(const NormArgs& a, const GnConfig& c, bool f64, bool drop, cudaStream_t s);

template <typename T, int VEC, int OP, bool DROP>
void gn_run(const NormArgs& a, const GnConfig& c, cudaStream_t s) {
  if (c.local) {
    gn_local_kernel<T, VEC, OP, DROP, gn_reg_rows(OP)><<<c.grid, GN_THREADS, 0, s>>>(a);
    return;
  }
  gn_partial_kernel<T, VEC, OP, DROP><<<c.grid, GN_THREADS, 0, s>>>(a);
  const int64_t warps = int64_t(a.B) * a.lay.n_groups();
  gn_final_kernel<OP, VEC><<<unsigned((warps * 32 + GN_THREADS - 1) / GN_THREADS), GN_THREADS, 0, s>>>(a);
  if (OP != GN_BWD || a.o0 != nullptr) gn_apply_kernel<T, VEC, OP, DROP><<<c.grid, GN_THREADS, 0, s>>>(a);
}

template <int OP>
e3_status gn_launch(const NormArgs& a, const GnConfig& c, bool f64, bool drop, cudaStream_t s) {
#define GN_CASE(T, V) (drop ? gn_run<T, V, OP, true>(a, c, s) : gn_run<T, V, OP, false>(a, c, s))
  if (f64) {
    if (c.vec == 2) GN_CASE(double, 2);
    else GN_CASE(double, 1);
  } else {
    if (c.vec == 4) GN_CASE(float, 4);
    else GN_CASE(float, 1);
  }
#undef GN_CASE
  const cudaError_t err = cudaGetLastError();
  if (err != cudaSuccess) return fail(E3_ERR_CUDA, "group norm launch failed: %s", cudaGetErrorString(err));
  return E3_OK;
}

}  // namespace e3b
