// Dropout of whole channels of feature rows from a counter-based generator.
//
// out = keep ? x / (1 - p) : 0 (+ residual).  The mask is a function of (seed, offset, row, block,
// channel), so nothing but x (and the residual) is read and nothing but out is written: the kernel
// is bound by HBM.  A thread keeps one 16-byte column of the rows and walks down them, so the place of
// its column in the irreps layout is worked out once; one generator call (ten rounds, about 70 instructions)
// serves one vector.  Measured (B200, float32): 24000 x 2048 with a residual 97 us = 6.1 TB/s (93% of a copy),
// 1.2 M x 64 scalars 109 us = 5.6 TB/s (86%: one word per value, the generator's instructions show); 400 x 576 in
// 3.3 us.  Four rows in flight per thread and eight CTAs per SM's worth of chunks keep HBM busy.
#include <algorithm>

#include "internal.h"
#include "rows.cuh"

namespace e3b {
namespace {

constexpr int DR_THREADS = 256;
constexpr int DR_UNROLL = 4;  // rows in flight per thread

struct DropoutArgs {
  int64_t N;
  const void* x;
  const void* residual;
  void* out;
  int tx;            // vector columns per CTA
  int64_t rows_cta;  // rows per CTA
  DropArgs drop;
  RowLayout lay;
};

template <typename T, int VEC, bool DROP, bool RES>
__global__ void __launch_bounds__(DR_THREADS) dropout_kernel(const __grid_constant__ DropoutArgs a) {
  const int tx = int(threadIdx.x) % a.tx, ty = int(threadIdx.x) / a.tx, TY = DR_THREADS / a.tx;
  const int col = (int(blockIdx.y) * a.tx + tx) * VEC;
  if (col >= a.lay.dim || ty >= TY) return;
  DropCol<VEC> dc;
  if (DROP) dc.init(a.lay, a.drop, col);
  const T scale = T(a.drop.scale);
  const T* x = static_cast<const T*>(a.x) + col;
  const T* res = static_cast<const T*>(a.residual) + (RES ? col : 0);
  T* out = static_cast<T*>(a.out) + col;
  const int64_t D = a.lay.dim, r0 = int64_t(blockIdx.x) * a.rows_cta, r1 = min(a.N, r0 + a.rows_cta);
  for (int64_t r = r0 + ty; r < r1; r += int64_t(DR_UNROLL) * TY) {
    RowVec<T, VEC> v[DR_UNROLL], q[DR_UNROLL];
#pragma unroll
    for (int i = 0; i < DR_UNROLL; ++i) {
      const int64_t row = r + int64_t(i) * TY;
      if (row < r1) {
        v[i] = load_row<T, VEC>(x + row * D);
        if (RES) q[i] = load_row<T, VEC>(res + row * D);
      }
    }
#pragma unroll
    for (int i = 0; i < DR_UNROLL; ++i) {
      const int64_t row = r + int64_t(i) * TY;
      if (row < r1) {
        const uint32_t keep = DROP ? dc.keep(row) : ~0u;
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const T d = DropCol<VEC>::kept(keep, j) ? (DROP ? v[i].v[j] * scale : v[i].v[j]) : T(0);
          v[i].v[j] = RES ? d + q[i].v[j] : d;
        }
        store_row<T, VEC>(out + row * D, v[i]);
      }
    }
  }
}

template <typename T, int VEC>
void launch_dropout(DropoutArgs& a, bool on, cudaStream_t s) {
  const int cols = a.lay.dim / VEC;
  a.tx = std::min(cols, DR_THREADS);
  const int ny = (cols + a.tx - 1) / a.tx, TY = DR_THREADS / a.tx;
  // about eight CTAs per SM in all, at least one unrolled step each
  const int64_t want = std::max<int64_t>(1, int64_t(8) * sm_count() / ny);
  const int64_t step = int64_t(TY) * DR_UNROLL;
  a.rows_cta = std::max((a.N + want - 1) / want, step);
  a.rows_cta = (a.rows_cta + step - 1) / step * step;
  const dim3 grid(unsigned((a.N + a.rows_cta - 1) / a.rows_cta), unsigned(ny));
  if (on && a.residual)
    dropout_kernel<T, VEC, true, true><<<grid, DR_THREADS, 0, s>>>(a);
  else if (on)
    dropout_kernel<T, VEC, true, false><<<grid, DR_THREADS, 0, s>>>(a);
  else if (a.residual)
    dropout_kernel<T, VEC, false, true><<<grid, DR_THREADS, 0, s>>>(a);
  else
    dropout_kernel<T, VEC, false, false><<<grid, DR_THREADS, 0, s>>>(a);
}

// 16-byte vectors need every row and block to start on one (and so every dropout quad to hold
// whole vectors).
template <typename T>
bool blocks_vectorise(const RowLayout& L) {
  constexpr int VEC = 16 / sizeof(T);
  for (int b = 0; b < L.n_blocks; ++b)
    if (L.blk[b].mul * L.blk[b].d % VEC != 0) return false;
  return true;
}

}  // namespace
}  // namespace e3b

using namespace e3b;

extern "C" e3_status e3_dropout(const e3_features* f, int64_t N, const void* x, const void* residual,
                                const e3_dropout_spec* drop, void* out, void* stream) {
  clear_error();
  e3_status st = check_features_device(f);
  if (st != E3_OK) return st;
  if (N < 0 || N >= (int64_t(1) << 31)) return fail(E3_ERR_SHAPE, "N = %lld", (long long)N);
  DropoutArgs a{};
  bool on = false;
  if ((st = drop_args(drop, N, &a.drop, &on)) != E3_OK) return st;
  if (N == 0) return E3_OK;
  if (x == nullptr || out == nullptr) return fail(E3_ERR_INVALID_ARG, "x or out is NULL");
  const void* ptrs[3] = {x, residual, out};
  for (const void* p : ptrs)
    if (reinterpret_cast<uintptr_t>(p) & 15u) return fail(E3_ERR_INVALID_ARG, "a pointer is not 16-byte aligned");
  if ((st = ensure_device_tables()) != E3_OK) return st;
  a.N = N;
  a.x = x;
  a.residual = residual;
  a.out = out;
  a.lay = f->lay;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (f->dtype == E3_F32) {
    if (blocks_vectorise<float>(f->lay)) launch_dropout<float, 4>(a, on, s);
    else launch_dropout<float, 1>(a, on, s);
  } else {
    if (blocks_vectorise<double>(f->lay)) launch_dropout<double, 2>(a, on, s);
    else launch_dropout<double, 1>(a, on, s);
  }
  const cudaError_t err = cudaGetLastError();
  if (err != cudaSuccess) return fail(E3_ERR_CUDA, "dropout launch failed: %s", cudaGetErrorString(err));
  return E3_OK;
}
