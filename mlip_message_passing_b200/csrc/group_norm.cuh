// Group norm of feature rows: kernels shared by the forward, the backward and the double backward.
//
// Mathematics (one segment, one group of n values; even scalars are centred, other irreps are not):
//   z = (x - mu) r,  t = w z + b,  y = m a(t)      (m: dropout factor, a: activation)
//   first derivative:   h = m g a'(t), c = w h,  dx = r (c - mean(c) - z mean(c z)),
//                       dw = sum h z, db = sum h
//   second derivative:  zd = r (u - m1 - z m2), m1 = mean(u), m2 = mean(z u), td = w zd + uw z + ub,
//                       dg = m a'(t) td, q = m g a''(t) td, db = sum q, dw = sum (q z + h zd),
//                       C = w q + uw h - r m2 c - r mean(c z) u,
//                       dx = r (C - mean(C) - z mean(z C)) - r z mean(c zd)
// with mean(c), m1 and mean(C) taken as 0 for irreps that are not centred.  q depends on m1 and m2,
// but linearly, so all the means follow from twelve sums that one pass over (x, g, u) collects.
//
// Every form is two passes over the rows: sums, then the pointwise result.  Nothing else is
// O(N dim), so the kernels are bound by memory; what matters is that the second pass finds the rows
// on chip.  Two variants:
//   local  a CTA holds a whole segment x some whole groups in registers between the passes (one
//          read); longer segments are read again (from L2);
//   split  long segments: row chunks x column tiles write partial sums, a small kernel joins them,
//          a second pass reads the rows again.
// Partial sums: the rows' type over at most GN_FLUSH rows of a thread, double from there on, joined in
// a fixed order.  A thread's variance sum is taken around its own first value: (pivot - mean)^2 is a
// term of the true sum, so the cancellation costs at most the thread's number of values in
// epsilons, whatever the offset of the data.
#pragma once

#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "internal.h"
#include "rows.cuh"

namespace e3b {

constexpr int GN_THREADS = 256;
constexpr int GN_FLUSH = 64;
constexpr int GN_MAXSLAB = 64;
enum GnOp { GN_FWD = 0, GN_BWD = 1, GN_DBL = 2 };
// sums a thread publishes: forward (mean, M2, count), backward (sum c, sum c z), double backward 12
__host__ __device__ constexpr int gn_sums(int op) { return op == GN_FWD ? 3 : op == GN_BWD ? 2 : 12; }
// values a (segment, group) needs in the second pass besides (mu, r)
__host__ __device__ constexpr int gn_coefs(int op) { return op == GN_FWD ? 2 : op == GN_BWD ? 2 : 6; }

struct NormArgs {
  int64_t N;
  int32_t B;
  const int32_t* row_ptr;  // NULL: one segment of all rows
  const void *x, *g, *u;   // rows: features, grad_y, u_x (may be NULL)
  const void *w, *b, *uw, *ub;
  void *o0, *o1;           // y | grad_x | d_x ; d_grad_y (each may be NULL in the backwards)
  double* stats;           // [B][groups][2]
  double* part;            // split: [chunks + B][groups + tiles][sums]
  double* coef;            // split: [B][groups][coefs]
  double* colpart;         // [col_parts][2][dim]: sums for dw, db per column (NULL: not wanted)
  double eps;
  int32_t act;
  int* status;
  int32_t tx, k, j, lanes;  // thread layout: columns, row lanes of a segment, segments, lanes of a join
  int32_t n_tiles;          // split: column tiles of tx vectors
  int64_t rows_cta;         // split: rows of a chunk
  int64_t n_chunks;
  int32_t n_slabs;          // local: slabs of whole groups, first vector column of each
  int32_t slab[GN_MAXSLAB + 1];
  DropArgs drop;
  RowLayout lay;
};

// Rows [s, e) of segment b, clamped into [0, N); a bad row pointer is recorded.
__device__ __forceinline__ void gn_segment(const NormArgs& a, int64_t b, int64_t& s, int64_t& e) {
  if (a.row_ptr == nullptr) {
    s = 0;
    e = a.N;
    return;
  }
  s = a.row_ptr[b];
  e = a.row_ptr[b + 1];
  if (s < 0 || e < s || e > a.N || (b == 0 && s != 0)) {
    atomicCAS(a.status, 0, int(E3_ERR_INDEX));
    s = min(max(s, int64_t(0)), a.N);
    e = min(max(e, s), a.N);
  }
}
// First padding row.
__device__ __forceinline__ int64_t gn_rows_end(const NormArgs& a) {
  return a.row_ptr == nullptr ? a.N : min(max(int64_t(a.row_ptr[a.B]), int64_t(0)), a.N);
}

template <typename T>
struct GnStat {
  T hi, lo, r;  // mu = hi + lo
  __device__ __forceinline__ void set(double mu, double rs) {
    hi = T(mu);
    lo = T(mu - double(hi));
    r = T(rs);
  }
  __device__ __forceinline__ T z(T x) const { return ((x - hi) - lo) * r; }
};

__device__ __forceinline__ float gn_sigmoid(float t) { return __fdividef(1.f, 1.f + expf(-t)); }
__device__ __forceinline__ double gn_sigmoid(double t) { return 1.0 / (1.0 + exp(-t)); }

// What a thread knows of its vector column.
template <typename T, int VEC, int OP, bool DROP>
struct GnCol {
  int col, g, lg, g0, g1;  // first column, group, group within the CTA, its vector range in the CTA
  bool scalar, act;
  T w[VEC], b[VEC], uw[VEC], ub[VEC];
  DropCol<VEC> dc;
  T scale;

  __device__ __forceinline__ void init(const NormArgs& a, int v0, int width, int tx) {
    const RowLayout& L = a.lay;
    col = (v0 + tx) * VEC;
    const int bi = block_of(L, col);
    const RowBlock& k = L.blk[bi];
    const int gi = (col - k.col0) / k.group_cols, gc = k.col0 + gi * k.group_cols;
    g = bi * L.groups + gi;
    lg = g - group_of(L, v0 * VEC);
    g0 = max(gc / VEC - v0, 0);
    g1 = min((gc + k.group_cols) / VEC - v0, width);
    scalar = k.bias0 >= 0;
    act = scalar && a.act == E3_ACT_SILU;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const int u = (col + i - k.col0) / k.d;
      w[i] = a.w ? static_cast<const T*>(a.w)[k.chan0 + u] : T(1);
      b[i] = scalar && a.b ? static_cast<const T*>(a.b)[k.bias0 + u] : T(0);
      if (OP == GN_DBL) {
        uw[i] = a.uw ? static_cast<const T*>(a.uw)[k.chan0 + u] : T(0);
        ub[i] = scalar && a.ub ? static_cast<const T*>(a.ub)[k.bias0 + u] : T(0);
      }
    }
    if (DROP) {
      dc.init(L, a.drop, col);
      scale = T(a.drop.scale);
    }
  }
  __device__ __forceinline__ uint32_t keep(int64_t row) const { return DROP ? dc.keep(row) : ~0u; }
  __device__ __forceinline__ T drop(uint32_t kp, int i, T v) const {
    return DROP ? ((kp >> i & 1u) ? v * scale : T(0)) : v;
  }
};

// The sums of one thread over the rows of one segment.
template <typename T, int VEC, int OP, bool DROP>
struct GnAcc;

template <typename T, int VEC, bool DROP>
struct GnAcc<T, VEC, GN_FWD, DROP> {
  T piv, s1[VEC], s2[VEC];
  double S1, S2;
  int64_t rows;
  __device__ __forceinline__ void start() {
    S1 = S2 = 0.0;
    rows = 0;
    piv = T(0);
    clear();
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < VEC; ++i) s1[i] = s2[i] = T(0);
  }
  template <typename COL>
  __device__ __forceinline__ void add(const COL& c, const GnStat<T>&, RowVec<T, VEC>& x, RowVec<T, VEC>&,
                                      const RowVec<T, VEC>&, int64_t) {
    if (rows == 0 && c.scalar) piv = x.v[0];
    ++rows;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const T d = x.v[i] - piv;
      s1[i] += d;
      s2[i] += d * d;
    }
  }
  template <typename COL>
  __device__ __forceinline__ void flush(const COL&, double*, double*) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      S1 += double(s1[i]);
      S2 += double(s2[i]);
    }
    clear();
  }
  template <typename COL>
  __device__ __forceinline__ void publish(const COL& c, double* buf) const {
    const double n = double(rows) * VEC;
    // centred groups: (mean, sum of squares around it, count); others: (0, sum of squares, count)
    const double m = c.scalar && rows > 0 ? S1 / n : 0.0;
    buf[0] = c.scalar ? double(piv) + m : 0.0;
    buf[GN_THREADS] = c.scalar ? S2 - m * S1 : S2;
    buf[2 * GN_THREADS] = n;
  }
};

template <typename T, int VEC, bool DROP>
struct GnAcc<T, VEC, GN_BWD, DROP> {
  T cw[VEC], cb[VEC];
  double S1, S2;
  __device__ __forceinline__ void start() {
    S1 = S2 = 0.0;
    clear();
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < VEC; ++i) cw[i] = cb[i] = T(0);
  }
  // x becomes z, g becomes c = w h
  template <typename COL>
  __device__ __forceinline__ void add(const COL& c, const GnStat<T>& st, RowVec<T, VEC>& x, RowVec<T, VEC>& g,
                                      const RowVec<T, VEC>&, int64_t row) {
    const uint32_t kp = c.keep(row);
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const T z = st.z(x.v[i]);
      T h = c.drop(kp, i, g.v[i]);
      if (c.act) {
        const T t = c.w[i] * z + c.b[i], s = gn_sigmoid(t);
        h *= s * (T(1) + t * (T(1) - s));
      }
      cw[i] += h * z;
      cb[i] += h;
      x.v[i] = z;
      g.v[i] = c.w[i] * h;
    }
  }
  // the group's sums are the columns' times the weights
  template <typename COL>
  __device__ __forceinline__ void flush(const COL& c, double* colw, double* colb) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      S1 += double(c.w[i]) * double(cb[i]);
      S2 += double(c.w[i]) * double(cw[i]);
      colw[i] += double(cw[i]);
      colb[i] += double(cb[i]);
    }
    clear();
  }
  template <typename COL>
  __device__ __forceinline__ void publish(const COL&, double* buf) const {
    buf[0] = S1;
    buf[GN_THREADS] = S2;
  }
};

// h, q's factor m g a''(t), m a'(t) and z of one value
template <typename T>
struct GnSecond {
  T z, h, q1, d1;
};
template <typename T, int VEC, bool DROP>
__device__ __forceinline__ GnSecond<T> gn_second(const GnCol<T, VEC, GN_DBL, DROP>& c, const GnStat<T>& st, uint32_t kp,
                                                 int i, T x, T g) {
  GnSecond<T> o;
  o.z = st.z(x);
  const T gm = c.drop(kp, i, g);
  o.d1 = c.drop(kp, i, T(1));
  o.h = gm;
  o.q1 = T(0);
  if (c.act) {
    const T t = c.w[i] * o.z + c.b[i], s = gn_sigmoid(t), d1 = s * (T(1) + t * (T(1) - s));
    o.h = gm * d1;
    o.d1 *= d1;
    o.q1 = gm * (s * (T(1) - s) * (T(2) + t * (T(1) - T(2) * s)));
  }
  return o;
}

template <typename T, int VEC, bool DROP>
struct GnAcc<T, VEC, GN_DBL, DROP> {
  T s[12];
  double S[12];
  __device__ __forceinline__ void start() {
#pragma unroll
    for (int i = 0; i < 12; ++i) S[i] = 0.0;
    clear();
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < 12; ++i) s[i] = T(0);
  }
  template <typename COL>
  __device__ __forceinline__ void add(const COL& c, const GnStat<T>& st, RowVec<T, VEC>& x, RowVec<T, VEC>& g,
                                      const RowVec<T, VEC>& u, int64_t row) {
    const uint32_t kp = c.keep(row);
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const GnSecond<T> e = gn_second<T, VEC, DROP>(c, st, kp, i, x.v[i], g.v[i]);
      const T ux = u.v[i], cc = c.w[i] * e.h;
      s[0] += ux;
      s[1] += e.z * ux;
      s[2] += cc;
      s[3] += cc * e.z;
      s[4] += cc * ux;
      T v = c.uw[i] * e.h;
      if (c.act) {
        const T wq = c.w[i] * c.w[i] * e.q1;
        v += c.w[i] * e.q1 * (c.uw[i] * e.z + c.ub[i]);
        s[5] += wq;
        s[6] += wq * e.z;
        s[7] += wq * e.z * e.z;
        s[8] += wq * ux;
        s[9] += wq * ux * e.z;
      }
      s[10] += v;
      s[11] += v * e.z;
    }
  }
  template <typename COL>
  __device__ __forceinline__ void flush(const COL&, double*, double*) {
#pragma unroll
    for (int i = 0; i < 12; ++i) S[i] += double(s[i]);
    clear();
  }
  template <typename COL>
  __device__ __forceinline__ void publish(const COL&, double* buf) const {
#pragma unroll
    for (int i = 0; i < 12; ++i) buf[i * GN_THREADS] = S[i];
  }
};

// The coefficients of a (segment, group) from its joined sums S and its n values.
// Forward: {mu, r}.  Backward: {mean c, mean cz}.  Double backward: {m1, m2, mean cz, mean C, mean zC, mean c zd}.
template <int OP>
__device__ __forceinline__ void gn_finish(const double* S, double n, bool scalar, double r, double eps, double* o) {
  const double in = n > 0.0 ? 1.0 / n : 0.0;
  if (OP == GN_FWD) {
    o[0] = S[0];
    o[1] = 1.0 / sqrt(S[1] * in + eps);
  } else if (OP == GN_BWD) {
    o[0] = scalar ? S[0] * in : 0.0;
    o[1] = S[1] * in;
  } else {
    const double m1 = scalar ? S[0] * in : 0.0, m2 = S[1] * in, mcz = S[3] * in;
    o[0] = m1;
    o[1] = m2;
    o[2] = mcz;
    o[3] = scalar ? in * (r * (S[8] - m1 * S[5] - m2 * S[6]) + S[10] - r * m2 * S[2] - r * mcz * S[0]) : 0.0;
    o[4] = in * (r * (S[9] - m1 * S[6] - m2 * S[7]) + S[11] - r * m2 * S[3] - r * mcz * S[1]);
    o[5] = in * (r * (S[4] - m1 * S[2] - m2 * S[3]));
  }
}

// Join what the threads published: item (jj, lg) sums the entries of K row lanes x the group's vectors.
// Called by all threads; `lanes` (a power of two) threads share an item.  done(item, S) runs on one of
// them.  Forward: S = {mean, M2, count}.
template <int OP, typename F>
__device__ __forceinline__ void gn_join(const double* buf, const int2* gs, int nlg, int J, int K, int TX, int lanes,
                                        F done) {
  constexpr int NS = gn_sums(OP);
  const int per = GN_THREADS / lanes, lane = int(threadIdx.x) % lanes, sub = int(threadIdx.x) / lanes;
  const int items = J * nlg;
  for (int base = 0; base < items; base += per) {
    const int it = base + sub;
    const bool ok = it < items;
    int w = 0, first = 0;
    if (ok) {
      const int2 r = gs[it % nlg];
      first = (it / nlg) * K * TX + r.x;
      w = r.y - r.x;
    }
    const int E = ok ? K * w : 0;
    double S[NS];
#pragma unroll
    for (int s = 0; s < NS; ++s) S[s] = 0.0;
    for (int e = lane; e < E; e += lanes) {
      const int t = first + (e / w) * TX + e % w;
      if (OP == GN_FWD) {
        S[0] += buf[t] * buf[2 * GN_THREADS + t];
        S[NS - 1] += buf[2 * GN_THREADS + t];
      } else {
#pragma unroll
        for (int s = 0; s < NS; ++s) S[s] += buf[s * GN_THREADS + t];
      }
    }
    for (int o = lanes / 2; o > 0; o /= 2) {
#pragma unroll
      for (int s = 0; s < NS; ++s)
        if (OP != GN_FWD || s != 1) S[s] += __shfl_xor_sync(~0u, S[s], o);
    }
    if (OP == GN_FWD) {
      const double mean = S[NS - 1] > 0.0 ? S[0] / S[NS - 1] : 0.0;
      double m2 = 0.0;
      for (int e = lane; e < E; e += lanes) {
        const int t = first + (e / w) * TX + e % w;
        const double d = buf[t] - mean, n = buf[2 * GN_THREADS + t];
        if (n > 0.0) m2 += buf[GN_THREADS + t] + n * d * d;
      }
      for (int o = lanes / 2; o > 0; o /= 2) m2 += __shfl_xor_sync(~0u, m2, o);
      S[0] = mean;
      S[1] = m2;
    }
    if (ok && lane == 0) done(it, S);
  }
}

// Pointwise results of one vector.  In the backward x and g hold z and c.
template <typename T, int VEC, int OP, bool DROP>
__device__ __forceinline__ void gn_apply(const NormArgs& a, const GnCol<T, VEC, OP, DROP>& c, const GnStat<T>& st,
                                         const T* k, const RowVec<T, VEC>& x, const RowVec<T, VEC>& g,
                                         const RowVec<T, VEC>& u, int64_t row, T* cw, T* cb) {
  const int64_t at = row * a.lay.dim + c.col;
  RowVec<T, VEC> o;
  if (OP == GN_FWD) {
    const uint32_t kp = c.keep(row);
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const T t = c.w[i] * st.z(x.v[i]) + c.b[i];
      o.v[i] = c.drop(kp, i, c.act ? t * gn_sigmoid(t) : t);
    }
    store_row<T, VEC>(static_cast<T*>(a.o0) + at, o);
  } else if (OP == GN_BWD) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) o.v[i] = st.r * (g.v[i] - k[0] - x.v[i] * k[1]);
    if (a.o0 != nullptr) store_row<T, VEC>(static_cast<T*>(a.o0) + at, o);
  } else {
    if constexpr (OP == GN_DBL) {
      const uint32_t kp = c.keep(row);
      RowVec<T, VEC> dg;
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const GnSecond<T> e = gn_second<T, VEC, DROP>(c, st, kp, i, x.v[i], g.v[i]);
        const T ux = u.v[i], cc = c.w[i] * e.h;
        const T zd = st.r * (ux - k[0] - e.z * k[1]);
        const T td = c.w[i] * zd + c.uw[i] * e.z + c.ub[i];
        const T q = e.q1 * td;
        const T C = c.w[i] * q + c.uw[i] * e.h - st.r * (k[1] * cc + k[2] * ux);
        dg.v[i] = e.d1 * td;
        o.v[i] = st.r * (C - k[3] - e.z * k[4] - e.z * k[5]);
        cw[i] += q * e.z + e.h * zd;
        cb[i] += q;
      }
      if (a.o0 != nullptr) store_row<T, VEC>(static_cast<T*>(a.o0) + at, o);
      if (a.o1 != nullptr) store_row<T, VEC>(static_cast<T*>(a.o1) + at, dg);
    }
  }
}

// Zero rows [from, to) of the outputs in this thread's column.
template <typename T, int VEC, int OP>
__device__ __forceinline__ void gn_zero_rows(const NormArgs& a, int col, int64_t from, int64_t to, int64_t step) {
  RowVec<T, VEC> zero;
#pragma unroll
  for (int i = 0; i < VEC; ++i) zero.v[i] = T(0);
  for (int64_t r = from; r < to; r += step) {
    if (a.o0 != nullptr) store_row<T, VEC>(static_cast<T*>(a.o0) + r * a.lay.dim + col, zero);
    if (OP == GN_DBL && a.o1 != nullptr) store_row<T, VEC>(static_cast<T*>(a.o1) + r * a.lay.dim + col, zero);
  }
}

// Column sums of a CTA (all row lanes of a vector column) into its slot of colpart.
template <int VEC>
__device__ __forceinline__ void gn_store_columns(const NormArgs& a, double* buf, int64_t slot, bool active, int col,
                                                 int tx, int ty, int TX, int TY, const double* colw,
                                                 const double* colb) {
#pragma unroll
  for (int i = 0; i < 2 * VEC; ++i) {
    __syncthreads();
    buf[threadIdx.x] = active ? (i < VEC ? colw[i] : colb[i - VEC]) : 0.0;
    __syncthreads();
    if (active && ty == 0) {
      double s = 0.0;
      for (int y = 0; y < TY; ++y) s += buf[y * TX + tx];
      a.colpart[(2 * slot + (i < VEC ? 0 : 1)) * a.lay.dim + col + i % VEC] = s;
    }
  }
}

template <typename T, int VEC, int OP>
__device__ __forceinline__ void gn_load(const NormArgs& a, int64_t at, RowVec<T, VEC>& x, RowVec<T, VEC>& g,
                                        RowVec<T, VEC>& u) {
  x = load_row<T, VEC>(static_cast<const T*>(a.x) + at);
  if (OP != GN_FWD) g = load_row<T, VEC>(static_cast<const T*>(a.g) + at);
  if (OP == GN_DBL) {
    if (a.u != nullptr) {
      u = load_row<T, VEC>(static_cast<const T*>(a.u) + at);
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) u.v[i] = T(0);
    }
  }
}

// local: thread (j, k, tx) owns vector column tx of the CTA's slab, row lane k of segment j of the
// CTA's current batch of J segments.
template <typename T, int VEC, int OP, bool DROP, int RP>
__global__ void __launch_bounds__(GN_THREADS) gn_local_kernel(const __grid_constant__ NormArgs a) {
  constexpr int NS = gn_sums(OP), NC = gn_coefs(OP);
  __shared__ double buf[NS * GN_THREADS];
  __shared__ double res[NC * GN_THREADS];
  __shared__ int2 gs[GN_THREADS];
  const int v0 = a.slab[blockIdx.y], W = a.slab[blockIdx.y + 1] - v0;
  const int TX = a.tx, K = a.k, J = a.j;
  const int tx = int(threadIdx.x) % TX, ty = int(threadIdx.x) / TX;
  const int j = ty / K, k = ty % K;
  const bool active = tx < W && j < J;
  const int nlg = group_of(a.lay, (v0 + W) * VEC - 1) - group_of(a.lay, v0 * VEC) + 1;
  GnCol<T, VEC, OP, DROP> c;
  c.init(a, v0, W, active ? tx : 0);
  if (active && ty == 0 && tx == c.g0) gs[c.lg] = make_int2(c.g0, c.g1);
  const int64_t D = a.lay.dim, G = a.lay.n_blocks * a.lay.groups;
  const int gfirst = c.g - c.lg;
  double colw[VEC], colb[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) colw[i] = colb[i] = 0.0;

  for (int64_t b0 = int64_t(blockIdx.x) * J; b0 < a.B; b0 += int64_t(gridDim.x) * J) {
    const int64_t b = b0 + j;
    const bool live = active && b < a.B;
    int64_t s = 0, e = 0;
    if (live) gn_segment(a, b, s, e);
    const int64_t chunks = (e - s + int64_t(K) * RP - 1) / (int64_t(K) * RP);
    GnStat<T> st;
    if (OP != GN_FWD && live) {
      const double* p = a.stats + 2 * (b * G + c.g);
      st.set(p[0], p[1]);
    }
    RowVec<T, VEC> x[RP], g[RP], u[RP];
    GnAcc<T, VEC, OP, DROP> acc;
    acc.start();
    for (int64_t ch = 0; ch < chunks; ++ch) {
      const int64_t r0 = s + ch * K * RP + k;
#pragma unroll
      for (int i = 0; i < RP; ++i)
        if (r0 + i * K < e) gn_load<T, VEC, OP>(a, (r0 + i * K) * D + c.col, x[i], g[i], u[i]);
#pragma unroll
      for (int i = 0; i < RP; ++i)
        if (r0 + i * K < e) acc.add(c, st, x[i], g[i], u[i], r0 + i * K);
      acc.flush(c, colw, colb);
    }
    if (live) acc.publish(c, buf + threadIdx.x);
    __syncthreads();
    gn_join<OP>(buf, gs, nlg, J, K, TX, a.lanes, [&](int it, const double* S) {
      const int64_t bb = b0 + it / nlg;
      if (bb >= a.B) return;
      const int gg = gfirst + it % nlg;
      int64_t ss, ee;
      gn_segment(a, bb, ss, ee);
      const RowBlock& blk = a.lay.blk[gg / a.lay.groups];
      double* sg = a.stats + 2 * (bb * G + gg);
      gn_finish<OP>(S, double(ee - ss) * blk.group_cols, blk.bias0 >= 0, OP == GN_DBL ? sg[1] : 0.0, a.eps,
                    res + NC * it);
      if (OP == GN_FWD) {
        sg[0] = res[NC * it];
        sg[1] = res[NC * it + 1];
      }
    });
    __syncthreads();
    if (live) {
      const double* q = res + NC * (j * nlg + c.lg);
      T kf[NC];
      if (OP == GN_FWD) {
        st.set(q[0], q[1]);
      } else {
#pragma unroll
        for (int i = 0; i < NC; ++i) kf[i] = T(q[i]);
      }
      T cw[VEC], cb[VEC];
      for (int64_t ch = 0; ch < chunks; ++ch) {
        const int64_t r0 = s + ch * K * RP + k;
        if (chunks > 1) {  // a segment longer than the registers hold: read again
          GnAcc<T, VEC, OP, DROP> again;
          again.start();
#pragma unroll
          for (int i = 0; i < RP; ++i)
            if (r0 + i * K < e) {
              gn_load<T, VEC, OP>(a, (r0 + i * K) * D + c.col, x[i], g[i], u[i]);
              if (OP == GN_BWD) again.add(c, st, x[i], g[i], u[i], r0 + i * K);
            }
        }
#pragma unroll
        for (int i = 0; i < VEC; ++i) cw[i] = cb[i] = T(0);
#pragma unroll
        for (int i = 0; i < RP; ++i)
          if (r0 + i * K < e) gn_apply<T, VEC, OP, DROP>(a, c, st, kf, x[i], g[i], u[i], r0 + i * K, cw, cb);
        if (OP == GN_DBL) {
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            colw[i] += double(cw[i]);
            colb[i] += double(cb[i]);
          }
        }
      }
    }
  }
  if (active)
    gn_zero_rows<T, VEC, OP>(a, c.col, gn_rows_end(a) + int64_t(blockIdx.x) * (J * K) + ty, a.N,
                             int64_t(gridDim.x) * (J * K));
  if (OP != GN_FWD && a.colpart != nullptr)
    gn_store_columns<VEC>(a, buf, blockIdx.x, active, c.col, tx, ty, TX, J * K, colw, colb);
}

// Last segment that starts at or before row r.
__device__ __forceinline__ int64_t gn_first_segment(const NormArgs& a, int64_t r) {
  if (a.row_ptr == nullptr) return 0;
  int64_t lo = 0, hi = a.B - 1;
  while (lo < hi) {
    const int64_t m = (lo + hi + 1) / 2;
    if (int64_t(a.row_ptr[m]) <= r) lo = m;
    else hi = m - 1;
  }
  return lo;
}

// split, first pass: partial sums of (chunk, segment) pieces x (tile, group) parts.  Pieces in row order
// raise the chunk or the segment by one, so chunk + segment numbers them; parts likewise.
template <typename T, int VEC, int OP, bool DROP>
__global__ void __launch_bounds__(GN_THREADS) gn_partial_kernel(const __grid_constant__ NormArgs a) {
  constexpr int NS = gn_sums(OP), U = 4;
  __shared__ double buf[NS * GN_THREADS];
  __shared__ int2 gs[GN_THREADS];
  const int TX = a.tx, K = a.k;
  const int tile = int(blockIdx.y), v0 = tile * TX, W = min(TX, a.lay.dim / VEC - v0);
  const int tx = int(threadIdx.x) % TX, ty = int(threadIdx.x) / TX;
  const bool active = tx < W && ty < K;
  const int nlg = group_of(a.lay, (v0 + W) * VEC - 1) - group_of(a.lay, v0 * VEC) + 1;
  GnCol<T, VEC, OP, DROP> c;
  c.init(a, v0, W, active ? tx : 0);
  if (active && ty == 0 && tx == c.g0) gs[c.lg] = make_int2(c.g0, c.g1);
  const int64_t D = a.lay.dim, G = a.lay.n_blocks * a.lay.groups;
  const int gfirst = c.g - c.lg;
  double colw[VEC], colb[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) colw[i] = colb[i] = 0.0;
  const int64_t lo = int64_t(blockIdx.x) * a.rows_cta, hi = min(a.N, lo + a.rows_cta);
  for (int64_t b = gn_first_segment(a, lo); b < a.B; ++b) {
    int64_t s, e;
    gn_segment(a, b, s, e);
    if (s >= hi) break;
    s = max(s, lo);
    e = min(e, hi);
    if (s >= e) continue;
    GnStat<T> st;
    if (OP != GN_FWD) {
      const double* p = a.stats + 2 * (b * G + c.g);
      st.set(p[0], p[1]);
    }
    GnAcc<T, VEC, OP, DROP> acc;
    acc.start();
    if (active) {
      for (int64_t f = s; f < e; f += int64_t(K) * GN_FLUSH) {
        const int64_t fe = min(e, f + int64_t(K) * GN_FLUSH);
        for (int64_t r = f + ty; r < fe; r += int64_t(K) * U) {
          RowVec<T, VEC> x[U], g[U], u[U];
#pragma unroll
          for (int i = 0; i < U; ++i)
            if (r + i * K < fe) gn_load<T, VEC, OP>(a, (r + i * K) * D + c.col, x[i], g[i], u[i]);
#pragma unroll
          for (int i = 0; i < U; ++i)
            if (r + i * K < fe) acc.add(c, st, x[i], g[i], u[i], r + i * K);
        }
        acc.flush(c, colw, colb);
      }
      acc.publish(c, buf + threadIdx.x);
    }
    __syncthreads();
    double* slot = a.part + ((int64_t(blockIdx.x) + b) * (G + a.n_tiles) + tile) * NS;
    gn_join<OP>(buf, gs, nlg, 1, K, TX, a.lanes, [&](int it, const double* S) {
#pragma unroll
      for (int i = 0; i < NS; ++i) slot[int64_t(gfirst + it) * NS + i] = S[i];
    });
    __syncthreads();
  }
  if (OP == GN_BWD && a.colpart != nullptr)
    gn_store_columns<VEC>(a, buf, blockIdx.x, active, c.col, tx, ty, TX, K, colw, colb);
}

// split, between the passes: one warp per (segment, group) joins its pieces x parts.
template <int OP, int VEC>
__global__ void __launch_bounds__(GN_THREADS) gn_final_kernel(const __grid_constant__ NormArgs a) {
  constexpr int NS = gn_sums(OP), NC = gn_coefs(OP);
  const int64_t G = a.lay.n_blocks * a.lay.groups;
  const int64_t it = (int64_t(blockIdx.x) * GN_THREADS + threadIdx.x) / 32;
  const int lane = int(threadIdx.x) % 32;
  if (it >= a.B * G) return;
  const int64_t b = it / G;
  const int g = int(it % G);
  int64_t s, e;
  gn_segment(a, b, s, e);
  const RowBlock& blk = a.lay.blk[g / a.lay.groups];
  const int gc = group_col(a.lay, g);
  const int t0 = gc / VEC / a.tx, nt = (gc + blk.group_cols - 1) / VEC / a.tx - t0 + 1;
  const int64_t c0 = s / a.rows_cta, nc = e > s ? (e - 1) / a.rows_cta - c0 + 1 : 0;
  const int64_t E = nc * nt;
  double S[NS];
#pragma unroll
  for (int i = 0; i < NS; ++i) S[i] = 0.0;
  auto at = [&](int64_t i) {
    return a.part + ((c0 + i / nt + b) * (G + a.n_tiles) + g + t0 + i % nt) * NS;
  };
  for (int64_t i = lane; i < E; i += 32) {
    const double* p = at(i);
    if (OP == GN_FWD) {
      S[0] += p[0] * p[NS - 1];
      S[NS - 1] += p[NS - 1];
    } else {
#pragma unroll
      for (int q = 0; q < NS; ++q) S[q] += p[q];
    }
  }
  for (int o = 16; o > 0; o /= 2) {
#pragma unroll
    for (int q = 0; q < NS; ++q) S[q] += __shfl_xor_sync(~0u, S[q], o);
  }
  if (OP == GN_FWD) {
    const double mean = S[NS - 1] > 0.0 ? S[0] / S[NS - 1] : 0.0;
    double m2 = 0.0;
    for (int64_t i = lane; i < E; i += 32) {
      const double* p = at(i);
      const double d = p[0] - mean;
      m2 += p[1] + p[NS - 1] * d * d;
    }
    for (int o = 16; o > 0; o /= 2) m2 += __shfl_xor_sync(~0u, m2, o);
    S[0] = mean;
    S[1] = m2;
  }
  if (lane == 0) {
    double o[NC];
    double* st = a.stats + 2 * it;
    gn_finish<OP>(S, double(e - s) * blk.group_cols, blk.bias0 >= 0, OP == GN_DBL ? st[1] : 0.0, a.eps, o);
    double* dst = OP == GN_FWD ? st : a.coef + NC * it;
#pragma unroll
    for (int i = 0; i < NC; ++i) dst[i] = o[i];
  }
}

// split, second pass: pointwise results.
template <typename T, int VEC, int OP, bool DROP>
__global__ void __launch_bounds__(GN_THREADS) gn_apply_kernel(const __grid_constant__ NormArgs a) {
  constexpr int NC = gn_coefs(OP), U = 4;
  __shared__ double buf[GN_THREADS];
  const int TX = a.tx, K = a.k;
  const int v0 = int(blockIdx.y) * TX, W = min(TX, a.lay.dim / VEC - v0);
  const int tx = int(threadIdx.x) % TX, ty = int(threadIdx.x) / TX;
  const bool active = tx < W && ty < K;
  GnCol<T, VEC, OP, DROP> c;
  c.init(a, v0, W, active ? tx : 0);
  const int64_t D = a.lay.dim, G = a.lay.n_blocks * a.lay.groups;
  double colw[VEC], colb[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) colw[i] = colb[i] = 0.0;
  const int64_t lo = int64_t(blockIdx.x) * a.rows_cta, hi = min(a.N, lo + a.rows_cta);
  if (active) {
    for (int64_t b = gn_first_segment(a, lo); b < a.B; ++b) {
      int64_t s, e;
      gn_segment(a, b, s, e);
      if (s >= hi) break;
      s = max(s, lo);
      e = min(e, hi);
      if (s >= e) continue;
      GnStat<T> st;
      const double* p = a.stats + 2 * (b * G + c.g);
      st.set(p[0], p[1]);
      T k[NC];
      if (OP != GN_FWD) {
        const double* q = a.coef + NC * (b * G + c.g);
#pragma unroll
        for (int i = 0; i < NC; ++i) k[i] = T(q[i]);
      }
      for (int64_t f = s; f < e; f += int64_t(K) * GN_FLUSH) {
        const int64_t fe = min(e, f + int64_t(K) * GN_FLUSH);
        T cw[VEC], cb[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) cw[i] = cb[i] = T(0);
        for (int64_t r = f + ty; r < fe; r += int64_t(K) * U) {
          RowVec<T, VEC> x[U], g[U], u[U];
#pragma unroll
          for (int i = 0; i < U; ++i)
            if (r + i * K < fe) gn_load<T, VEC, OP>(a, (r + i * K) * D + c.col, x[i], g[i], u[i]);
#pragma unroll
          for (int i = 0; i < U; ++i)
            if (r + i * K < fe) {
              if (OP == GN_BWD) {  // z and c again
                GnAcc<T, VEC, OP, DROP> again;
                again.start();
                again.add(c, st, x[i], g[i], u[i], r + i * K);
              }
              gn_apply<T, VEC, OP, DROP>(a, c, st, k, x[i], g[i], u[i], r + i * K, cw, cb);
            }
        }
        if (OP == GN_DBL) {
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            colw[i] += double(cw[i]);
            colb[i] += double(cb[i]);
          }
        }
      }
    }
    gn_zero_rows<T, VEC, OP>(a, c.col, max(lo, gn_rows_end(a)) + ty, hi, K);
  }
  if (OP == GN_DBL && a.colpart != nullptr)
    gn_store_columns<VEC>(a, buf, blockIdx.x, active, c.col, tx, ty, TX, K, colw, colb);
}

}  // namespace e3b
