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
// O(N dim), so the kernels are bound by memory, and the second pass has to find the rows on chip.
// Two kernels, one launch each:
//   local  a CTA, or a cluster of CTAs that divide the rows, holds whole segments x whole groups in
//          registers between the passes (one read);
//   grid   longer segments: a resident grid takes a slab of columns after another; in each, row chunks x
//          column tiles publish partial sums, the grid meets, and every CTA joins the sums that it
//          needs and reads its rows again, from L2 if the slab is small enough.
// Sums run in the rows' type over a few rows of a thread (at most GN_FLUSH; the grid kernel goes on in
// double from there), then over the threads, CTAs and chunks of a segment in a fixed order.  Variances are
// sums around a thread's own mean, joined by the distances of the means, all taken from one
// value of the segment (for float rows, so that an offset of the data costs no digits): a thread's
// first value is its pivot, and (pivot - mean)^2 is a term of the true sum, so the cancellation
// costs at most the thread's number of values in epsilons.
#pragma once

#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "internal.h"
#include "rows.cuh"

namespace e3b {

constexpr int GN_THREADS = 256;
constexpr int GN_FLUSH = 64;
constexpr int GN_MAXTILE = 512;
enum GnOp { GN_FWD = 0, GN_BWD = 1, GN_DBL = 2 };
// sums of a (segment, group): forward (pivot, mean - pivot, sum of squares around the mean, count),
// backward (sum c, sum c z), double backward 12
__host__ __device__ constexpr int gn_sums(int op) { return op == GN_FWD ? 4 : op == GN_BWD ? 2 : 12; }
// what the second pass needs of a (segment, group): forward (mean high, mean low, r), backward (mean c,
// mean cz), double backward (m1, m2, mean cz, mean C, mean zC, mean c zd)
__host__ __device__ constexpr int gn_coefs(int op) { return op == GN_FWD ? 3 : op == GN_BWD ? 2 : 6; }

struct NormArgs {
  int64_t N;
  int32_t B;
  const int32_t* row_ptr;  // NULL: one segment of all rows
  const void *x, *g, *u;   // rows: features, grad_y, u_x (may be NULL)
  const void *w, *b, *uw, *ub;
  void *o0, *o1;           // y | grad_x | d_x ; d_grad_y (each may be NULL in the backwards)
  void *gw, *gb;           // gradients of weight and bias (may be NULL)
  double* stats;           // [B][groups][2]
  void* part;              // grid: partial sums, see gn_slot
  void* coef;              // grid: [B][groups][coefs] of segments that lie inside one chunk (backwards)
  double* colpart;         // [parts][2][dim]: sums for gw, gb per column (NULL: not wanted)
  double eps;
  int32_t act;
  int* status;
  int32_t tx, k, j, lanes;  // thread layout: columns, row lanes of a segment, segments, lanes of a join
  int32_t cs;               // local: CTAs of a cluster
  int32_t wide;             // grid: some group is cut into several tiles
  int32_t n_tiles, cx;      // tiles of columns, tiles of a slab
  int32_t chunks;           // grid: row chunks
  int64_t rows_cta;         // grid: rows of a chunk
  DropArgs drop;
  RowLayout lay;
  int32_t tile[GN_MAXTILE + 1];  // first vector column of each tile
};

// Rows [s, e) of segment b, clamped into [0, N); a bad row pointer is recorded.
__device__ __forceinline__ void gn_segment(const NormArgs& a, int b, int& s, int& e) {
  if (a.row_ptr == nullptr) {
    s = 0;
    e = int(a.N);
    return;
  }
  const int n = int(a.N);
  s = a.row_ptr[b];
  e = a.row_ptr[b + 1];
  if (s < 0 || e < s || e > n || (b == 0 && s != 0)) {
    atomicCAS(a.status, 0, int(E3_ERR_INDEX));
    s = min(max(s, 0), n);
    e = min(max(e, s), n);
  }
}
// First padding row.
__device__ __forceinline__ int gn_rows_end(const NormArgs& a) {
  return a.row_ptr == nullptr ? int(a.N) : min(max(a.row_ptr[a.B], 0), int(a.N));
}

template <typename T>
struct GnStat {
  T hi, lo, r;  // mu = hi + lo
  __device__ __forceinline__ void set(const double* p) {
    hi = T(p[0]);
    lo = T(p[0] - double(hi));
    r = T(p[1]);
  }
};

__device__ __forceinline__ float gn_sigmoid(float t) { return __fdividef(1.f, 1.f + expf(-t)); }
__device__ __forceinline__ double gn_sigmoid(double t) { return 1.0 / (1.0 + exp(-t)); }

// Kinds of columns: 0 not centred, 1 even scalars, 2 even scalars with the activation.
enum { GN_PLAIN = 0, GN_CENTRED = 1, GN_ACT = 2 };

// What a thread knows of its vector column.
template <typename T, int VEC, int OP, bool DROP>
struct GnCol {
  int col, g, lg, g0, g1;  // first column, group, group within the tile, its vector range in the tile
  int kind;
  T w[VEC], b[VEC], uw[VEC], ub[VEC];
  DropCol<VEC> dc;
  T scale;

  __device__ __forceinline__ void init(const NormArgs& a, int v0, int width, int tx) {
    const RowLayout& L = a.lay;
    col = (v0 + tx) * VEC;
    const int bi = block_of(L, col);
    const RowBlock& k = L.blk[bi];
    const int gi = int(fast_div(uint32_t(col - k.col0), k.div_group)), gc = k.col0 + gi * k.group_cols;
    g = bi * L.groups + gi;
    lg = g - group_of(L, v0 * VEC);
    g0 = max(gc / VEC - v0, 0);
    g1 = min((gc + k.group_cols) / VEC - v0, width);
    kind = k.bias0 < 0 ? GN_PLAIN : a.act == E3_ACT_SILU ? GN_ACT : GN_CENTRED;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const int u = int(fast_div(uint32_t(col + i - k.col0), k.div_d));
      w[i] = a.w ? static_cast<const T*>(a.w)[k.chan0 + u] : T(1);
      b[i] = kind != GN_PLAIN && a.b ? static_cast<const T*>(a.b)[k.bias0 + u] : T(0);
      if (OP == GN_DBL) {
        uw[i] = a.uw ? static_cast<const T*>(a.uw)[k.chan0 + u] : T(0);
        ub[i] = kind != GN_PLAIN && a.ub ? static_cast<const T*>(a.ub)[k.bias0 + u] : T(0);
      }
    }
    if (DROP) {
      dc.init(L, a.drop, col);
      scale = T(a.drop.scale);
    }
  }
  __device__ __forceinline__ uint32_t keep(int row) const { return DROP ? dc.keep(row) : ~0u; }
  __device__ __forceinline__ T drop(uint32_t kp, int i, T v) const {
    return DROP ? ((kp >> i & 1u) ? v * scale : T(0)) : v;
  }
  template <int KIND>
  __device__ __forceinline__ T z(const GnStat<T>& st, T x) const {
    return KIND == GN_PLAIN ? x * st.r : ((x - st.hi) - st.lo) * st.r;
  }
};

// Vectors of one row.
template <typename T, int VEC>
struct GnRow {
  RowVec<T, VEC> x, g, u;
};
template <typename T, int VEC, int OP>
__device__ __forceinline__ void gn_load(const NormArgs& a, int64_t at, GnRow<T, VEC>& v) {
  v.x = load_row<T, VEC>(static_cast<const T*>(a.x) + at);
  if (OP != GN_FWD) v.g = load_row<T, VEC>(static_cast<const T*>(a.g) + at);
  if (OP == GN_DBL) {
    if (a.u != nullptr) {
      v.u = load_row<T, VEC>(static_cast<const T*>(a.u) + at);
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) v.u.v[i] = T(0);
    }
  }
}

// h, q's factor m g a''(t), m a'(t) and z of one value
template <typename T>
struct GnSecond {
  T z, h, q1, d1;
};
template <int KIND, typename T, int VEC, bool DROP>
__device__ __forceinline__ GnSecond<T> gn_second(const GnCol<T, VEC, GN_DBL, DROP>& c, const GnStat<T>& st, uint32_t kp,
                                                 int i, T x, T g) {
  GnSecond<T> o;
  o.z = c.template z<KIND>(st, x);
  const T gm = c.drop(kp, i, g);
  o.d1 = c.drop(kp, i, T(1));
  o.h = gm;
  o.q1 = T(0);
  if (KIND == GN_ACT) {
    const T t = c.w[i] * o.z + c.b[i], s = gn_sigmoid(t), d1 = s * (T(1) + t * (T(1) - s));
    o.h = gm * d1;
    o.d1 *= d1;
    o.q1 = gm * (s * (T(1) - s) * (T(2) + t * (T(1) - T(2) * s)));
  }
  return o;
}

// The sums of one thread over a few rows of one segment, in the rows' type.  Forward: s1, s2 around piv.
// Backward: s1 = sum h z, s2 = sum h per column (the group's sums are these times the weights).
template <typename T, int VEC, int OP, bool DROP>
struct GnAcc {
  T s1[VEC], s2[VEC];
  template <typename COL>
  __device__ __forceinline__ void clear(const COL&) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) s1[i] = s2[i] = T(0);
  }
  // backward: x becomes z, g becomes c = w h
  template <int KIND, typename COL>
  __device__ __forceinline__ void add(const COL& c, const GnStat<T>& st, T piv, GnRow<T, VEC>& v, int row) {
    if (OP == GN_FWD) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        if (KIND == GN_PLAIN) {
          s2[i] += v.x.v[i] * v.x.v[i];
        } else {
          const T d = v.x.v[i] - piv;
          s1[i] += d;
          s2[i] += d * d;
        }
      }
    } else {
      const uint32_t kp = c.keep(row);
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const T z = c.template z<KIND>(st, v.x.v[i]);
        T h = c.drop(kp, i, v.g.v[i]);
        if (KIND == GN_ACT) {
          const T t = c.w[i] * z + c.b[i], s = gn_sigmoid(t);
          h *= s * (T(1) + t * (T(1) - s));
        }
        s1[i] += h * z;
        if (KIND != GN_PLAIN) s2[i] += h;
        v.x.v[i] = z;
        v.g.v[i] = c.w[i] * h;
      }
    }
  }
};
template <typename T, int VEC, bool DROP>
struct GnAcc<T, VEC, GN_DBL, DROP> {
  T s[12];
  template <typename COL>
  __device__ __forceinline__ void clear(const COL&) {
#pragma unroll
    for (int i = 0; i < 12; ++i) s[i] = T(0);
  }
  template <int KIND, typename COL>
  __device__ __forceinline__ void add(const COL& c, const GnStat<T>& st, T, GnRow<T, VEC>& v, int row) {
    const uint32_t kp = c.keep(row);
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const GnSecond<T> e = gn_second<KIND, T, VEC, DROP>(c, st, kp, i, v.x.v[i], v.g.v[i]);
      const T ux = v.u.v[i], cc = c.w[i] * e.h;
      T q = c.uw[i] * e.h;
      s[1] += e.z * ux;
      s[3] += cc * e.z;
      s[4] += cc * ux;
      if (KIND != GN_PLAIN) {
        s[0] += ux;
        s[2] += cc;
      }
      if (KIND == GN_ACT) {
        const T wq = c.w[i] * c.w[i] * e.q1;
        q += c.w[i] * e.q1 * (c.uw[i] * e.z + c.ub[i]);
        s[5] += wq;
        s[6] += wq * e.z;
        s[7] += wq * e.z * e.z;
        s[8] += wq * ux;
        s[9] += wq * ux * e.z;
      }
      if (KIND != GN_PLAIN) s[10] += q;
      s[11] += q * e.z;
    }
  }
};

// The second pass' coefficients of a (segment, group) from its joined sums S and its n values.
// Forward: o = {mean high, mean low, r}, and (mean, r) into sg.
template <int OP, typename T>
__device__ __forceinline__ void gn_finish(const T* s, T n, bool scalar, double* sg, bool keep, double eps, T* o) {
  const T in = n > T(0) ? T(1) / n : T(0);
  if (OP == GN_FWD) {
    const double mean = double(s[0]) + double(s[1]);
    const T r = T(1) / sqrt(s[2] * in + T(eps));
    o[0] = T(mean);
    o[1] = T(mean - double(o[0]));
    o[2] = r;
    if (keep) {
      sg[0] = mean;
      sg[1] = double(r);
    }
  } else if (OP == GN_BWD) {
    o[0] = scalar ? s[0] * in : T(0);
    o[1] = s[1] * in;
  } else {
    const T r = T(sg[1]);
    const T m1 = scalar ? s[0] * in : T(0), m2 = s[1] * in, mcz = s[3] * in;
    o[0] = m1;
    o[1] = m2;
    o[2] = mcz;
    o[3] = scalar ? in * (r * (s[8] - m1 * s[5] - m2 * s[6]) + s[10] - r * m2 * s[2] - r * mcz * s[0]) : T(0);
    o[4] = in * (r * (s[9] - m1 * s[6] - m2 * s[7]) + s[11] - r * m2 * s[3] - r * mcz * s[1]);
    o[5] = in * (r * (s[4] - m1 * s[2] - m2 * s[3]));
  }
}

// Pointwise result of one vector.  In the backward x and g hold z and c.
template <int KIND, typename T, int VEC, int OP, bool DROP>
__device__ __forceinline__ void gn_apply(const NormArgs& a, const GnCol<T, VEC, OP, DROP>& c, const GnStat<T>& st,
                                         const T* k, const GnRow<T, VEC>& v, int64_t at, int row, T* cw, T* cb) {
  RowVec<T, VEC> o;
  if constexpr (OP == GN_FWD) {
    const uint32_t kp = c.keep(row);
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      T t = c.w[i] * c.template z<KIND>(st, v.x.v[i]);
      if (KIND != GN_PLAIN) t += c.b[i];
      o.v[i] = c.drop(kp, i, KIND == GN_ACT ? t * gn_sigmoid(t) : t);
    }
    store_row<T, VEC>(static_cast<T*>(a.o0) + at, o);
  } else if constexpr (OP == GN_BWD) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const T d = v.g.v[i] - v.x.v[i] * k[1];
      o.v[i] = st.r * (KIND == GN_PLAIN ? d : d - k[0]);
    }
    if (a.o0 != nullptr) store_row<T, VEC>(static_cast<T*>(a.o0) + at, o);
  } else {
    const uint32_t kp = c.keep(row);
    RowVec<T, VEC> dg;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const GnSecond<T> e = gn_second<KIND, T, VEC, DROP>(c, st, kp, i, v.x.v[i], v.g.v[i]);
      const T ux = v.u.v[i], cc = c.w[i] * e.h;
      const T zd = st.r * (ux - k[0] - e.z * k[1]);
      const T td = c.w[i] * zd + c.uw[i] * e.z + c.ub[i];
      const T q = KIND == GN_ACT ? e.q1 * td : T(0);
      const T C = c.w[i] * q + c.uw[i] * e.h - st.r * (k[1] * cc + k[2] * ux);
      dg.v[i] = e.d1 * td;
      o.v[i] = st.r * (C - k[3] - e.z * (k[4] + k[5]));
      cw[i] += q * e.z + e.h * zd;
      cb[i] += q;
    }
    if (a.o0 != nullptr) store_row<T, VEC>(static_cast<T*>(a.o0) + at, o);
    if (a.o1 != nullptr) store_row<T, VEC>(static_cast<T*>(a.o1) + at, dg);
  }
}

// Zero rows [from, to) of the outputs in this thread's column.
template <typename T, int VEC, int OP>
__device__ __forceinline__ void gn_zero_rows(const NormArgs& a, int col, int64_t from, int64_t to, int64_t step) {
  RowVec<T, VEC> zero;
#pragma unroll
  for (int i = 0; i < VEC; ++i) zero.v[i] = T(0);
#pragma unroll 1
  for (int64_t r = from; r < to; r += step) {
    if (a.o0 != nullptr) store_row<T, VEC>(static_cast<T*>(a.o0) + r * a.lay.dim + col, zero);
    if (OP == GN_DBL && a.o1 != nullptr) store_row<T, VEC>(static_cast<T*>(a.o1) + r * a.lay.dim + col, zero);
  }
}

// Column sums of a CTA: thread slots colacc[2 VEC][GN_THREADS] (weights, then biases) added over the row
// lanes of a column into slot `part` of colpart.  All threads call it.
template <int VEC>
__device__ __forceinline__ void gn_store_columns(const NormArgs& a, const double* colacc, int part, int v0, int W,
                                                 int TX, int TY) {
  __syncthreads();
  for (int q = int(threadIdx.x); q < 2 * VEC * W; q += GN_THREADS) {
    const int which = q / (VEC * W), cc = q % (VEC * W), tx = cc / VEC, i = cc % VEC;
    const double* p = colacc + (which * VEC + i) * GN_THREADS + tx;
    double s = 0.0;
    for (int y = 0; y < TY; ++y) s += p[y * TX];
    a.colpart[(2 * int64_t(part) + which) * a.lay.dim + v0 * VEC + cc] = s;
  }
  __syncthreads();
}

// Gradients of the weights and biases of a tile's channels from the column sums of all `parts` CTAs, after
// the grid has met; CTA `rank` of `ranks` takes its share.  A tile holds whole channels.
template <typename T, int VEC>
__device__ __forceinline__ void gn_finish_columns(const NormArgs& a, int parts, int v0, int W, int rank, int ranks) {
  constexpr int WARPS = GN_THREADS / 32;
  const int lane = int(threadIdx.x) % 32, n = W * VEC;
  for (int q = rank * WARPS + int(threadIdx.x) / 32; q < n; q += ranks * WARPS) {
    const int col = v0 * VEC + q;
    const RowBlock& b = a.lay.blk[block_of(a.lay, col)];
    const int u = int(fast_div(uint32_t(col - b.col0), b.div_d));
    if (u * b.d != col - b.col0) continue;
    const bool bias = b.bias0 >= 0 && a.gb != nullptr;
    double sw = 0.0, sb = 0.0;
    for (int p = lane; p < parts; p += 32) {
      const double* r = a.colpart + 2 * int64_t(p) * a.lay.dim + col;
      for (int m = 0; m < b.d; ++m) sw += __ldcg(r + m);
      if (bias) sb += __ldcg(r + a.lay.dim);
    }
    for (int o = 16; o > 0; o /= 2) {
      sw += __shfl_xor_sync(~0u, sw, o);
      sb += __shfl_xor_sync(~0u, sb, o);
    }
    if (lane == 0) {
      if (a.gw != nullptr) static_cast<T*>(a.gw)[b.chan0 + u] = T(sw);
      if (bias) static_cast<T*>(a.gb)[b.bias0 + u] = T(sb);
    }
  }
}

// Local groups of a tile: their vector ranges.
struct GnRange {
  int first, w;
  uint32_t div_w;
};
__device__ __forceinline__ GnRange gn_range(int g0, int g1) {
  GnRange r;
  r.first = g0;
  r.w = g1 - g0;
  r.div_w = r.w > 1 ? 0xFFFFFFFFu / uint32_t(r.w) + 1u : 0u;
  return r;
}

// A tile as its CTA sees it.
struct GnTile {
  int t, v0, W, gfirst, nlg;
};
template <int VEC>
__device__ __forceinline__ GnTile gn_tile(const NormArgs& a, int t) {
  GnTile x;
  x.t = t;
  x.v0 = a.tile[t];
  x.W = a.tile[t + 1] - x.v0;
  x.gfirst = group_of(a.lay, x.v0 * VEC);
  x.nlg = group_of(a.lay, (x.v0 + x.W) * VEC - 1) - x.gfirst + 1;
  return x;
}

// A thread's sums of one segment into its slots of buf.
template <int KIND, int OP, typename T, int VEC, typename ACC, typename COL>
__device__ __forceinline__ void gn_publish(const COL& c, const ACC& acc, T piv, int rows, T* buf, int stride) {
  if constexpr (OP == GN_FWD) {
    T s1 = T(0), s2 = T(0);
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      s1 += acc.s1[i];
      s2 += acc.s2[i];
    }
    if (KIND != GN_PLAIN) {
      const T n = T(rows * VEC), m = rows > 0 ? s1 / n : T(0);
      buf[0] = piv;
      buf[stride] = m;
      buf[2 * stride] = s2 - m * s1;
      buf[3 * stride] = n;
    } else {
      buf[2 * stride] = s2;
    }
  } else if constexpr (OP == GN_BWD) {
    T s1 = T(0), s2 = T(0);
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      s1 += c.w[i] * acc.s2[i];
      s2 += c.w[i] * acc.s1[i];
    }
    buf[0] = s1;
    buf[stride] = s2;
  } else {
#pragma unroll
    for (int i = 0; i < 12; ++i) buf[i * stride] = acc.s[i];
  }
}

// Join E entries: `lanes` consecutive threads share them, entry i's sums are at(i)[0], at(i)[stride], ..; every
// thread of the warp calls it.  All of the lanes get S.
template <int OP, typename T, typename F>
__device__ __forceinline__ void gn_join(int E, int lane, int lanes, int stride, bool scalar, T* S, F at) {
  constexpr int NS = gn_sums(OP);
  if constexpr (OP == GN_FWD) {
    T piv = T(0), mean = T(0), n = T(0), m2 = T(0);
    if (__any_sync(~0u, scalar)) {
      if (scalar && E > 0) {
        piv = *at(0);
#pragma unroll 2
        for (int i = lane; i < E; i += lanes) {
          const T* p = at(i);
          const T cnt = p[3 * stride];
          n += cnt;
          mean += cnt * ((p[0] - piv) + p[stride]);
        }
      }
      for (int o = lanes / 2; o > 0; o /= 2) {
        mean += __shfl_xor_sync(~0u, mean, o);
        n += __shfl_xor_sync(~0u, n, o);
      }
      if (n > T(0)) mean /= n;
    }
#pragma unroll 2
    for (int i = lane; i < E; i += lanes) {
      const T* p = at(i);
      m2 += p[2 * stride];
      if (scalar) {
        const T d = ((p[0] - piv) + p[stride]) - mean;
        m2 += p[3 * stride] * d * d;
      }
    }
    for (int o = lanes / 2; o > 0; o /= 2) m2 += __shfl_xor_sync(~0u, m2, o);
    S[0] = piv;
    S[1] = mean;
    S[2] = m2;
    S[3] = n;
  } else {
#pragma unroll
    for (int p = 0; p < NS; ++p) S[p] = T(0);
#pragma unroll 2
    for (int i = lane; i < E; i += lanes) {
      const T* e = at(i);
#pragma unroll
      for (int p = 0; p < NS; ++p) S[p] += e[p * stride];
    }
    for (int o = lanes / 2; o > 0; o /= 2) {
#pragma unroll
      for (int p = 0; p < NS; ++p) S[p] += __shfl_xor_sync(~0u, S[p], o);
    }
  }
}

// ------------------------------------------------------------------------------------- local ---
// Thread (j, k, tx) owns vector column tx of the CTA's tile and row lane k of segments j, j + J, ..
// (M of them) of the current batch; it keeps R rows of each in registers.  With CL a cluster's CTAs have K
// row lanes each of one segment; each writes its sums into the shared memory of all.
template <typename T, int VEC, int OP, int R, int M, bool CL>
struct GnLocal {
  static constexpr int NS = gn_sums(OP), NC = gn_coefs(OP);
  static constexpr size_t buf_bytes = sizeof(T) * NS * M * GN_THREADS;
  static constexpr size_t res_bytes = sizeof(T) * NC * M * GN_THREADS;
  // sums of a cluster's CTAs, twice: [parity][sum][rank][local group]
  static constexpr int ALL_GROUPS = 32;
  static constexpr size_t all_bytes = CL ? sizeof(T) * 2 * NS * 16 * ALL_GROUPS : 0;
  static constexpr size_t col_bytes = OP == GN_FWD ? 0 : sizeof(double) * 2 * VEC * GN_THREADS;
  static constexpr size_t smem = buf_bytes + res_bytes + all_bytes + col_bytes + sizeof(GnRange) * GN_THREADS;
};

// A thread's part of a batch: rows row0[m] + i step, i < n[m].
template <typename T, int VEC, int R, int M>
struct GnBatch {
  GnRow<T, VEC> v[R * M];
  int row0[M], n[M];
};

template <int KIND, typename T, int VEC, int OP, bool DROP, int R, int M>
__device__ __forceinline__ void gn_local_sums(const GnCol<T, VEC, OP, DROP>& c, const GnStat<T> (&st)[M],
                                              GnBatch<T, VEC, R, M>& t, int step, T* buf, T* cw, T* cb) {
#pragma unroll
  for (int m = 0; m < M; ++m) {
    GnAcc<T, VEC, OP, DROP> acc;
    acc.clear(c);
    const T piv = OP == GN_FWD && KIND != GN_PLAIN && t.n[m] > 0 ? t.v[m * R].x.v[0] : T(0);
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (i < t.n[m]) acc.template add<KIND>(c, st[m], piv, t.v[m * R + i], t.row0[m] + i * step);
    gn_publish<KIND, OP, T, VEC>(c, acc, piv, t.n[m], buf + m * GN_THREADS, M * GN_THREADS);
    if constexpr (OP == GN_BWD) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        cw[i] += acc.s1[i];
        if (KIND != GN_PLAIN) cb[i] += acc.s2[i];
      }
    }
  }
}

template <int KIND, typename T, int VEC, int OP, bool DROP, int R, int M>
__device__ __forceinline__ void gn_local_apply(const NormArgs& a, const GnCol<T, VEC, OP, DROP>& c,
                                               GnStat<T> (&st)[M], GnBatch<T, VEC, R, M>& t, int step, const T* res,
                                               int res_step, T* cw, T* cb) {
  constexpr int NC = gn_coefs(OP);
#pragma unroll
  for (int m = 0; m < M; ++m) {
    T kf[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) kf[i] = res[m * res_step + i];
    if (OP == GN_FWD) {
      st[m].hi = kf[0];
      st[m].lo = kf[1];
      st[m].r = kf[2];
    }
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (i < t.n[m]) {
        const int r = t.row0[m] + i * step;
        gn_apply<KIND>(a, c, st[m], kf, t.v[m * R + i], int64_t(r) * a.lay.dim + c.col, r, cw, cb);
      }
  }
}

// CTAs that have to fit an SM: what the registers of a batch allow
__host__ __device__ constexpr int gn_local_ctas(int op, int m) { return op == GN_FWD ? 3 : m > 1 ? 3 : 2; }

template <typename T, int VEC, int OP, bool DROP, int R, int M, bool CL>
__global__ void __launch_bounds__(GN_THREADS, gn_local_ctas(OP, M))
gn_local_kernel(const __grid_constant__ NormArgs a) {
  using L = GnLocal<T, VEC, OP, R, M, CL>;
  constexpr int NS = L::NS, NC = L::NC, STRIDE = M * GN_THREADS;
  extern __shared__ __align__(16) unsigned char smem[];
  double* colbase = reinterpret_cast<double*>(smem);
  T* buf = reinterpret_cast<T*>(smem + L::col_bytes);
  T* res = buf + NS * STRIDE;
  T* all = res + NC * STRIDE;
  GnRange* gs = reinterpret_cast<GnRange*>(smem + L::col_bytes + L::buf_bytes + L::res_bytes + L::all_bytes);
  const int CS = CL ? a.cs : 1, rank = CL ? int(blockIdx.x) % CS : 0;
  const int part = CL ? int(blockIdx.x) / CS : int(blockIdx.x), parts = CL ? int(gridDim.x) / CS : int(gridDim.x);
  const int tid = int(threadIdx.x), tx = tid % a.tx, ty = tid / a.tx;
  const int K = a.k, step = K * CS, J = a.j;
  const int v0 = a.tile[blockIdx.y], W = a.tile[blockIdx.y + 1] - v0;
  const int j = ty / K, k = rank * K + ty - j * K;
  const bool active = tx < W && j < J;
  const int64_t G = a.lay.n_groups();

  GnCol<T, VEC, OP, DROP> c;
  c.col = (v0 + (active ? tx : 0)) * VEC;
  GnBatch<T, VEC, R, M> t;
  const uint32_t div_step = step > 1 ? 0xFFFFFFFFu / uint32_t(step) + 1u : 0u;
  // rows of the batch of segments b0 .. and their loads
  auto fetch = [&](int64_t b0) {
#pragma unroll
    for (int m = 0; m < M; ++m) {
      t.n[m] = 0;
      const int64_t b = b0 + m * J + j;
      if (active && b < a.B) {
        int s, e;
        gn_segment(a, int(b), s, e);
        if (e - s > R * step) {  // longer than the caller said
          atomicCAS(a.status, 0, int(E3_ERR_INDEX));
          e = s + R * step;
        }
        t.row0[m] = s + k;
        const int left = e - s - k + step - 1;
        t.n[m] = left > 0 ? (R == 1 ? (e > s + k) : int(fast_div(uint32_t(left), div_step))) : 0;
      }
    }
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (i < t.n[m])
          gn_load<T, VEC, OP>(a, int64_t(t.row0[m] + i * step) * a.lay.dim + c.col, t.v[m * R + i]);
  };
  int64_t b0 = int64_t(part) * (J * M);
  fetch(b0);

  c.init(a, v0, W, active ? tx : 0);
  const int gfirst = c.g - c.lg, nlg = group_of(a.lay, (v0 + W) * VEC - 1) - gfirst + 1;
  if (active && ty == 0 && tx == c.g0) gs[c.lg] = gn_range(c.g0, c.g1);
  const bool columns = OP != GN_FWD && a.colpart != nullptr;
  T cw[VEC], cb[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) cw[i] = cb[i] = T(0);
  if (columns) {
#pragma unroll
    for (int i = 0; i < 2 * VEC; ++i) colbase[i * GN_THREADS + tid] = 0.0;
  }
  const uint32_t div_nlg = nlg > 1 ? 0xFFFFFFFFu / uint32_t(nlg) + 1u : 0u;
  const uint32_t div_j = J > 1 ? 0xFFFFFFFFu / uint32_t(J) + 1u : 0u;
  const int lane = tid & (a.lanes - 1), sub = tid / a.lanes, per = GN_THREADS / a.lanes;
  const int items = M * J * nlg;
  int rows_held = 0, parity = 0;
  if (CL) cooperative_groups::this_cluster().sync();  // every CTA of the cluster has started
  for (; b0 < a.B; parity ^= 1) {
    GnStat<T> st[M];
    if (OP != GN_FWD) {
#pragma unroll
      for (int m = 0; m < M; ++m) {
        const int64_t b = b0 + m * J + j;
        if (t.n[m] > 0) st[m].set(a.stats + 2 * (b * G + c.g));
      }
    }
    if (c.kind == GN_PLAIN) gn_local_sums<GN_PLAIN>(c, st, t, step, buf + tid, cw, cb);
    else if (c.kind == GN_CENTRED) gn_local_sums<GN_CENTRED>(c, st, t, step, buf + tid, cw, cb);
    else gn_local_sums<GN_ACT>(c, st, t, step, buf + tid, cw, cb);
    __syncthreads();
    // item (m, jj, lg): K row lanes x the group's vectors
    for (int base = 0; base < items; base += per) {
      const int it = base + sub, mj = int(fast_div(uint32_t(it), div_nlg)), lg = it - mj * nlg;
      const int m = M == 1 ? 0 : int(fast_div(uint32_t(mj), div_j)), jj = mj - m * J;
      const int64_t b = b0 + mj;
      const bool ok = it < items && b < a.B;
      const int g = gfirst + lg;
      const RowBlock& blk = a.lay.blk[fast_div(uint32_t(g), a.lay.div_groups)];
      const bool scalar = blk.bias0 >= 0;
      GnRange gr{0, 1, 0};
      if (ok) gr = gs[lg];
      const T* q = buf + m * GN_THREADS + jj * K * a.tx + gr.first;
      const int hop = a.tx - gr.w;
      T S[NS];
      gn_join<OP, T>(ok ? K * gr.w : 0, lane, a.lanes, STRIDE, scalar, S,
                     [&](int i) { return q + i + (K > 1 ? int(fast_div(uint32_t(i), gr.div_w)) * hop : 0); });
      if (CL) {
        // lane r hands the sums to rank r
        if (ok) {
          for (int r = lane; r < CS; r += a.lanes) {
            T* to = cooperative_groups::this_cluster().map_shared_rank(all, r) +
                    (parity * NS * 16 + rank) * L::ALL_GROUPS + lg;
#pragma unroll
            for (int p = 0; p < NS; ++p) to[p * 16 * L::ALL_GROUPS] = S[p];
          }
        }
      } else if (ok && lane == 0) {
        int s = 0, e = int(a.N);
        if (a.row_ptr != nullptr) gn_segment(a, int(b), s, e);
        gn_finish<OP, T>(S, T(e - s) * T(blk.group_cols), scalar, a.stats + 2 * (b * G + g), true, a.eps,
                         res + NC * it);
      }
    }
    if (CL) {
      cooperative_groups::this_cluster().sync();
      for (int base = 0; base < nlg; base += GN_THREADS / 16) {
        const int lg = base + tid / 16, g = gfirst + (lg < nlg ? lg : 0);
        const RowBlock& blk = a.lay.blk[fast_div(uint32_t(g), a.lay.div_groups)];
        const bool scalar = blk.bias0 >= 0;
        const T* q = all + parity * NS * 16 * L::ALL_GROUPS + lg;
        T S[NS];
        gn_join<OP, T>(lg < nlg ? CS : 0, tid % 16, 16, 16 * L::ALL_GROUPS, scalar, S,
                       [&](int i) { return q + i * L::ALL_GROUPS; });
        if (lg < nlg && tid % 16 == 0) {
          int s = 0, e = int(a.N);
          if (a.row_ptr != nullptr) gn_segment(a, int(b0), s, e);
          gn_finish<OP, T>(S, T(e - s) * T(blk.group_cols), scalar, a.stats + 2 * (b0 * G + g), rank == 0, a.eps,
                           res + NC * lg);
        }
      }
    }
    __syncthreads();
    {
      const T* q = res + NC * ((active ? j : 0) * nlg + c.lg);
      const int res_step = NC * J * nlg;
      if (c.kind == GN_PLAIN) gn_local_apply<GN_PLAIN>(a, c, st, t, step, q, res_step, cw, cb);
      else if (c.kind == GN_CENTRED) gn_local_apply<GN_CENTRED>(a, c, st, t, step, q, res_step, cw, cb);
      else gn_local_apply<GN_ACT>(a, c, st, t, step, q, res_step, cw, cb);
    }
    rows_held += R * M;
    if (columns && rows_held >= GN_FLUSH) {
      rows_held = 0;
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        colbase[i * GN_THREADS + tid] += double(cw[i]);
        colbase[(VEC + i) * GN_THREADS + tid] += double(cb[i]);
        cw[i] = cb[i] = T(0);
      }
    }
    b0 += int64_t(parts) * (J * M);
    fetch(b0);
  }
  if (active)
    gn_zero_rows<T, VEC, OP>(a, c.col, gn_rows_end(a) + int64_t(blockIdx.x) * (J * K) + ty, a.N,
                             int64_t(gridDim.x) * (J * K));
  if (columns) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      colbase[i * GN_THREADS + tid] += double(cw[i]);
      colbase[(VEC + i) * GN_THREADS + tid] += double(cb[i]);
    }
    gn_store_columns<VEC>(a, colbase, int(blockIdx.x), v0, W, a.tx, J * K);
    cooperative_groups::this_grid().sync();
    gn_finish_columns<T, VEC>(a, int(gridDim.x), v0, W, int(blockIdx.x), int(gridDim.x));
  }
}

// -------------------------------------------------------------------------------------- grid ---
// CTA (rc, ct): row chunk rc, column tile s cx + ct of slab s.  A segment that lies in one chunk is
// finished there (unless its group is cut into tiles); the others leave partial sums:
//   slot of (chunk, segment), part of (tile, group):  part[slot][groups + tiles][sums]
// slots: 2 chunk (the segment began earlier) or 2 chunk + 1 (it begins here and goes on); with cut
// groups chunk + segment, which rises by one from piece to piece.  Parts likewise are group + tile.
template <int OP, typename T>
__device__ __forceinline__ T* gn_slot(const NormArgs& a, int chunk, int64_t b, bool begins, int tile, int g) {
  const int64_t G = a.lay.n_groups();
  const int64_t slot = a.wide ? chunk + b : 2 * int64_t(chunk) + (begins ? 1 : 0);
  return static_cast<T*>(a.part) + (slot * (G + a.n_tiles) + g + tile) * gn_sums(OP);
}

// Last segment that starts at or before row r.
__device__ __forceinline__ int gn_first_segment(const NormArgs& a, int r) {
  if (a.row_ptr == nullptr) return 0;
  int lo = 0, hi = a.B - 1;
  while (lo < hi) {
    const int m = lo + (hi - lo + 1) / 2;
    if (a.row_ptr[m] <= r) lo = m;
    else hi = m - 1;
  }
  return lo;
}

template <typename T, int VEC, int OP>
struct GnGrid {
  static constexpr int NS = gn_sums(OP), NC = gn_coefs(OP);
  static constexpr int U = OP == GN_FWD ? 8 : OP == GN_BWD ? 4 : 2;  // rows in flight per thread
  static constexpr size_t long_bytes = OP == GN_DBL ? sizeof(double) * NS * GN_THREADS : 0;
  static constexpr size_t buf_bytes = sizeof(T) * NS * GN_THREADS;
  static constexpr size_t res_bytes = sizeof(T) * NC * GN_THREADS;
  static constexpr size_t col_bytes = OP == GN_FWD ? 0 : sizeof(double) * 2 * VEC * GN_THREADS;
  static constexpr size_t smem = long_bytes + col_bytes + buf_bytes + res_bytes + sizeof(GnRange) * GN_THREADS;
};
struct GnGridSmem {
  double *sums, *columns;  // a thread's long sums (double backward) and column sums
  void *buf, *res;
  GnRange* gs;
};

// A thread's sums over rows s + ty, s + ty + K, .. of a piece into its slots of buf (and of the columns).
template <int KIND, typename T, int VEC, int OP, bool DROP>
__device__ __forceinline__ void gn_grid_sums(const NormArgs& a, const GnCol<T, VEC, OP, DROP>& c, const GnStat<T>& st,
                                             int s, int e, int ty, int K, T* buf, double* sums, double* colacc) {
  constexpr int U = GnGrid<T, VEC, OP>::U;
  const int64_t D = a.lay.dim;
  T piv = T(0);
  if (OP == GN_FWD && KIND != GN_PLAIN && s + ty < e) piv = static_cast<const T*>(a.x)[(s + ty) * D + c.col];
  GnAcc<T, VEC, OP, DROP> acc;
  acc.clear(c);
  double l1 = 0.0, l2 = 0.0;  // the sums of earlier flushes
  if (OP == GN_DBL) {
#pragma unroll
    for (int i = 0; i < 12; ++i) sums[i * GN_THREADS] = 0.0;
  }
#pragma unroll 1
  for (int f = s + ty; f < e; f += K * GN_FLUSH) {
    const int fe = min(e, f + K * GN_FLUSH);
#pragma unroll 1
    for (int r = f; r < fe; r += K * U) {
      GnRow<T, VEC> v[U];
#pragma unroll
      for (int i = 0; i < U; ++i)  // past the end: the last row again
        gn_load<T, VEC, OP>(a, min(r + i * K, fe - 1) * D + c.col, v[i]);
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (r + i * K < fe) acc.template add<KIND>(c, st, piv, v[i], r + i * K);
    }
    if constexpr (OP == GN_FWD) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        l1 += double(acc.s1[i]);
        l2 += double(acc.s2[i]);
      }
      acc.clear(c);
    } else if constexpr (OP == GN_BWD) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        l1 += double(c.w[i]) * double(acc.s2[i]);
        l2 += double(c.w[i]) * double(acc.s1[i]);
        if (colacc != nullptr) {
          colacc[i * GN_THREADS] += double(acc.s1[i]);
          if (KIND != GN_PLAIN) colacc[(VEC + i) * GN_THREADS] += double(acc.s2[i]);
        }
      }
      acc.clear(c);
    } else {
#pragma unroll
      for (int i = 0; i < 12; ++i) sums[i * GN_THREADS] += double(acc.s[i]);
      acc.clear(c);
    }
  }
  if constexpr (OP == GN_FWD) {
    const int rows = s + ty < e ? (e - s - ty + K - 1) / K : 0;
    const double n = double(rows) * VEC, m = KIND != GN_PLAIN && rows > 0 ? l1 / n : 0.0;
    buf[0] = piv;
    buf[GN_THREADS] = T(m);
    buf[2 * GN_THREADS] = T(l2 - m * l1);
    buf[3 * GN_THREADS] = T(n);
  } else if constexpr (OP == GN_BWD) {
    buf[0] = T(l1);
    buf[GN_THREADS] = T(l2);
  } else {
#pragma unroll
    for (int i = 0; i < 12; ++i) buf[i * GN_THREADS] = T(sums[i * GN_THREADS]);
  }
}

template <int KIND, typename T, int VEC, int OP, bool DROP>
__device__ __forceinline__ void gn_grid_apply(const NormArgs& a, const GnCol<T, VEC, OP, DROP>& c, const GnStat<T>& st,
                                              const T* kf, int s, int e, int ty, int K, double* colacc) {
  constexpr int U = GnGrid<T, VEC, OP>::U;
  const int64_t D = a.lay.dim;
  if (OP == GN_BWD && a.o0 == nullptr) return;
#pragma unroll 1
  for (int f = s + ty; f < e; f += K * GN_FLUSH) {
    const int fe = min(e, f + K * GN_FLUSH);
    T cw[VEC], cb[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) cw[i] = cb[i] = T(0);
#pragma unroll 1
    for (int r = f; r < fe; r += K * U) {
      GnRow<T, VEC> v[U];
#pragma unroll
      for (int i = 0; i < U; ++i) gn_load<T, VEC, OP>(a, min(r + i * K, fe - 1) * D + c.col, v[i]);
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (r + i * K < fe) {
          if constexpr (OP == GN_BWD) {  // z and c again
            GnAcc<T, VEC, OP, DROP> z;
            z.clear(c);
            z.template add<KIND>(c, st, T(0), v[i], r + i * K);
          }
          gn_apply<KIND>(a, c, st, kf, v[i], (r + i * K) * D + c.col, r + i * K, cw, cb);
        }
    }
    if (OP == GN_DBL && colacc != nullptr) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        colacc[i * GN_THREADS] += double(cw[i]);
        colacc[(VEC + i) * GN_THREADS] += double(cb[i]);
      }
    }
  }
}

// First pass over rows [lo, hi) of a tile.
template <typename T, int VEC, int OP, bool DROP>
__device__ __forceinline__ void gn_grid_first(const NormArgs& a, const GnTile& tl, int rc, int lo, int hi,
                                              const GnGridSmem& sm) {
  constexpr int NS = gn_sums(OP), NC = gn_coefs(OP);
  const int tid = int(threadIdx.x), tx = tid % a.tx, ty = tid / a.tx;
  const int64_t G = a.lay.n_groups();
  const bool active = tx < tl.W && ty < a.k;
  T* buf = static_cast<T*>(sm.buf);
  GnCol<T, VEC, OP, DROP> c;
  c.init(a, tl.v0, tl.W, active ? tx : 0);
  __syncthreads();
  if (active && ty == 0 && tx == c.g0) sm.gs[c.lg] = gn_range(c.g0, c.g1);
  double* colacc = nullptr;
  if (OP == GN_BWD && a.colpart != nullptr) {
    colacc = sm.columns + tid;
#pragma unroll
    for (int i = 0; i < 2 * VEC; ++i) colacc[i * GN_THREADS] = 0.0;
  }
  const int lane = tid & (a.lanes - 1), sub = tid / a.lanes, per = GN_THREADS / a.lanes;
#pragma unroll 1
  for (int b = gn_first_segment(a, lo); b < a.B; ++b) {
    int s, e;
    gn_segment(a, b, s, e);
    if (s >= hi) break;
    const int ps = max(s, lo), pe = min(e, hi);
    if (ps >= pe) continue;
    if (active) {
      GnStat<T> st;
      if (OP != GN_FWD) st.set(a.stats + 2 * (b * G + c.g));
      if (c.kind == GN_PLAIN)
        gn_grid_sums<GN_PLAIN>(a, c, st, ps, pe, ty, a.k, buf + tid, sm.sums + tid, colacc);
      else if (c.kind == GN_CENTRED)
        gn_grid_sums<GN_CENTRED>(a, c, st, ps, pe, ty, a.k, buf + tid, sm.sums + tid, colacc);
      else gn_grid_sums<GN_ACT>(a, c, st, ps, pe, ty, a.k, buf + tid, sm.sums + tid, colacc);
    }
    __syncthreads();
    const bool whole = ps == s && pe == e && !a.wide;
    for (int base = 0; base < tl.nlg; base += per) {
      const int lg = base + sub, g = tl.gfirst + (lg < tl.nlg ? lg : 0);
      const RowBlock& blk = a.lay.blk[fast_div(uint32_t(g), a.lay.div_groups)];
      const bool scalar = blk.bias0 >= 0;
      GnRange gr{0, 1, 0};
      if (lg < tl.nlg) gr = sm.gs[lg];
      T S[NS];
      gn_join<OP, T>(lg < tl.nlg ? a.k * gr.w : 0, lane, a.lanes, GN_THREADS, scalar, S, [&](int i) {
        const int kk = int(fast_div(uint32_t(i), gr.div_w));
        return buf + kk * a.tx + gr.first + i - kk * gr.w;
      });
      if (lg < tl.nlg && lane == 0) {
        if (whole) {
          T o[NC];
          gn_finish<OP, T>(S, T(e - s) * T(blk.group_cols), scalar, a.stats + 2 * (b * G + g), true, a.eps, o);
          if (OP != GN_FWD) {
            T* dst = static_cast<T*>(a.coef) + NC * (b * G + g);
#pragma unroll
            for (int p = 0; p < NC; ++p) dst[p] = o[p];
          }
        } else {
          T* dst = gn_slot<OP, T>(a, rc, b, s >= lo, tl.t, g);
#pragma unroll
          for (int p = 0; p < NS; ++p) dst[p] = S[p];
        }
      }
    }
    __syncthreads();
  }
  if (OP == GN_BWD && a.colpart != nullptr) gn_store_columns<VEC>(a, sm.columns, rc, tl.v0, tl.W, a.tx, a.k);
}

// res[lg] = coefficients of segment b (rows [s, e)), whose sums are spread over chunks and tiles.
template <int VEC, int OP, typename T>
__device__ __forceinline__ void gn_grid_join(const NormArgs& a, const GnTile& tl, int rc, int b, int s, int e, T* res) {
  constexpr int NS = gn_sums(OP), NC = gn_coefs(OP);
  const int c0 = int(s / a.rows_cta), nc = int((e - 1) / a.rows_cta) - c0 + 1;
  const int lanes = nc > 16 || a.wide ? 32 : nc > 8 ? 16 : 8;
  const int sub = int(threadIdx.x) / lanes, lane = int(threadIdx.x) % lanes;
  for (int base = 0; base < tl.nlg; base += GN_THREADS / lanes) {
    const int lg = base + sub, g = tl.gfirst + (lg < tl.nlg ? lg : 0);
    const RowBlock& blk = a.lay.blk[fast_div(uint32_t(g), a.lay.div_groups)];
    const bool scalar = blk.bias0 >= 0;
    int t0 = tl.t, nt = 1;
    if (a.wide) {  // the tiles that hold parts of this group
      while (t0 > 0 && group_of(a.lay, a.tile[t0] * VEC - 1) == g) --t0;
      while (t0 + nt < a.n_tiles && group_of(a.lay, a.tile[t0 + nt] * VEC) == g) ++nt;
    }
    T S[NS];
    gn_join<OP, T>(lg < tl.nlg ? nc * nt : 0, lane, lanes, 1, scalar, S, [&](int i) {
      const int ch = c0 + (nt == 1 ? i : i / nt);
      return gn_slot<OP, T>(a, ch, b, ch == c0, t0 + (nt == 1 ? 0 : i % nt), g);
    });
    if (lg < tl.nlg && lane == 0)
      gn_finish<OP, T>(S, T(e - s) * T(blk.group_cols), scalar,
                       a.stats + 2 * (int64_t(b) * a.lay.n_groups() + g), rc == c0, a.eps, res + NC * lg);
  }
}

// Second pass over rows [lo, hi) of a tile.
template <typename T, int VEC, int OP, bool DROP>
__device__ __forceinline__ void gn_grid_second(const NormArgs& a, const GnTile& tl, int rc, int lo, int hi,
                                               const GnGridSmem& sm) {
  constexpr int NC = gn_coefs(OP);
  const int tid = int(threadIdx.x), tx = tid % a.tx, ty = tid / a.tx;
  const int64_t G = a.lay.n_groups();
  const bool active = tx < tl.W && ty < a.k;
  T* res = static_cast<T*>(sm.res);
  GnCol<T, VEC, OP, DROP> c;
  c.init(a, tl.v0, tl.W, active ? tx : 0);
  double* colacc = nullptr;
  if (OP == GN_DBL && a.colpart != nullptr) {
    colacc = sm.columns + tid;
#pragma unroll
    for (int i = 0; i < 2 * VEC; ++i) colacc[i * GN_THREADS] = 0.0;
  }
#pragma unroll 1
  for (int b = gn_first_segment(a, lo); b < a.B; ++b) {
    int s, e;
    gn_segment(a, b, s, e);
    if (s >= hi) break;
    const int ps = max(s, lo), pe = min(e, hi);
    if (ps >= pe) continue;
    const bool whole = ps == s && pe == e && !a.wide;
    if (!whole) {
      __syncthreads();
      gn_grid_join<VEC, OP, T>(a, tl, rc, b, s, e, res);
      __syncthreads();
    }
    if (!active) continue;
    GnStat<T> st;
    T kf[NC];
    const T* q = whole ? static_cast<const T*>(a.coef) + NC * (b * G + c.g) : res + NC * c.lg;
#pragma unroll
    for (int i = 0; i < NC; ++i) kf[i] = OP == GN_FWD && whole ? T(0) : q[i];
    if (OP == GN_FWD && !whole) {
      st.hi = kf[0];
      st.lo = kf[1];
      st.r = kf[2];
    } else {
      st.set(a.stats + 2 * (b * G + c.g));
    }
    if (c.kind == GN_PLAIN) gn_grid_apply<GN_PLAIN>(a, c, st, kf, ps, pe, ty, a.k, colacc);
    else if (c.kind == GN_CENTRED) gn_grid_apply<GN_CENTRED>(a, c, st, kf, ps, pe, ty, a.k, colacc);
    else gn_grid_apply<GN_ACT>(a, c, st, kf, ps, pe, ty, a.k, colacc);
  }
  if (active) gn_zero_rows<T, VEC, OP>(a, c.col, max(lo, gn_rows_end(a)) + ty, hi, a.k);
  if (OP == GN_BWD && a.colpart != nullptr) gn_finish_columns<T, VEC>(a, a.chunks, tl.v0, tl.W, rc, a.chunks);
  if (OP == GN_DBL && a.colpart != nullptr) gn_store_columns<VEC>(a, sm.columns, rc, tl.v0, tl.W, a.tx, a.k);
}

template <typename T, int VEC, int OP, bool DROP>
__global__ void __launch_bounds__(GN_THREADS, OP == GN_FWD ? 3 : 2) gn_grid_kernel(const __grid_constant__ NormArgs a) {
  using L = GnGrid<T, VEC, OP>;
  extern __shared__ __align__(16) unsigned char smem[];
  unsigned char* at = smem;
  GnGridSmem sm;
  sm.sums = reinterpret_cast<double*>(at);
  sm.columns = reinterpret_cast<double*>(at += L::long_bytes);
  sm.buf = at += L::col_bytes;
  sm.res = at += L::buf_bytes;
  sm.gs = reinterpret_cast<GnRange*>(at += L::res_bytes);
  const int rc = int(blockIdx.x) / a.cx, ct = int(blockIdx.x) % a.cx;
  const int lo = int(min(a.N, rc * a.rows_cta)), hi = int(min(a.N, (rc + 1) * a.rows_cta));
  auto grid = cooperative_groups::this_grid();
  const int slabs = (a.n_tiles + a.cx - 1) / a.cx;
  // a CTA that has left its sums of slab s goes on with the second pass of slab s - 1 before it waits
#pragma unroll 1
  for (int s = 0; s <= slabs; ++s) {
    const int now = s * a.cx + ct, last = now - a.cx;
    if (now < a.n_tiles) gn_grid_first<T, VEC, OP, DROP>(a, gn_tile<VEC>(a, now), rc, lo, hi, sm);
    cooperative_groups::grid_group::arrival_token token{};
    if (s < slabs) token = grid.barrier_arrive();
    if (s > 0 && last < a.n_tiles) gn_grid_second<T, VEC, OP, DROP>(a, gn_tile<VEC>(a, last), rc, lo, hi, sm);
    if (s < slabs) grid.barrier_wait(std::move(token));
  }
  if (OP == GN_DBL && a.colpart != nullptr) {
    grid.sync();
    for (int t = ct; t < a.n_tiles; t += a.cx)
      gn_finish_columns<T, VEC>(a, a.chunks, a.tile[t], a.tile[t + 1] - a.tile[t], rc, a.chunks);
  }
}

}  // namespace e3b
