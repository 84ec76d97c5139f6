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
//          shared memory between the passes (one read);
//   grid   longer segments: the CTAs of a resident grid leave partial sums of row chunks x column
//          tiles, meet, join them, meet, and read their rows again.
// Measured (B200, float32, one call): local, 24000 one-row segments of 2048 columns, forward 97 us = 4.1 TB/s
// (62% of a copy): two CTAs of 512 threads, bound by the chain from barrier to barrier; 512 segments of 34 rows x
// 512 columns with dropout, forward 29 us and backward 51 us.  Grid, one segment of 24000 x 2048: forward 108 us
// (590 MB in three passes), backward 190 us with dropout (983 MB in five).  L2 serves a part of the second reads: with
// dropout 494 and 909 MB pass DRAM, 50 and 60 % of its rate under ncu, so the forward is bound by the latency of
// memory (20 warps an SM), the backward by its instructions (16), and neither by DRAM.
// Tried for the grid kernel and dropped: slabs of columns small enough for L2, one after another (24, 50, 100 MB:
// forward 197, 152, 136 us; a meeting and a join per slab, and narrow tiles, cost more than the re-read; L2 also keeps
// only about 60 MB of what one pass read for the next); rows through registers instead of cp.async; sharing the
// dropout words of neighbouring vectors within a warp (forward 127 to 123 us, backward 190 to 203).
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
constexpr int GN_FLUSH = 64;     // rows that a thread sums in the rows' type
constexpr int GN_MAXTILE = 512;  // column tiles at most
constexpr int GN_LOCAL_TILES = 64;  // of the local kernel
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
  void* coef;              // grid: [B][groups][coefs] (backwards)
  double* colpart;         // sums for gw, gb per column, by CTA (NULL: not wanted)
  double eps;
  int32_t act;
  int* status;
  int32_t tx, k, j, lanes;  // thread layout: columns, row lanes of a segment, segments, lanes of a join
  int32_t cs, cap;          // local: CTAs of a cluster; rows of a segment that a thread may have
  int32_t wide;             // grid: some group is cut into several tiles
  int32_t n_tiles;          // tiles of columns
  int32_t tile_groups;      // most groups that a tile holds (parts of)
  int32_t chunks;           // grid: row chunks
  int64_t rows_cta;         // grid: rows of a chunk
  int32_t parts;            // grid: parts of a chunk in the second pass
  int32_t* tickets;         // by tile.  grid: its next part; clusters: CTAs that have left their column sums (0 before)
  DropArgs drop;
  RowLayout lay;
  int32_t tile[GN_MAXTILE + 1];  // first vector column of each tile
  int32_t start[GN_LOCAL_TILES + 1];  // local: first CTA of each tile
  int32_t even;                       // local: all tiles have the same number of CTAs (blockIdx.y: the tile)
  int32_t meet;                       // local: the parameters' gradients add up more CTAs than one cluster
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
    return DROP ? (DropCol<VEC>::kept(kp, i) ? v * scale : T(0)) : v;
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

// Rows on their way through shared memory.  Every thread copies (cp.async) the vectors it will read
// itself into slots of its own, so no barrier is needed, and many rows are in flight without
// registers: slot i of a thread holds its vectors of one row, at base + i * SLOT.
template <typename T, int VEC, int OP, int NT = GN_THREADS>
struct GnSlots {
  static constexpr int ARRAYS = OP + 1;
  static constexpr int LANE = int(sizeof(T)) * VEC;        // bytes of a vector
  static constexpr int SLOT = ARRAYS * LANE * NT;  // bytes of a slot of all threads
  unsigned char* base;  // this thread's vector of slot 0
  const unsigned char *x, *g, *u;

  __device__ __forceinline__ void init(const NormArgs& a, unsigned char* smem) {
    base = smem + int(threadIdx.x) * LANE;
    x = static_cast<const unsigned char*>(a.x);
    g = static_cast<const unsigned char*>(a.g);
    u = static_cast<const unsigned char*>(a.u);
  }
  static __device__ __forceinline__ void copy(unsigned char* to, const unsigned char* from) {
    const uint32_t d = uint32_t(__cvta_generic_to_shared(to));
    if constexpr (LANE == 16)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(from) : "memory");
    else
      asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(d), "l"(from), "n"(LANE) : "memory");
  }
  // start copying the vectors at byte `at` of the rows
  __device__ __forceinline__ void fetch(int slot, int64_t at) const {
    unsigned char* to = base + slot * SLOT;
    copy(to, x + at);
    if (OP != GN_FWD) copy(to + LANE * NT, g + at);
    if (OP == GN_DBL && u != nullptr) copy(to + 2 * LANE * NT, u + at);
  }
  static __device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
  template <int N>
  static __device__ __forceinline__ void wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
  }
  // the vectors at column `col` of rows row, row + step, .. into slots 0 .., waiting for them
  __device__ __forceinline__ void reload(int row, int n, int step, int dim, int col) const {
    int64_t at = (int64_t(row) * dim + col) * int64_t(sizeof(T));
    for (int i = 0; i < n; ++i, at += int64_t(step) * dim * int64_t(sizeof(T))) fetch(i, at);
    commit();
    wait<0>();
  }
  __device__ __forceinline__ RowVec<T, VEC> get(int slot, int array) const {
    return load_row<T, VEC>(reinterpret_cast<const T*>(base + slot * SLOT + array * LANE * NT));
  }
  __device__ __forceinline__ void read(int slot, GnRow<T, VEC>& v) const {
    v.x = get(slot, 0);
    if (OP != GN_FWD) v.g = get(slot, 1);
    if (OP == GN_DBL) {
      if (u != nullptr) {
        v.u = get(slot, 2);
      } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) v.u.v[i] = T(0);
      }
    }
  }
  __device__ __forceinline__ void write(int slot, int array, const RowVec<T, VEC>& v) const {
    store_row<T, VEC>(reinterpret_cast<T*>(base + slot * SLOT + array * LANE * NT), v);
  }
};

// A product that is rounded by itself, never fused into a sum.  The double backward takes differences of sums that
// cancel altogether in a group of one even scalar (z = 0, so nothing depends on x there, while r is up to
// eps^(-1/2)): both sides have to round alike.
__device__ __forceinline__ float gn_mul(float a, float b) { return __fmul_rn(a, b); }
__device__ __forceinline__ double gn_mul(double a, double b) { return __dmul_rn(a, b); }
__device__ __forceinline__ float gn_fma(float a, float b, float c) { return __fmaf_rn(a, b, c); }
__device__ __forceinline__ double gn_fma(double a, double b, double c) { return __fma_rn(a, b, c); }

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
      T q = gn_mul(c.uw[i], e.h);
      s[1] += e.z * ux;
      s[3] += cc * e.z;
      s[4] += cc * ux;
      if (KIND != GN_PLAIN) {
        s[0] += ux;
        s[2] += cc;
      }
      if (KIND == GN_ACT) {
        const T wq = c.w[i] * c.w[i] * e.q1;
        q = gn_fma(c.w[i], gn_mul(e.q1, gn_fma(c.uw[i], e.z, c.ub[i])), q);
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

__device__ __forceinline__ float gn_rsqrt(float v) {
  const float r = rsqrtf(v);
  const float n = fmaf(0.5f * r, fmaf(-v * r, r, 1.f), r);  // one Newton step: the hardware's result is 2 ulp off
  return r > 0.f ? n : r;                                   // 0 for an infinite v, where the step is inf * 0
}
__device__ __forceinline__ double gn_rsqrt(double v) { return 1.0 / sqrt(v); }
__device__ __forceinline__ float gn_recip(float v) { return __fdividef(1.f, v); }
__device__ __forceinline__ double gn_recip(double v) { return 1.0 / v; }

// The second pass' coefficients of a (segment, group) from its joined sums S and its n values.  `r` is the
// stored one (double backward only).
template <int OP, typename T>
__device__ __forceinline__ void gn_finish(const T* s, T n, bool scalar, T r, T eps, T* o) {
  const T in = n > T(0) ? gn_recip(n) : T(0);
  if (OP == GN_FWD) {
    // pivot + (mean - pivot) as a high and a low part (their exact sum: Knuth, TAOCP 2, 4.2.2)
    const T hi = s[0] + s[1], back = hi - s[0];
    o[0] = hi;
    o[1] = (s[0] - (hi - back)) + (s[1] - back);
    o[2] = gn_rsqrt(s[2] * in + eps);
  } else if (OP == GN_BWD) {
    o[0] = scalar ? s[0] * in : T(0);
    o[1] = s[1] * in;
  } else {
    const T m1 = scalar ? s[0] * in : T(0), m2 = s[1] * in, mcz = s[3] * in;
    o[0] = m1;
    o[1] = m2;
    o[2] = mcz;
    o[3] = scalar ? in * (r * (s[8] - gn_mul(m1, s[5]) - m2 * s[6]) + s[10] - r * m2 * s[2] - r * mcz * s[0]) : T(0);
    o[4] = in * (r * (s[9] - m1 * s[6] - m2 * s[7]) + s[11] - r * m2 * s[3] - r * mcz * s[1]);
    o[5] = in * (r * (s[4] - m1 * s[2] - m2 * s[3]));
  }
}
// (mean, r) of the forward as the caller keeps them.
template <typename T>
__device__ __forceinline__ void gn_store_stats(const T* o, double* sg) {
  sg[0] = double(o[0]) + double(o[1]);
  sg[1] = double(o[2]);
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
    store_row_last<T, VEC>(static_cast<T*>(a.o0) + at, o);
  } else if constexpr (OP == GN_BWD) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const T d = v.g.v[i] - v.x.v[i] * k[1];
      o.v[i] = st.r * (KIND == GN_PLAIN ? d : d - k[0]);
    }
    if (a.o0 != nullptr) store_row_last<T, VEC>(static_cast<T*>(a.o0) + at, o);
  } else {
    const uint32_t kp = c.keep(row);
    RowVec<T, VEC> dg;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const GnSecond<T> e = gn_second<KIND, T, VEC, DROP>(c, st, kp, i, v.x.v[i], v.g.v[i]);
      const T ux = v.u.v[i], cc = c.w[i] * e.h;
      const T zd = st.r * (ux - k[0] - e.z * k[1]);
      const T td = gn_fma(c.w[i], zd, gn_fma(c.uw[i], e.z, c.ub[i]));
      const T q = KIND == GN_ACT ? gn_mul(e.q1, td) : T(0);
      const T C = gn_fma(c.w[i], q, gn_mul(c.uw[i], e.h)) - st.r * (k[1] * cc + k[2] * ux);
      dg.v[i] = e.d1 * td;
      o.v[i] = st.r * (C - k[3] - e.z * (k[4] + k[5]));
      cw[i] += q * e.z + e.h * zd;
      cb[i] += q;
    }
    if (a.o0 != nullptr) store_row_last<T, VEC>(static_cast<T*>(a.o0) + at, o);
    if (a.o1 != nullptr) store_row_last<T, VEC>(static_cast<T*>(a.o1) + at, dg);
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
    if (a.o0 != nullptr) store_row_last<T, VEC>(static_cast<T*>(a.o0) + r * a.lay.dim + col, zero);
    if (OP == GN_DBL && a.o1 != nullptr) store_row_last<T, VEC>(static_cast<T*>(a.o1) + r * a.lay.dim + col, zero);
  }
}

// Column sums of a CTA: thread slots colacc[2 VEC][threads] (weights, then biases) added over the row
// lanes of a column into `out` (weights; biases `apart` further on).  All threads call it.
template <int VEC, int NT = GN_THREADS>
__device__ __forceinline__ void gn_store_columns(const double* colacc, double* out, int64_t apart, int W, int TX,
                                                 int TY) {
  __syncthreads();
  for (int q = int(threadIdx.x); q < 2 * VEC * W; q += NT) {
    const int which = q / (VEC * W), cc = q % (VEC * W), tx = cc / VEC, i = cc % VEC;
    const double* p = colacc + (which * VEC + i) * NT + tx;
    double s = 0.0;
    for (int y = 0; y < TY; ++y) s += p[y * TX];
    out[which * apart + cc] = s;
  }
  __syncthreads();
}

// Gradients of the weights and biases of a tile's channels from the column sums of its `parts` CTAs (2 `apart`
// between CTAs), once all have left them; CTA `rank` of the `of` that call it takes its share.
// All columns of a channel are read here: either a tile holds whole channels (local kernels), or `apart` is the
// whole row and every tile's CTAs have left their sums (the grid kernel's tiles end anywhere, also in a channel).
template <typename T, int VEC, int NT = GN_THREADS>
__device__ __forceinline__ void gn_finish_columns(const NormArgs& a, const double* sums, int64_t apart, int parts,
                                                  int v0, int W, int rank, int of) {
  constexpr int WARPS = NT / 32;
  const int lane = int(threadIdx.x) % 32, n = W * VEC;
  for (int q = rank * WARPS + int(threadIdx.x) / 32; q < n; q += of * WARPS) {
    const int col = v0 * VEC + q;
    const RowBlock& b = a.lay.blk[block_of(a.lay, col)];
    const int u = int(fast_div(uint32_t(col - b.col0), b.div_d));
    if (u * b.d != col - b.col0) continue;
    const bool bias = b.bias0 >= 0 && a.gb != nullptr;
    double sw = 0.0, sb = 0.0;
    for (int p = lane; p < parts; p += 32) {
      const double* r = sums + 2 * int64_t(p) * apart + q;
      for (int m = 0; m < b.d; ++m) sw += __ldcg(r + m);
      if (bias) sb += __ldcg(r + apart);
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

// Is this CTA the last of `ctas` to come here?  What each stored before is then visible to it; nothing waits.
// The counter starts at 0.  All threads call it; `flag` is an int of shared memory that no one else uses.
__device__ __forceinline__ bool gn_comes_last(int32_t* counter, int ctas, int* flag) {
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    *flag = atomicAdd(counter, 1) == ctas - 1;
    __threadfence();
  }
  __syncthreads();
  return *flag != 0;
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
      const T n = T(rows * VEC), m = rows > 0 ? s1 * gn_recip(n) : T(0);
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

// Sum of v over groups of `lanes` (a power of two) consecutive threads.
template <typename T>
__device__ __forceinline__ T gn_lanes_sum(T v, int lanes) {
#pragma unroll
  for (int o = 16; o > 0; o /= 2)
    if (o < lanes) v += __shfl_xor_sync(~0u, v, o);
  return v;
}

// Join E entries: `lanes` consecutive threads share them, entry i's sums are at(i)[0], at(i)[stride], ..; every
// thread of the warp calls it.  All of the lanes get S.  This sits between two barriers, so what counts
// is the length of its chain of dependent instructions: a lane keeps its first CACHE entries in registers.
template <int OP, typename T, int CACHE = 1, typename F>
__device__ __forceinline__ void gn_join(int E, int lane, int lanes, int stride, bool scalar, T* S, F at) {
  constexpr int NS = gn_sums(OP);
  if constexpr (OP == GN_FWD) {
    T piv = T(0), mean = T(0), n = T(0), m2 = T(0);
    if (__any_sync(~0u, scalar)) {
      T d[CACHE], cnt[CACHE];
      if (scalar && E > 0) piv = *at(0);
#pragma unroll
      for (int c = 0; c < CACHE; ++c) {
        d[c] = cnt[c] = T(0);
        const int i = lane + c * lanes;
        if (scalar && i < E) {
          const T* p = at(i);
          cnt[c] = p[3 * stride];
          d[c] = (p[0] - piv) + p[stride];
          m2 += p[2 * stride];
        }
        n += cnt[c];
        mean += cnt[c] * d[c];
      }
      for (int i = lane + CACHE * lanes; scalar && i < E; i += lanes) {
        const T* p = at(i);
        const T w = p[3 * stride];
        n += w;
        mean += w * ((p[0] - piv) + p[stride]);
      }
      mean = gn_lanes_sum(mean, lanes);
      n = gn_lanes_sum(n, lanes);
      if (n > T(0)) mean *= gn_recip(n);
#pragma unroll
      for (int c = 0; c < CACHE; ++c) m2 += cnt[c] * (d[c] - mean) * (d[c] - mean);
      for (int i = lane + CACHE * lanes; scalar && i < E; i += lanes) {
        const T* p = at(i);
        const T e = ((p[0] - piv) + p[stride]) - mean;
        m2 += p[2 * stride] + p[3 * stride] * e * e;
      }
    }
    if (!scalar) {
#pragma unroll 4
      for (int i = lane; i < E; i += lanes) m2 += at(i)[2 * stride];
    }
    S[0] = piv;
    S[1] = mean;
    S[2] = gn_lanes_sum(m2, lanes);
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
#pragma unroll
    for (int p = 0; p < NS; ++p) S[p] = gn_lanes_sum(S[p], lanes);
  }
}

// ------------------------------------------------------------------------------------- local ---
// Thread (j, k, tx) owns vector column tx of the CTA's tile and row lane k of segments j, j + J, ..
// (M of them) of the current batch; R rows of each wait in its slots, which the next batch takes as
// soon as they are read the second time.  (A second set of slots, filled a batch ahead, was slower: a batch
// spends far longer between the barriers than on its way, so shared memory is better spent on more rows.)
// Rows of a thread beyond R, at most GN_FLUSH in all, take the slots in turns and are read again for the
// second pass, from L2.  With CL a cluster's CTAs have K row lanes each of one segment; each writes its
// sums into the shared memory of all.
template <typename T, int VEC, int OP, int R, int M, bool CL, int NT>
struct GnLocal {
  static constexpr int NS = gn_sums(OP), NC = gn_coefs(OP);
  static constexpr size_t slot_bytes = size_t(R) * M * GnSlots<T, VEC, OP, NT>::SLOT;
  static constexpr size_t col_bytes = OP == GN_FWD ? 0 : sizeof(double) * 2 * VEC * NT;
  static constexpr size_t buf_bytes = sizeof(T) * NS * M * NT;
  // sums of a cluster's CTAs, twice: [parity][sum][rank][local group]
  static constexpr int ALL_GROUPS = 32;
  static constexpr size_t all_bytes = CL ? sizeof(T) * 2 * NS * 16 * ALL_GROUPS : 0;
  static constexpr size_t fixed = slot_bytes + col_bytes + buf_bytes + all_bytes;
  // + per item of a batch its coefficients, per group of a tile its range, per segment of two batches its rows
  static size_t smem(const NormArgs& a) {
    return fixed + sizeof(T) * NC * M * a.j * a.tile_groups + sizeof(GnRange) * a.tile_groups + 8 * M * a.j;
  }
};

template <bool V>
struct GnFlag {
  static constexpr bool value = V;
};

// A thread's part of a batch: rows row0[m] + i step, i < n[m].
template <int M>
struct GnBatch {
  int row0[M], n[M];
};

template <int KIND, bool TURNS, typename T, int VEC, int OP, bool DROP, int R, int M, int NT>
__device__ __forceinline__ void gn_local_sums(const NormArgs& a, const GnCol<T, VEC, OP, DROP>& c,
                                              const GnStat<T> (&st)[M], const GnSlots<T, VEC, OP, NT>& sl,
                                              const GnBatch<M>& t, int step, T* buf, T* cw, T* cb) {
#pragma unroll
  for (int m = 0; m < M; ++m) {
    GnAcc<T, VEC, OP, DROP> acc;
    acc.clear(c);
    T piv = T(0);
    if (OP == GN_FWD && KIND != GN_PLAIN && t.n[m] > 0) piv = sl.get(m * R, 0).v[0];
    auto rows = [&](int row, int n) {
#pragma unroll 4
      for (int i = 0; i < n; ++i) {
        GnRow<T, VEC> v;
        sl.read(m * R + i, v);
        acc.template add<KIND>(c, st[m], piv, v, row + i * step);
        if (OP == GN_BWD) {  // z and c for the second pass
          sl.write(m * R + i, 0, v.x);
          sl.write(m * R + i, 1, v.g);
        }
      }
    };
    rows(t.row0[m], min(t.n[m], R));
    if (TURNS) {
#pragma unroll 1
      for (int from = R; from < t.n[m]; from += R) {
        const int row = t.row0[m] + from * step, n = min(t.n[m] - from, R);
        sl.reload(row, n, step, a.lay.dim, c.col);
        rows(row, n);
      }
    }
    gn_publish<KIND, OP, T, VEC>(c, acc, piv, t.n[m], buf + m * NT, M * NT);
    if constexpr (OP == GN_BWD) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        cw[i] += acc.s1[i];
        if (KIND != GN_PLAIN) cb[i] += acc.s2[i];
      }
    }
  }
}

template <int KIND, bool TURNS, typename T, int VEC, int OP, bool DROP, int R, int M, int NT>
__device__ __forceinline__ void gn_local_apply(const NormArgs& a, const GnCol<T, VEC, OP, DROP>& c,
                                               GnStat<T> (&st)[M], const GnSlots<T, VEC, OP, NT>& sl,
                                               const GnBatch<M>& t, int step, const T* res, int res_step, T* cw,
                                               T* cb) {
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
    auto rows = [&](int row, int n, auto again) {
#pragma unroll 4
      for (int i = 0; i < n; ++i) {
        const int r = row + i * step;
        GnRow<T, VEC> v;
        sl.read(m * R + i, v);
        if constexpr (OP == GN_BWD && again.value) {
          GnAcc<T, VEC, OP, DROP> z;
          z.clear(c);
          z.template add<KIND>(c, st[m], T(0), v, r);
        }
        gn_apply<KIND>(a, c, st[m], kf, v, int64_t(r) * a.lay.dim + c.col, r, cw, cb);
      }
    };
    if (!TURNS || t.n[m] <= R) {
      rows(t.row0[m], min(t.n[m], R), GnFlag<false>{});
    } else {  // more rows than slots: the first ones are gone
#pragma unroll 1
      for (int from = 0; from < t.n[m]; from += R) {
        const int row = t.row0[m] + from * step, n = min(t.n[m] - from, R);
        sl.reload(row, n, step, a.lay.dim, c.col);
        rows(row, n, GnFlag<true>{});
      }
    }
  }
}

// CTAs that have to fit an SM
__host__ __device__ constexpr int gn_local_ctas(int op, int threads) {
  return threads > GN_THREADS ? (op == GN_FWD ? 2 : 1) : op == GN_FWD ? 3 : 2;
}

template <typename T, int VEC, int OP, bool DROP, int R, int M, bool CL, int NT>
__global__ void __launch_bounds__(NT, gn_local_ctas(OP, NT))
gn_local_kernel(const __grid_constant__ NormArgs a) {
  using L = GnLocal<T, VEC, OP, R, M, CL, NT>;
  constexpr int NS = L::NS, NC = L::NC, STRIDE = M * NT;
  constexpr bool TURNS = !CL && R > 1;  // a thread may have more rows than slots
  extern __shared__ __align__(16) unsigned char smem[];
  unsigned char* sp = smem + L::slot_bytes;
  double* colbase = reinterpret_cast<double*>(sp);
  T* buf = reinterpret_cast<T*>(sp + L::col_bytes);
  T* all = buf + NS * STRIDE;
  T* res = reinterpret_cast<T*>(sp + L::col_bytes + L::buf_bytes + L::all_bytes);
  GnRange* gs = reinterpret_cast<GnRange*>(res + NC * M * a.j * a.tile_groups);
  int* lens = reinterpret_cast<int*>(gs + a.tile_groups);  // rows of a batch's segments: [parity][M J]
  // this CTA among its tile's (a cluster's CTAs are neighbours, and tiles start with a cluster)
  int tile = int(blockIdx.y), at = int(blockIdx.x), ctas = int(gridDim.x);
  if (!a.even) {
    for (tile = 0; int(blockIdx.x) >= a.start[tile + 1];) ++tile;
    at = int(blockIdx.x) - a.start[tile];
    ctas = a.start[tile + 1] - a.start[tile];
  }
  const int CS = CL ? a.cs : 1, rank = CL ? at % CS : 0, part = CL ? at / CS : at, parts = CL ? ctas / CS : ctas;
  const int tid = int(threadIdx.x), tx = tid % a.tx, ty = tid / a.tx;
  const int K = a.k, step = K * CS, J = a.j;
  const int v0 = a.tile[tile], W = a.tile[tile + 1] - v0;
  const int j = ty / K, k = rank * K + ty - j * K;
  const bool active = tx < W && j < J;
  const int64_t G = a.lay.n_groups();

  GnSlots<T, VEC, OP, NT> sl;
  sl.init(a, smem);
  const int col = (v0 + (active ? tx : 0)) * VEC;
  const uint32_t div_step = step > 1 ? 0xFFFFFFFFu / uint32_t(step) + 1u : 0u;
  const int64_t hop_b = int64_t(parts) * (J * M);
  int lo[M], hi[M];  // row pointers of the batch after the one on its way
  auto point = [&](int64_t b0) {
#pragma unroll
    for (int m = 0; m < M; ++m) {
      lo[m] = hi[m] = 0;
      const int64_t b = b0 + m * J + j;
      if (active && b < a.B) {
        lo[m] = a.row_ptr != nullptr ? a.row_ptr[b] : 0;
        hi[m] = a.row_ptr != nullptr ? a.row_ptr[b + 1] : int(a.N);
        if (b == 0 && lo[m] != 0) hi[m] = -1;  // reported below
      }
    }
  };
  // rows of the batch that lo and hi point to, on their way into the slots
  auto fetch = [&](int half, GnBatch<M>& t) {
#pragma unroll
    for (int m = 0; m < M; ++m) {
      int s = lo[m], e = hi[m];
      if (s < 0 || e < s || e > int(a.N) || e - s > a.cap * step) {  // no row pointer, or longer than the caller said
        atomicCAS(a.status, 0, int(E3_ERR_INDEX));
        s = min(max(s, 0), int(a.N));
        e = s + min(min(max(e, s), int(a.N)) - s, a.cap * step);
      }
      t.row0[m] = s + k;
      const int left = e - s - k + step - 1;
      t.n[m] = !active ? 0 : R == 1 ? int(e > s + k) : left > 0 ? int(fast_div(uint32_t(left), div_step)) : 0;
      if (active && tx == 0 && ty == j * K) lens[(half * M + m) * J + j] = e - s;
    }
    const int64_t hop = int64_t(step) * a.lay.dim * int64_t(sizeof(T));
#pragma unroll
    for (int m = 0; m < M; ++m) {
      int64_t at = (int64_t(t.row0[m]) * a.lay.dim + col) * int64_t(sizeof(T));
#pragma unroll 4
      for (int i = 0; i < min(t.n[m], R); ++i, at += hop) sl.fetch(m * R + i, at);
    }
    sl.commit();
  };
  int64_t b0 = int64_t(part) * (J * M);
  GnBatch<M> t;
  point(b0);
  fetch(0, t);
  point(b0 + hop_b);

  GnCol<T, VEC, OP, DROP> c;
  c.init(a, v0, W, active ? tx : 0);
  const int gfirst = c.g - c.lg, nlg = group_of(a.lay, (v0 + W) * VEC - 1) - gfirst + 1;
  if (active && ty == 0 && tx == c.g0) gs[c.lg] = gn_range(c.g0, c.g1);
  const bool columns = OP != GN_FWD && a.colpart != nullptr;
  T cw[VEC], cb[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) cw[i] = cb[i] = T(0);
  if (columns) {
#pragma unroll
    for (int i = 0; i < 2 * VEC; ++i) colbase[i * NT + tid] = 0.0;
  }
  const uint32_t div_nlg = nlg > 1 ? 0xFFFFFFFFu / uint32_t(nlg) + 1u : 0u;
  const uint32_t div_j = J > 1 ? 0xFFFFFFFFu / uint32_t(J) + 1u : 0u;
  const int lane = tid & (a.lanes - 1), sub = tid / a.lanes, per = NT / a.lanes;
  const int items = M * J * nlg;
  const int held = M * (TURNS ? a.cap : R);  // rows of a thread in a batch at most
  int rows_held = 0, parity = 0;
  if (CL) cooperative_groups::this_cluster().sync();  // every CTA of the cluster has started
  for (; b0 < a.B; b0 += hop_b, parity ^= 1) {
    GnStat<T> st[M];
    if (OP != GN_FWD) {
#pragma unroll
      for (int m = 0; m < M; ++m) {
        const int64_t b = b0 + m * J + j;
        if (t.n[m] > 0) st[m].set(a.stats + 2 * (b * G + c.g));
      }
    }
    sl.template wait<0>();
    if (c.kind == GN_PLAIN) gn_local_sums<GN_PLAIN, TURNS, T, VEC, OP, DROP, R, M, NT>(a, c, st, sl, t, step, buf + tid, cw, cb);
    else if (c.kind == GN_CENTRED)
      gn_local_sums<GN_CENTRED, TURNS, T, VEC, OP, DROP, R, M, NT>(a, c, st, sl, t, step, buf + tid, cw, cb);
    else gn_local_sums<GN_ACT, TURNS, T, VEC, OP, DROP, R, M, NT>(a, c, st, sl, t, step, buf + tid, cw, cb);
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
      const T* q = buf + m * NT + jj * K * a.tx + gr.first;
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
        const T r = OP == GN_DBL ? T(a.stats[2 * (b * G + g) + 1]) : T(0);
        gn_finish<OP, T>(S, T(lens[parity * M * J + mj]) * T(blk.group_cols), scalar, r, T(a.eps), res + NC * it);
      }
    }
    if (CL) {
      cooperative_groups::this_cluster().sync();
      for (int base = 0; base < nlg; base += NT / 16) {
        const int lg = base + tid / 16, g = gfirst + (lg < nlg ? lg : 0);
        const RowBlock& blk = a.lay.blk[fast_div(uint32_t(g), a.lay.div_groups)];
        const bool scalar = blk.bias0 >= 0;
        const T* q = all + parity * NS * 16 * L::ALL_GROUPS + lg;
        T S[NS];
        gn_join<OP, T>(lg < nlg ? CS : 0, tid % 16, 16, 16 * L::ALL_GROUPS, scalar, S,
                       [&](int i) { return q + i * L::ALL_GROUPS; });
        if (lg < nlg && tid % 16 == 0) {
          const T r = OP == GN_DBL ? T(a.stats[2 * (b0 * G + g) + 1]) : T(0);
          gn_finish<OP, T>(S, T(lens[parity]) * T(blk.group_cols), scalar, r, T(a.eps), res + NC * lg);
        }
      }
    }
    __syncthreads();
    if (OP == GN_FWD && rank == 0) {
      for (int it = tid; it < items; it += NT) {
        const int mj = int(fast_div(uint32_t(it), div_nlg)), lg = it - mj * nlg;
        if (b0 + mj < a.B) gn_store_stats(res + NC * it, a.stats + 2 * ((b0 + mj) * G + gfirst + lg));
      }
    }
    const T* q = res + NC * ((active ? j : 0) * nlg + c.lg);
    const int hop_res = NC * J * nlg;
    if (c.kind == GN_PLAIN)
      gn_local_apply<GN_PLAIN, TURNS, T, VEC, OP, DROP, R, M, NT>(a, c, st, sl, t, step, q, hop_res, cw, cb);
    else if (c.kind == GN_CENTRED)
      gn_local_apply<GN_CENTRED, TURNS, T, VEC, OP, DROP, R, M, NT>(a, c, st, sl, t, step, q, hop_res, cw, cb);
    else gn_local_apply<GN_ACT, TURNS, T, VEC, OP, DROP, R, M, NT>(a, c, st, sl, t, step, q, hop_res, cw, cb);
    rows_held += held;
    if (columns && rows_held > GN_FLUSH - held) {  // another batch could pass GN_FLUSH rows
      rows_held = 0;
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        colbase[i * NT + tid] += double(cw[i]);
        colbase[(VEC + i) * NT + tid] += double(cb[i]);
        cw[i] = cb[i] = T(0);
      }
    }
    fetch(parity ^ 1, t);
    point(b0 + 2 * hop_b);
  }
  if (active)
    gn_zero_rows<T, VEC, OP>(a, c.col, gn_rows_end(a) + int64_t(at) * (J * K) + ty, a.N, int64_t(ctas) * (J * K));
  if (columns) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      colbase[i * NT + tid] += double(cw[i]);
      colbase[(VEC + i) * NT + tid] += double(cb[i]);
    }
    const int apart = a.tx * VEC;
    double* sums = a.colpart + 2 * int64_t(a.start[tile]) * apart;
    gn_store_columns<VEC, NT>(colbase, sums + 2 * int64_t(at) * apart, apart, W, a.tx, J * K);
    if (CL && a.meet) {
      // Clusters never meet across the grid: no launch has both a cluster dimension and a grid barrier.  The CTA
      // of the tile that comes last adds up the sums of all, in the order of their numbers whichever it is.
      if (gn_comes_last(a.tickets + tile, ctas, lens)) gn_finish_columns<T, VEC, NT>(a, sums, apart, ctas, v0, W, 0, 1);
      return;
    }
    if (CL) cooperative_groups::this_cluster().sync();  // one cluster has all of the tile's segments
    else cooperative_groups::this_grid().sync();
    gn_finish_columns<T, VEC, NT>(a, sums, apart, ctas, v0, W, at, ctas);
  }
}

// -------------------------------------------------------------------------------------- grid ---
// CTA (rc, ct): row chunk rc, column tile ct; all CTAs are resident.  A segment that lies in one chunk is
// finished there (unless its group is cut into tiles); the others leave partial sums:
//   slot of (chunk, segment), part of (tile, group):  part[slot][groups + tiles][sums]
// slots: 2 chunk (the segment began earlier) or 2 chunk + 1 (it begins here and goes on); with cut
// groups chunk + segment, which rises by one from piece to piece.  Parts likewise are group + tile.
// The grid meets, the CTAs that hold a segment share the joining of its groups, the grid meets again, and
// every CTA reads its rows a second time, from the last one back: those are still in L2.
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
  static constexpr int U = OP == GN_FWD ? 4 : OP == GN_BWD ? 2 : 1;  // rows that a thread takes at a time
  static constexpr int STAGES = 4;                                   // such groups in flight
  static constexpr size_t slot_bytes = size_t(STAGES) * U * GnSlots<T, VEC, OP>::SLOT;
  static constexpr size_t long_bytes = OP == GN_DBL ? sizeof(double) * NS * GN_THREADS : 0;
  static constexpr size_t buf_bytes = sizeof(T) * NS * GN_THREADS;
  static constexpr size_t col_bytes = OP == GN_FWD ? 0 : sizeof(double) * 2 * VEC * GN_THREADS;
  static constexpr size_t smem = slot_bytes + long_bytes + col_bytes + buf_bytes + sizeof(GnRange) * GN_THREADS;
};

// A thread's rows of a piece, in order or backwards, through a ring of slots.
template <typename T, int VEC, int OP>
struct GnStream {
  static constexpr int U = GnGrid<T, VEC, OP>::U, STAGES = GnGrid<T, VEC, OP>::STAGES;
  GnSlots<T, VEC, OP> sl;
  int64_t at, step;  // bytes: the next row to fetch, the way from a row to the next
  int left;          // rows still to fetch
  int put, take;     // ring positions

  __device__ __forceinline__ void issue() {
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (i < left) {
        sl.fetch(put * U + i, at);
        at += step;
      }
    left -= U;
    put = (put + 1) % STAGES;
    sl.commit();
  }
  // n rows from row r0 on, every K-th; `back`: from the last one down
  __device__ __forceinline__ void start(const NormArgs& a, int col, int r0, int n, int K, bool back) {
    const int64_t row = int64_t(a.lay.dim) * sizeof(T);
    step = back ? -K * row : K * row;
    at = (back ? int64_t(r0) + int64_t(n - 1) * K : int64_t(r0)) * row + col * int64_t(sizeof(T));
    left = n;
    put = take = 0;
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) issue();
  }
  // f(i, row's vectors) for the rows of the next group that are there
  template <typename F>
  __device__ __forceinline__ void next(int n, F f) {
    sl.template wait<STAGES - 2>();
    GnRow<T, VEC> v[U];
#pragma unroll
    for (int i = 0; i < U; ++i) sl.read(take * U + i, v[i]);
    issue();  // into the slots read in the step before
    take = (take + 1) % STAGES;
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (i < n) f(i, v[i]);
  }
};

// The pieces (segment x chunk) of a chunk of rows, in order.
struct GnPiece {
  int b, s, e, ps, pe;  // segment, its rows, the rows in the chunk
  __device__ __forceinline__ bool next(const NormArgs& a, int lo, int hi) {
    for (++b; b < a.B; ++b) {
      gn_segment(a, b, s, e);
      if (s >= hi) return false;
      ps = max(s, lo);
      pe = min(e, hi);
      if (ps < pe) return true;
    }
    return false;
  }
  __device__ __forceinline__ bool whole(const NormArgs& a) const { return ps == s && pe == e && !a.wide; }
};

// A thread's sums over the rows of a stream into its slots of buf (and of the columns).
template <int KIND, typename T, int VEC, int OP, bool DROP>
__device__ __forceinline__ void gn_grid_sums(const NormArgs& a, const GnCol<T, VEC, OP, DROP>& c, const GnStat<T>& st,
                                             GnStream<T, VEC, OP>& q, int r0, int n, int K, T* buf, double* sums,
                                             double* colacc) {
  constexpr int U = GnGrid<T, VEC, OP>::U;
  T piv = T(0);
  GnAcc<T, VEC, OP, DROP> acc;
  acc.clear(c);
  double l1 = 0.0, l2 = 0.0;  // the sums of earlier flushes
  if (OP == GN_DBL) {
#pragma unroll
    for (int i = 0; i < 12; ++i) sums[i * GN_THREADS] = 0.0;
  }
#pragma unroll 1
  for (int f = 0; f < n; f += GN_FLUSH) {
    const int fe = min(n, f + GN_FLUSH);
#pragma unroll 1
    for (int r = f; r < fe; r += U)
      q.next(fe - r, [&](int i, GnRow<T, VEC>& v) {
        if (OP == GN_FWD && KIND != GN_PLAIN && r + i == 0) piv = v.x.v[0];
        acc.template add<KIND>(c, st, piv, v, r0 + (r + i) * K);
      });
    if constexpr (OP == GN_FWD) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        l1 += double(acc.s1[i]);
        l2 += double(acc.s2[i]);
      }
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
    } else {
#pragma unroll
      for (int i = 0; i < 12; ++i) sums[i * GN_THREADS] += double(acc.s[i]);
    }
    acc.clear(c);
  }
  if constexpr (OP == GN_FWD) {
    const double cnt = double(n) * VEC, m = KIND != GN_PLAIN && n > 0 ? l1 / cnt : 0.0;
    buf[0] = piv;
    buf[GN_THREADS] = T(m);
    buf[2 * GN_THREADS] = T(l2 - m * l1);
    buf[3 * GN_THREADS] = T(cnt);
  } else if constexpr (OP == GN_BWD) {
    buf[0] = T(l1);
    buf[GN_THREADS] = T(l2);
  } else {
#pragma unroll
    for (int i = 0; i < 12; ++i) buf[i * GN_THREADS] = T(sums[i * GN_THREADS]);
  }
}

// Pointwise results of the rows of a stream that runs backwards from row r0 + (n - 1) K.
template <int KIND, typename T, int VEC, int OP, bool DROP>
__device__ __forceinline__ void gn_grid_apply(const NormArgs& a, const GnCol<T, VEC, OP, DROP>& c, const GnStat<T>& st,
                                              const T* kf, GnStream<T, VEC, OP>& q, int r0, int n, int K,
                                              double* colacc) {
  constexpr int U = GnGrid<T, VEC, OP>::U;
  const int64_t D = a.lay.dim;
  int row = r0 + (n - 1) * K;
#pragma unroll 1
  for (int f = 0; f < n; f += GN_FLUSH) {
    const int fe = min(n, f + GN_FLUSH);
    T cw[VEC], cb[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) cw[i] = cb[i] = T(0);
#pragma unroll 1
    for (int r = f; r < fe; r += U) {
      q.next(fe - r, [&](int i, GnRow<T, VEC>& v) {
        if constexpr (OP == GN_BWD) {  // z and c again
          GnAcc<T, VEC, OP, DROP> z;
          z.clear(c);
          z.template add<KIND>(c, st, T(0), v, row - i * K);
        }
        gn_apply<KIND>(a, c, st, kf, v, (row - i * K) * D + c.col, row - i * K, cw, cb);
      });
      row -= U * K;
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

template <typename T, int VEC, int OP, bool DROP>
__global__ void __launch_bounds__(GN_THREADS, OP == GN_FWD ? 3 : 2) gn_grid_kernel(const __grid_constant__ NormArgs a) {
  using L = GnGrid<T, VEC, OP>;
  constexpr int NS = L::NS, NC = L::NC;
  extern __shared__ __align__(16) unsigned char smem[];
  double* sums = reinterpret_cast<double*>(smem + L::slot_bytes);     // a thread's long sums (double backward)
  double* columns = reinterpret_cast<double*>(smem + L::slot_bytes + L::long_bytes);
  T* buf = reinterpret_cast<T*>(smem + L::slot_bytes + L::long_bytes + L::col_bytes);
  GnRange* gs = reinterpret_cast<GnRange*>(smem + L::slot_bytes + L::long_bytes + L::col_bytes + L::buf_bytes);
  const int rc = int(blockIdx.x) / a.n_tiles, tile = int(blockIdx.x) % a.n_tiles;
  int lo = int(min(a.N, rc * a.rows_cta)), hi = int(min(a.N, (rc + 1) * a.rows_cta));
  const int tid = int(threadIdx.x), tx = tid % a.tx, ty = tid / a.tx, K = a.k;
  const int v0 = a.tile[tile], W = a.tile[tile + 1] - v0;
  const bool active = tx < W && ty < K;
  const int64_t G = a.lay.n_groups();

  GnStream<T, VEC, OP> q;
  q.sl.init(a, smem);
  int first = gn_first_segment(a, lo) - 1;
  GnPiece p;
  int n = 0;  // this thread's rows of the piece
  auto open = [&](bool back) {
    const bool there = p.next(a, lo, hi);
    n = there && active && p.ps + ty < p.pe ? (p.pe - p.ps - ty + K - 1) / K : 0;
    if (OP == GN_BWD && back && a.o0 == nullptr) n = 0;
    q.start(a, (v0 + tx) * VEC, p.ps + ty, n, K, back);
    return there;
  };
  p.b = first;
  bool there = open(false);
  GnCol<T, VEC, OP, DROP> c;
  c.init(a, v0, W, active ? tx : 0);
  const int gfirst = c.g - c.lg, nlg = group_of(a.lay, (v0 + W) * VEC - 1) - gfirst + 1;
  if (active && ty == 0 && tx == c.g0) gs[c.lg] = gn_range(c.g0, c.g1);
  const bool col_sums = OP != GN_FWD && a.colpart != nullptr;
  double* colacc = col_sums ? columns + tid : nullptr;
  if (col_sums) {
#pragma unroll
    for (int i = 0; i < 2 * VEC; ++i) colacc[i * GN_THREADS] = 0.0;
  }
  // where the second pass finds the result of (segment b, group g)
  auto keep = [&](const T* o, int b, int g) {
    if (OP == GN_FWD) {
      gn_store_stats(o, a.stats + 2 * (b * G + g));
    } else {
      T* dst = static_cast<T*>(a.coef) + NC * (b * G + g);
#pragma unroll
      for (int i = 0; i < NC; ++i) dst[i] = o[i];
    }
  };

  // first pass
  const int lane = tid & (a.lanes - 1), sub = tid / a.lanes, per = GN_THREADS / a.lanes;
#pragma unroll 1
  for (; there; there = open(false)) {
    GnStat<T> st;
    if (OP != GN_FWD) st.set(a.stats + 2 * (p.b * G + c.g));
    double* acc = OP == GN_BWD ? colacc : nullptr;
    if (c.kind == GN_PLAIN) gn_grid_sums<GN_PLAIN>(a, c, st, q, p.ps + ty, n, K, buf + tid, sums + tid, acc);
    else if (c.kind == GN_CENTRED)
      gn_grid_sums<GN_CENTRED>(a, c, st, q, p.ps + ty, n, K, buf + tid, sums + tid, acc);
    else gn_grid_sums<GN_ACT>(a, c, st, q, p.ps + ty, n, K, buf + tid, sums + tid, acc);
    __syncthreads();
    for (int base = 0; base < nlg; base += per) {
      const int lg = base + sub, g = gfirst + (lg < nlg ? lg : 0);
      const RowBlock& blk = a.lay.blk[fast_div(uint32_t(g), a.lay.div_groups)];
      const bool scalar = blk.bias0 >= 0;
      GnRange gr{0, 1, 0};
      if (lg < nlg) gr = gs[lg];
      T S[NS];
      gn_join<OP, T>(lg < nlg ? K * gr.w : 0, lane, a.lanes, GN_THREADS, scalar, S, [&](int i) {
        const int kk = int(fast_div(uint32_t(i), gr.div_w));
        return buf + kk * a.tx + gr.first + i - kk * gr.w;
      });
      if (lg < nlg && lane == 0) {
        if (p.whole(a)) {
          T o[NC];
          const T r = OP == GN_DBL ? T(a.stats[2 * (p.b * G + g) + 1]) : T(0);
          gn_finish<OP, T>(S, T(p.e - p.s) * T(blk.group_cols), scalar, r, T(a.eps), o);
          keep(o, p.b, g);
        } else {
          T* dst = gn_slot<OP, T>(a, rc, p.b, p.s >= lo, tile, g);
#pragma unroll
          for (int i = 0; i < NS; ++i) dst[i] = S[i];
        }
      }
    }
    __syncthreads();
  }
  double* csum = col_sums ? a.colpart + v0 * VEC : nullptr;  // [chunk][weights, biases][dim]
  if (OP == GN_BWD && col_sums) gn_store_columns<VEC>(columns, csum + 2 * rc * int64_t(a.lay.dim), a.lay.dim, W, a.tx, K);
  if (rc == 0 && tid == 0) a.tickets[tile] = a.chunks;  // the first parts are handed out already
  auto grid = cooperative_groups::this_grid();
  grid.sync();

  // join the segments that are spread over chunks (or tiles): chunk rc of nc takes groups rc - c0, + nc, ..
#pragma unroll 1
  for (p.b = first; p.next(a, lo, hi);) {
    if (p.whole(a)) continue;
    const int c0 = int(p.s / a.rows_cta), nc = int((p.e - 1) / a.rows_cta) - c0 + 1;
#pragma unroll 1
    for (int lg = rc - c0; lg < nlg; lg += nc) {
      const int g = gfirst + lg;
      int nt = 1;
      if (a.wide) {  // the tiles that hold parts of this group: the first one's CTA joins it
        if (tile > 0 && group_of(a.lay, v0 * VEC - 1) == g) continue;
        while (tile + nt < a.n_tiles && group_of(a.lay, a.tile[tile + nt] * VEC) == g) ++nt;
      }
      const RowBlock& blk = a.lay.blk[fast_div(uint32_t(g), a.lay.div_groups)];
      const bool scalar = blk.bias0 >= 0;
      // every warp its share of the entries, then one warp the warps' sums
      constexpr int WARPS = GN_THREADS / 32;
      const int w = tid / 32, E = nc * nt, mine = E > w ? (E - w + WARPS - 1) / WARPS : 0;
      const T* part = gn_slot<OP, T>(a, c0, p.b, false, tile, g);
      const int64_t hop = (a.wide ? 1 : 2) * (G + a.n_tiles) * NS;  // from chunk to chunk
      const int64_t begin = a.wide ? 0 : (G + a.n_tiles) * NS;      // the first chunk's slot is the next one
      T S[NS];
      gn_join<OP, T, 2>(mine, tid % 32, 32, 1, scalar, S, [&](int i) {
        const int e = w + i * WARPS, ch = nt == 1 ? e : e / nt;
        return part + ch * hop + (ch == 0 ? begin : 0) + (nt == 1 ? 0 : (e - ch * nt) * NS);
      });
      if (tid % 32 == 0) {
#pragma unroll
        for (int i = 0; i < NS; ++i) buf[w * NS + i] = S[i];
      }
      __syncthreads();
      if (w == 0) {
        gn_join<OP, T>(min(WARPS, E), tid, 32, 1, scalar, S, [&](int i) { return buf + i * NS; });
        if (tid == 0) {
          T o[NC];
          const T r = OP == GN_DBL ? T(a.stats[2 * (p.b * G + g) + 1]) : T(0);
          gn_finish<OP, T>(S, T(p.e - p.s) * T(blk.group_cols), scalar, r, T(a.eps), o);
          keep(o, p.b, g);
        }
      }
      __syncthreads();
    }
  }
  // second pass: the chunks are cut into parts, the last ones first.  Without sums to keep (all forms but
  // the double backward) a CTA that is done draws another part of its tile: the CTAs' shares of the memory
  // bandwidth differ by a third, and the slowest would hold up the rest.
  int part = rc;
  auto bounds = [&]() {  // rows of part `part` of the tile
    if (a.parts == 1) return;
    const int ch = part % a.chunks, at = a.parts - 1 - part / a.chunks;
    const int64_t c_lo = ch * a.rows_cta, c_hi = min(a.N, c_lo + a.rows_cta);
    const int64_t size = (a.rows_cta + a.parts - 1) / a.parts;
    lo = int(min(c_hi, c_lo + at * size));
    hi = int(min(c_hi, c_lo + (at + 1) * size));
    first = gn_first_segment(a, lo) - 1;
  };
  bounds();
  p.b = first;
  there = lo < hi && open(true);  // the first rows are on their way while the grid meets
  if (OP == GN_BWD && col_sums) gn_finish_columns<T, VEC>(a, csum, a.lay.dim, a.chunks, v0, W, rc, a.chunks);
  grid.sync();

  while (true) {
    if (a.parts > 1 && tid == 0) gs[0].first = atomicAdd(a.tickets + tile, 1);
#pragma unroll 1
    for (; there; there = open(true)) {
      GnStat<T> st;
      st.set(a.stats + 2 * (p.b * G + c.g));
      T kf[NC];
      if (OP != GN_FWD) {
        const T* k = static_cast<const T*>(a.coef) + NC * (p.b * G + c.g);
#pragma unroll
        for (int i = 0; i < NC; ++i) kf[i] = k[i];
      }
      double* acc = OP == GN_DBL ? colacc : nullptr;
      if (c.kind == GN_PLAIN) gn_grid_apply<GN_PLAIN>(a, c, st, kf, q, p.ps + ty, n, K, acc);
      else if (c.kind == GN_CENTRED) gn_grid_apply<GN_CENTRED>(a, c, st, kf, q, p.ps + ty, n, K, acc);
      else gn_grid_apply<GN_ACT>(a, c, st, kf, q, p.ps + ty, n, K, acc);
    }
    if (active) gn_zero_rows<T, VEC, OP>(a, c.col, max(lo, gn_rows_end(a)) + ty, hi, K);
    if (a.parts == 1) break;
    __syncthreads();
    part = gs[0].first;
    __syncthreads();
    if (part >= a.chunks * a.parts) break;
    bounds();
    p.b = first;
    there = lo < hi && open(true);
  }
  if (OP == GN_DBL && col_sums) {
    gn_store_columns<VEC>(columns, csum + 2 * rc * int64_t(a.lay.dim), a.lay.dim, W, a.tx, K);
    grid.sync();
    gn_finish_columns<T, VEC>(a, csum, a.lay.dim, a.chunks, v0, W, rc, a.chunks);
  }
}

}  // namespace e3b
