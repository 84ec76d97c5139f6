// Group norm of feature rows: configuration, the parameters' gradients and the C ABI.
#include <cmath>

#include "group_norm_launch.h"

namespace e3b {
namespace {

// Row numbers plus a CTA's row lanes stay below 2^31.
constexpr int64_t GN_MAX_ROWS = (int64_t(1) << 31) - 65536;

size_t al256(size_t b) { return (b + 255) & ~size_t(255); }

void count_groups(const RowLayout& L, int vec, TileSet* t) {
  for (int i = 0; i + 1 < int(t->first.size()); ++i) {
    const int a = t->first[i] * vec, b = t->first[i + 1] * vec - 1;
    t->tx = std::max(t->tx, t->first[i + 1] - t->first[i]);
    t->groups = std::max(t->groups, group_of(L, b) - group_of(L, a) + 1);
    if (i > 0 && group_of(L, a - 1) == group_of(L, a)) t->cut = true;
  }
}

void count_scalars(const RowLayout& L, int vec, TileSet* t) {
  for (int i = 0; i < t->n(); ++i) {
    int32_t scalars = 0;
    for (int v = t->first[i]; v < t->first[i + 1]; ++v) scalars += L.blk[block_of(L, v * vec)].bias0 >= 0;
    t->scalars.push_back(scalars);
  }
}

// Tiles of whole groups, as many as fit `cap` vectors (cap >= the widest group), `most` at most.
TileSet cut_tiles(const RowLayout& L, int vec, int cap, int most = 1 << 30) {
  TileSet t;
  t.first.push_back(0);
  int at = 0, held = 0;
  for (int b = 0; b < L.n_blocks; ++b) {
    const int w = L.blk[b].group_cols / vec;
    for (int g = 0; g < L.groups; ++g) {
      if (held > 0 && (at + w - t.first.back() > cap || held == most)) {
        t.first.push_back(at);
        held = 0;
      }
      at += w;
      ++held;
    }
  }
  t.first.push_back(at);
  count_groups(L, vec, &t);
  return t;
}

// Equal tiles wherever they end: the widest of those that leave the fewest of a block's threads idle.
TileSet equal_tiles(const RowLayout& L, int vec) {
  const int V = L.dim / vec;
  int best = 0;
  double score = 0.0;
  for (int n = (V + GN_THREADS - 1) / GN_THREADS; n <= std::min(V, 256); ++n) {
    const int tx = (V + n - 1) / n, lanes = GN_THREADS / tx;
    const double u = double(V) / (double((V + tx - 1) / tx) * tx) * (double(tx) * lanes / GN_THREADS);
    if (u > score * 1.03) {
      score = u;
      best = tx;
    }
    if (tx <= 32) break;
  }
  TileSet t;
  for (int v = 0; v < V; v += best) t.first.push_back(v);
  t.first.push_back(V);
  count_groups(L, vec, &t);
  return t;
}

// The cut between `lo` and `hi` that leaves the fewest of a block's threads idle; of cuts within 3% of it the
// widest, whose rows are the longest runs of memory.
TileSet best_tiles(const RowLayout& L, int vec, int lo, int hi, int k, int threads, int most = 1 << 30) {
  TileSet best;
  double score = -1.0;
  const int V = L.dim / vec;
  for (int cap = lo; cap <= hi; ++cap) {
    TileSet t = cut_tiles(L, vec, cap, most);
    if (t.n() > GN_MAXTILE) continue;
    const int lanes = k > 0 ? k * std::max(1, threads / (t.tx * k)) : threads / t.tx;
    const double u = double(V) / (double(t.n()) * t.tx) * (double(t.tx) * lanes / threads);
    if (u >= score * 0.97) {
      score = std::max(score, u);
      best = std::move(t);
    }
    if (cap >= V) break;
  }
  return best;
}

// Work of a call: which kernel, and the thread layout.
GnConfig configure(const e3_features* f, int64_t N, int64_t B, int64_t max_rows, int op, NormArgs* a) {
  GnConfig c;
  a->N = N;
  a->B = int32_t(B);
  a->lay = f->lay;
  const int64_t most = max_rows > 0 ? std::min(max_rows, N) : N;
  const int RP = gn_reg_rows(op);
  // local: the rows of the longest segment fit one CTA's slots, or a cluster of up to 16 CTAs'; or they take
  // the slots in turns, where there are segments enough to fill the device
  int shift = 0;
  while ((int64_t(RP) << shift) < most && shift < 8 && f->local[shift + 1].n() > 0) ++shift;
  const TileSet* t = &f->local[shift];
  a->cs = 1;
  a->cap = RP;
  const bool held = (int64_t(RP) << shift) >= most;
  const bool turns = (int64_t(GN_FLUSH) << shift) >= most && B * t->n() >= sm_count();
  if (most <= 1 && f->rows.n() > 0 && f->rows.n() <= GN_LOCAL_TILES) {
    c.local = c.one_row = true;
    t = &f->rows;
    a->cap = a->k = 1;
    a->j = std::min(GN_ROW_THREADS / t->tx, std::max(1, GN_ROW_ITEMS / (gn_reg_segments(op, f->vec) * t->groups)));
  } else if (t->n() > 0 && t->n() <= GN_LOCAL_TILES && (held || turns)) {
    c.local = true;
    a->cap = held ? RP : GN_FLUSH;
    a->k = 1 << shift;
    a->j = std::min(std::max(1, GN_THREADS / (t->tx << shift)), std::max(1, 2048 / t->groups));
  }
  // clusters: when one CTA is too small, or when there are so few CTAs that dividing the rows further lets
  // more SMs load them
  if (f->cluster_ok && !c.one_row) {
    const TileSet* n = &f->narrow;
    const int k = GN_THREADS / n->tx;
    int cs = 1;
    while (cs < 16 && int64_t(RP) * k * cs < most) cs *= 2;
    // all clusters at once; in the backwards one CTA per SM, unless there is one cluster per tile
    const int64_t all = B * n->n();
    const int64_t room = op == GN_FWD || B == 1 ? 2 * sm_count() : 128;
    const bool fits = int64_t(RP) * k * cs >= most && all * cs <= room;
    if (fits && (!c.local || (held && a->j == 1 && int64_t(t->n()) * B < sm_count()))) {
      while (cs < 8 && all * cs * 2 <= room && most > 2 * k * cs) cs *= 2;
      c.local = true;
      t = n;
      a->cap = RP;
      a->k = k;
      a->j = 1;
      a->cs = cs;
    }
  }
  if (!c.local) {
    t = &f->grid;
    a->cs = 1;
    a->k = GN_THREADS / t->tx;
    a->j = 1;
  }
  std::copy(t->first.begin(), t->first.end(), a->tile);
  a->n_tiles = t->n();
  c.tiles = t;
  a->tx = t->tx;
  a->wide = t->cut;
  a->tile_groups = t->groups;
  // lanes of a join: enough for all entries, but no more than lets every item of a batch have its own at
  // once, unless that leaves a lane more than 16 entries (one-row segments of 64 columns in 16 groups: 8 lanes
  // and 32 rounds 336 us, 1 lane and 4 rounds 171 us)
  const int threads = c.one_row ? GN_ROW_THREADS : GN_THREADS;
  const int entries = a->k * std::min(f->wide, t->tx);
  const int items = (c.one_row ? gn_reg_segments(op, f->vec) : 1) * a->j * t->groups;
  a->lanes = 1;
  while (a->lanes < 32 && a->lanes < entries && (a->lanes * 2 * items <= threads || a->lanes * 16 < entries))
    a->lanes *= 2;
  return c;
}

e3_status check_workspace(const void* ws, size_t bytes, size_t need) {
  if (need == 0) return E3_OK;
  if (ws == nullptr || (reinterpret_cast<uintptr_t>(ws) & 15u))
    return fail(E3_ERR_INVALID_ARG, "workspace is NULL or not 16-byte aligned");
  if (bytes < need) return fail(E3_ERR_SHAPE, "workspace of %zu bytes, %zu needed", bytes, need);
  return E3_OK;
}

size_t workspace_bytes_of(const GnConfig& c, NormArgs a, int op, int vec) {
  const int64_t ctas = int64_t(GN_MAX_RESIDENT) * sm_count();
  if (c.local) return gn_local_layout(a, op, vec, std::max(ctas, int64_t(a.n_tiles) * a.cs));
  return gn_grid_layout(&a, op, ctas);
}

e3_status check_sizes(const e3_features* f, int64_t N, int64_t B, bool one_ok) {
  const e3_status st = check_features_device(f);
  if (st != E3_OK) return st;
  if (N < 0 || N > GN_MAX_ROWS) return fail(E3_ERR_SHAPE, "N = %lld", (long long)N);
  if (B < 1 || B >= (int64_t(1) << 31)) return fail(E3_ERR_SHAPE, "B = %lld", (long long)B);
  if (!one_ok && B != 1) return fail(E3_ERR_INVALID_ARG, "row_ptr is NULL but B is %lld", (long long)B);
  return E3_OK;
}

// Rows (and statistics) are moved in 16-byte vectors; `params` are read and written element by element.
e3_status check_pointers(const e3_features* f, const void* const* required, const char* const* names, int n,
                         const void* const* optional, int m, const void* const* params, int k) {
  for (int i = 0; i < n; ++i) {
    if (required[i] == nullptr) return fail(E3_ERR_INVALID_ARG, "%s is NULL", names[i]);
    if (reinterpret_cast<uintptr_t>(required[i]) & 15u)
      return fail(E3_ERR_INVALID_ARG, "%s is not 16-byte aligned", names[i]);
  }
  for (int i = 0; i < m; ++i)
    if (reinterpret_cast<uintptr_t>(optional[i]) & 15u)
      return fail(E3_ERR_INVALID_ARG, "an optional pointer is not 16-byte aligned");
  const uintptr_t element = f->dtype == E3_F64 ? 8 : 4;
  for (int i = 0; i < k; ++i)
    if (reinterpret_cast<uintptr_t>(params[i]) & (element - 1))
      return fail(E3_ERR_INVALID_ARG, "a weight, a bias or its gradient is not aligned to its type");
  return E3_OK;
}

// Common part of the three calls.
e3_status begin(const e3_features* f, int64_t N, int64_t B, const int32_t* row_ptr, int64_t max_rows, int op,
                e3_act act, const e3_dropout_spec* drop, void* ws, size_t ws_bytes, NormArgs* a, GnConfig* c,
                bool* drop_on) {
  e3_status st;
  if (act != E3_ACT_NONE && act != E3_ACT_SILU) return fail(E3_ERR_INVALID_ARG, "bad activation");
  if (reinterpret_cast<uintptr_t>(row_ptr) & 3u) return fail(E3_ERR_INVALID_ARG, "row_ptr is not 4-byte aligned");
  if ((st = drop_args(drop, N, &a->drop, drop_on)) != E3_OK) return st;
  *c = configure(f, N, B, max_rows, op, a);
  c->ws_bytes = ws_bytes;
  if (N > 0 && (st = check_workspace(ws, ws_bytes, workspace_bytes_of(*c, *a, op, f->vec))) != E3_OK) return st;
  if ((st = ensure_device_tables()) != E3_OK) return st;
  if ((st = device_status_ptr(&a->status)) != E3_OK) return st;
  a->row_ptr = row_ptr;
  a->act = act;
  return E3_OK;
}

e3_status zero_params(const e3_features* f, void* gw, void* gb, cudaStream_t s) {
  const size_t es = f->dtype == E3_F64 ? 8 : 4;
  if ((gw && cudaMemsetAsync(gw, 0, es * size_t(f->lay.n_channels), s) != cudaSuccess) ||
      (gb && f->lay.n_scalars && cudaMemsetAsync(gb, 0, es * size_t(f->lay.n_scalars), s) != cudaSuccess))
    return fail(E3_ERR_CUDA, "group norm: zeroing the gradients failed");
  return E3_OK;
}

}  // namespace

void make_tiles(e3_features* f) {
  const RowLayout& L = f->lay;
  // 16-byte vectors need every group to be a whole number of them (then every block, and the row, is)
  // (8 bytes for floats where the groups are even)
  f->vec = f->dtype == E3_F64 ? 2 : 4;
  for (int b = 0; b < L.n_blocks; ++b)
    while (L.blk[b].group_cols % f->vec != 0) f->vec /= 2;
  for (int b = 0; b < L.n_blocks; ++b) f->wide = std::max(f->wide, L.blk[b].group_cols / f->vec);
  for (int i = 0; i < 9; ++i)
    if ((f->wide << i) <= GN_THREADS)
      f->local[i] = best_tiles(L, f->vec, f->wide, GN_THREADS >> i, 1 << i, GN_THREADS);
  if (f->wide <= GN_ROW_THREADS) {
    // doubles: no more groups to a tile than a batch of one segment a thread has coefficients for
    const int most = f->dtype == E3_F64 ? GN_ROW_ITEMS / gn_reg_segments(GN_FWD, f->vec) : GN_ROW_THREADS;
    f->rows = best_tiles(L, f->vec, f->wide, GN_ROW_THREADS, 1, GN_ROW_THREADS, most);
  }
  f->grid = equal_tiles(L, f->vec);
  // narrow tiles for clusters, which leave the CTAs more row lanes
  if (f->wide <= 64) f->narrow = cut_tiles(L, f->vec, std::max(f->wide, 8));
  for (TileSet& t : f->local) count_scalars(L, f->vec, &t);
  count_scalars(L, f->vec, &f->rows);
  count_scalars(L, f->vec, &f->narrow);
  // clusters: few tiles, none with more groups than a CTA's table of its cluster's sums holds
  f->cluster_ok = f->narrow.n() > 0 && f->narrow.n() <= GN_LOCAL_TILES && f->narrow.groups <= 32;
}

// Bytes that a CTA reads for one part of the second pass (64 to 512 KB: 110 to 107 us for the forward of
// 24000 x 2048 floats, 203 to 191 us for the backward; parts start with an empty pipeline).
constexpr int64_t GN_PART_BYTES = 512 << 10;

size_t gn_grid_layout(NormArgs* a, int op, int64_t ctas) {
  const int64_t most = std::max<int64_t>(1, ctas / a->n_tiles);
  a->rows_cta = std::max<int64_t>((a->N + most - 1) / most, 2 * a->k);
  a->chunks = int32_t(std::max<int64_t>(1, (a->N + a->rows_cta - 1) / a->rows_cta));
  const size_t G = size_t(a->lay.n_groups());
  const size_t slots = a->wide ? size_t(most) + size_t(a->B) : 2 * size_t(most);
  const size_t coef = al256(slots * (G + size_t(a->n_tiles)) * gn_sums(op) * 8);
  const size_t col = coef + (op == GN_FWD ? 0 : al256(size_t(a->B) * G * gn_coefs(op) * 8));
  const int64_t bytes = a->rows_cta * a->tx * (op == GN_FWD ? 16 : 32);
  a->parts = op == GN_DBL ? 1 : int32_t(std::min<int64_t>(16, std::max<int64_t>(1, bytes / GN_PART_BYTES)));
  const size_t tickets = col + (op == GN_FWD ? 0 : al256(size_t(most) * 2 * size_t(a->lay.dim) * 8));
  a->part = nullptr;
  a->coef = reinterpret_cast<void*>(coef);   // offsets; the launcher adds the base
  a->colpart = reinterpret_cast<double*>(col);
  a->tickets = reinterpret_cast<int32_t*>(tickets);
  return tickets + al256(size_t(a->n_tiles) * 4);
}

size_t gn_column_bytes(const NormArgs& a, int op, int vec, int64_t ctas) {
  return op == GN_FWD ? 0 : al256(size_t(ctas) * 2 * size_t(a.tx) * size_t(vec) * 8);
}
size_t gn_local_layout(const NormArgs& a, int op, int vec, int64_t ctas) {
  return gn_column_bytes(a, op, vec, ctas) + (op != GN_FWD && a.cs > 1 ? al256(size_t(a.n_tiles) * 4) : 0);
}

// Even scalars with the activation take a batch half as long again (three quarters in the double backward);
// without it an eighth.  Every tile the same number of CTAs left some SMs with four times the instructions of
// others: 512 molecules of 34 rows x 512 columns, forward 32.0 to 29.6 us, backward 53.5 to 51.3, double
// backward 116 to 103; scalars at twice a batch: 34.2, 54.8, 111.
void gn_share(NormArgs* a, int op, const TileSet& t, int64_t batches, int64_t room) {
  const int n = t.n();
  const double extra = a->act != E3_ACT_SILU ? 0.125 : op == GN_DBL ? 0.75 : 0.5;
  auto cost = [&](int i) { return t.tx + extra * t.scalars[i]; };
  auto parts = [&](int i, double limit) {
    const double each = std::max(1.0, std::floor(limit / cost(i)));  // batches that a CTA does by the limit
    return std::max<int64_t>(1, std::min(batches, int64_t(std::ceil(double(batches) / each))));
  };
  auto total = [&](double limit) {
    int64_t s = 0;
    for (int i = 0; i < n; ++i) s += parts(i, limit);
    return s;
  };
  double hi = 0.0, lo = 0.0;  // the limit lies in (lo, hi]
  for (int i = 0; i < n; ++i) hi = std::max(hi, cost(i));
  if (total(hi) > room) {
    lo = hi;
    hi *= double(batches);
    for (int i = 0; i < 16 && hi > 1.01 * lo; ++i) {
      const double mid = std::sqrt(lo * hi);
      (total(mid) > room ? lo : hi) = mid;
    }
  }
  // what is left over goes to all of them
  const int64_t used = total(hi), left = std::max<int64_t>(0, room - used);
  a->start[0] = 0;
  a->even = 1;
  for (int i = 0; i < n; ++i) {
    const int64_t p = parts(i, hi);
    a->start[i + 1] = a->start[i] + int32_t(std::min(batches, p + p * left / used)) * a->cs;
    if (a->start[i + 1] != (i + 1) * a->start[1]) a->even = 0;
  }
}

}  // namespace e3b

using namespace e3b;

extern "C" e3_status e3_group_norm_workspace_size(const e3_features* f, int64_t N, int64_t B, int64_t max_rows,
                                                  size_t* bytes) {
  clear_error();
  if (f == nullptr || bytes == nullptr) return fail(E3_ERR_INVALID_ARG, "features or bytes is NULL");
  if (N < 0 || N > GN_MAX_ROWS || B < 1 || B >= (int64_t(1) << 31))
    return fail(E3_ERR_SHAPE, "N = %lld, B = %lld", (long long)N, (long long)B);
  *bytes = 0;
  for (int op = GN_FWD; op <= GN_DBL; ++op) {
    NormArgs a{};
    const GnConfig c = configure(f, N, B, max_rows, op, &a);
    *bytes = std::max(*bytes, workspace_bytes_of(c, a, op, f->vec));
  }
  return E3_OK;
}

extern "C" e3_status e3_group_norm_forward(const e3_features* f, int64_t N, int64_t B, const int32_t* row_ptr,
                                           int64_t max_rows, const void* x, const void* weight, const void* bias,
                                           double eps, e3_act act, const e3_dropout_spec* drop, void* y,
                                           double* stats, void* workspace, size_t workspace_bytes, void* stream) {
  clear_error();
  e3_status st = check_sizes(f, N, B, row_ptr != nullptr);
  if (st != E3_OK) return st;
  // the kernels add eps in the rows' type
  const double added = f->dtype == E3_F32 ? double(float(eps)) : eps;
  if (!(added > 0.0) || !std::isfinite(added))
    return fail(E3_ERR_INVALID_ARG, "eps = %g must be positive and finite in the rows' type", eps);
  NormArgs a{};
  GnConfig c;
  bool on = false;
  st = begin(f, N, B, row_ptr, max_rows, GN_FWD, act, drop, workspace, workspace_bytes, &a, &c, &on);
  if (st != E3_OK || N == 0) return st;
  const void* req[3] = {x, y, stats};
  const char* names[3] = {"x", "y", "stats"};
  const void* params[2] = {weight, bias};
  if ((st = check_pointers(f, req, names, 3, nullptr, 0, params, 2)) != E3_OK) return st;
  a.x = x;
  a.w = weight;
  a.b = bias;
  a.o0 = y;
  a.stats = stats;
  a.eps = eps;
  return gn_launch_fwd(a, c, f->dtype == E3_F64, f->vec, on, workspace, static_cast<cudaStream_t>(stream));
}

extern "C" e3_status e3_group_norm_backward(const e3_features* f, int64_t N, int64_t B, const int32_t* row_ptr,
                                            int64_t max_rows, const void* x, const double* stats, const void* weight,
                                            const void* bias, e3_act act, const e3_dropout_spec* drop,
                                            const void* grad_y, void* grad_x, void* grad_weight, void* grad_bias,
                                            void* workspace, size_t workspace_bytes, void* stream) {
  clear_error();
  e3_status st = check_sizes(f, N, B, row_ptr != nullptr);
  if (st != E3_OK) return st;
  NormArgs a{};
  GnConfig c;
  bool on = false;
  st = begin(f, N, B, row_ptr, max_rows, GN_BWD, act, drop, workspace, workspace_bytes, &a, &c, &on);
  if (st != E3_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (N == 0) return zero_params(f, grad_weight, grad_bias, s);
  const void* req[3] = {x, stats, grad_y};
  const char* names[3] = {"x", "stats", "grad_y"};
  const void* opt[1] = {grad_x};
  const void* params[4] = {weight, bias, grad_weight, grad_bias};
  if ((st = check_pointers(f, req, names, 3, opt, 1, params, 4)) != E3_OK) return st;
  a.x = x;
  a.g = grad_y;
  a.w = weight;
  a.b = bias;
  a.o0 = grad_x;
  a.stats = const_cast<double*>(stats);
  a.gw = grad_weight;
  a.gb = f->lay.n_scalars > 0 ? grad_bias : nullptr;
  if (a.o0 == nullptr && a.gw == nullptr && a.gb == nullptr) return E3_OK;
  return gn_launch_bwd(a, c, f->dtype == E3_F64, f->vec, on, workspace, s);
}

extern "C" e3_status e3_group_norm_double_backward(const e3_features* f, int64_t N, int64_t B, const int32_t* row_ptr,
                                                   int64_t max_rows, const void* x, const double* stats,
                                                   const void* weight, const void* bias, e3_act act,
                                                   const e3_dropout_spec* drop, const void* grad_y, const void* u_x,
                                                   const void* u_weight, const void* u_bias, void* d_grad_y,
                                                   void* d_x, void* d_weight, void* d_bias, void* workspace,
                                                   size_t workspace_bytes, void* stream) {
  clear_error();
  e3_status st = check_sizes(f, N, B, row_ptr != nullptr);
  if (st != E3_OK) return st;
  NormArgs a{};
  GnConfig c;
  bool on = false;
  st = begin(f, N, B, row_ptr, max_rows, GN_DBL, act, drop, workspace, workspace_bytes, &a, &c, &on);
  if (st != E3_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (N == 0) return zero_params(f, d_weight, d_bias, s);
  const void* req[3] = {x, stats, grad_y};
  const char* names[3] = {"x", "stats", "grad_y"};
  const void* opt[3] = {u_x, d_grad_y, d_x};
  const void* params[6] = {weight, bias, u_weight, u_bias, d_weight, d_bias};
  if ((st = check_pointers(f, req, names, 3, opt, 3, params, 6)) != E3_OK) return st;
  a.x = x;
  a.g = grad_y;
  a.u = u_x;
  a.w = weight;
  a.b = bias;
  a.uw = u_weight;
  a.ub = u_bias;
  a.o0 = d_x;
  a.o1 = d_grad_y;
  a.stats = const_cast<double*>(stats);
  a.gw = d_weight;
  a.gb = f->lay.n_scalars > 0 ? d_bias : nullptr;
  if (a.o0 == nullptr && a.o1 == nullptr && a.gw == nullptr && a.gb == nullptr) return E3_OK;
  return gn_launch_dbl(a, c, f->dtype == E3_F64, f->vec, on, workspace, s);
}
