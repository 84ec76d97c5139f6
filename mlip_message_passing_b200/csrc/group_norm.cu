// Group norm of feature rows: configuration, the parameters' gradients and the C ABI.
#include <cmath>

#include "group_norm_launch.h"

namespace e3b {
namespace {

size_t al256(size_t b) { return (b + 255) & ~size_t(255); }

// 16-byte vectors need every group to be a whole number of them (then every block, and the row, is).
int vec_of(const RowLayout& L, e3_dtype dt) {
  const int v = dt == E3_F64 ? 2 : 4;
  for (int b = 0; b < L.n_blocks; ++b)
    if (L.blk[b].group_cols % v != 0) return 1;
  return v;
}

int pow2_at_least(int64_t n) {
  int p = 1;
  while (p < n && p < 32) p *= 2;
  return p;
}

GnConfig configure(const e3_features* f, int64_t N, int64_t B, int64_t max_rows, int op, NormArgs* a) {
  const RowLayout& L = f->lay;
  GnConfig c;
  c.vec = vec_of(L, f->dtype);
  const int V = L.dim / c.vec;
  int wide = 0;  // widest group in vectors
  for (int b = 0; b < L.n_blocks; ++b) wide = std::max(wide, L.blk[b].group_cols / c.vec);
  const int64_t most = max_rows > 0 ? std::min(max_rows, N) : N;
  const int RP = gn_reg_rows(op);
  // local: a segment's widest group fits the registers of one CTA
  if (wide <= GN_THREADS && most <= int64_t(RP) * (GN_THREADS / wide)) {
    int K = int(std::max<int64_t>(1, (most + RP - 1) / RP));
    const int cap = std::max(wide, GN_THREADS / K);
    a->n_slabs = 0;
    a->slab[0] = 0;
    int tx = 0, at = 0;
    bool fits = true;
    for (int b = 0; b < L.n_blocks && fits; ++b)
      for (int g = 0; g < L.groups; ++g) {
        const int w = L.blk[b].group_cols / c.vec;
        if (at + w - a->slab[a->n_slabs] > cap) {
          if (a->n_slabs + 2 > GN_MAXSLAB) {
            fits = false;
            break;
          }
          a->slab[++a->n_slabs] = at;
        }
        at += w;
        tx = std::max(tx, at - a->slab[a->n_slabs]);
      }
    if (fits) {
      a->slab[++a->n_slabs] = at;
      c.local = true;
      a->tx = tx;
      a->j = std::max(1, GN_THREADS / (tx * K));
      a->k = a->j == 1 ? std::max(K, GN_THREADS / tx) : K;
      a->lanes = pow2_at_least(int64_t(a->k) * wide);
      const int64_t batches = (B + a->j - 1) / a->j;
      const int64_t want = std::max<int64_t>(1, int64_t(8) * sm_count() / a->n_slabs);
      c.grid = dim3(unsigned(std::min(batches, want)), unsigned(a->n_slabs));
      c.col_parts = c.grid.x;
    }
  }
  size_t at = 0;
  if (!c.local) {
    a->tx = std::min(V, 64);
    a->k = GN_THREADS / a->tx;
    a->j = 1;
    a->n_tiles = (V + a->tx - 1) / a->tx;
    a->lanes = pow2_at_least(int64_t(a->k) * std::min(wide, a->tx));
    const int64_t want = std::max<int64_t>(1, int64_t(4) * sm_count() / a->n_tiles);
    const int64_t least = int64_t(a->k) * 8;
    a->rows_cta = std::max((N + want - 1) / want, least);
    a->n_chunks = (N + a->rows_cta - 1) / a->rows_cta;
    c.grid = dim3(unsigned(a->n_chunks), unsigned(a->n_tiles));
    c.col_parts = a->n_chunks;
    const size_t G = size_t(L.n_groups());
    c.part = 0;
    c.coef = al256(size_t(a->n_chunks + B) * (G + size_t(a->n_tiles)) * gn_sums(op) * 8);
    at = c.coef + al256(size_t(B) * G * gn_coefs(op) * 8);
  }
  c.colpart = at;
  c.total = at + (op == GN_FWD ? 0 : al256(size_t(c.col_parts) * 2 * size_t(L.dim) * 8));
  c.total = std::max<size_t>(c.total, 256);
  return c;
}

// Gradients of the weights and biases: column sums of all CTAs, joined in order, then added over the
// components of a channel.  blockIdx.y: 0 weights, 1 biases.
constexpr int CS_COLS = 1024;
__host__ __device__ int cs_channels(int d) { return CS_COLS / d < 32 ? CS_COLS / d : 32; }

template <typename T>
__global__ void __launch_bounds__(256) gn_colsum_kernel(const double* colpart, int64_t parts, T* gw, T* gb,
                                                        const __grid_constant__ RowLayout L) {
  __shared__ double acc[8][33];
  __shared__ double cols[CS_COLS];
  int bi = 0, at = int(blockIdx.x);
  while (true) {
    const int n = (L.blk[bi].mul + cs_channels(L.blk[bi].d) - 1) / cs_channels(L.blk[bi].d);
    if (at < n) break;
    at -= n;
    ++bi;
  }
  const RowBlock& b = L.blk[bi];
  const bool bias = blockIdx.y == 1;
  if (bias ? (gb == nullptr || b.bias0 < 0) : gw == nullptr) return;
  const int u0 = at * cs_channels(b.d), nu = min(cs_channels(b.d), b.mul - u0), ncol = nu * b.d;
  const int tx = int(threadIdx.x) % 32, ty = int(threadIdx.x) / 32;
  for (int c0 = 0; c0 < ncol; c0 += 32) {
    double s = 0.0;
    if (c0 + tx < ncol) {
      const double* p = colpart + (bias ? L.dim : 0) + b.col0 + u0 * b.d + c0 + tx;
      for (int64_t i = ty; i < parts; i += 8) s += p[i * 2 * L.dim];
    }
    acc[ty][tx] = s;
    __syncthreads();
    if (ty == 0 && c0 + tx < ncol) {
#pragma unroll
      for (int i = 1; i < 8; ++i) s += acc[i][tx];
      cols[c0 + tx] = s;
    }
    __syncthreads();
  }
  if (int(threadIdx.x) < nu) {
    double s = 0.0;
    for (int m = 0; m < b.d; ++m) s += cols[int(threadIdx.x) * b.d + m];
    if (bias) gb[b.bias0 + u0 + threadIdx.x] = T(s);
    else gw[b.chan0 + u0 + threadIdx.x] = T(s);
  }
}

void launch_colsum(const e3_features* f, const GnConfig& c, const double* colpart, void* gw, void* gb, cudaStream_t s) {
  const RowLayout& L = f->lay;
  int n = 0;
  for (int b = 0; b < L.n_blocks; ++b) n += (L.blk[b].mul + cs_channels(L.blk[b].d) - 1) / cs_channels(L.blk[b].d);
  if (L.n_scalars == 0) gb = nullptr;
  if (gw == nullptr && gb == nullptr) return;
  const dim3 grid{unsigned(n), gb ? 2u : 1u};
  if (f->dtype == E3_F64)
    gn_colsum_kernel<double><<<grid, 256, 0, s>>>(colpart, c.col_parts, static_cast<double*>(gw),
                                                  static_cast<double*>(gb), L);
  else
    gn_colsum_kernel<float><<<grid, 256, 0, s>>>(colpart, c.col_parts, static_cast<float*>(gw),
                                                 static_cast<float*>(gb), L);
}

e3_status check_sizes(const e3_features* f, int64_t N, int64_t B, bool one_ok) {
  const e3_status st = check_features_device(f);
  if (st != E3_OK) return st;
  if (N < 0 || N >= (int64_t(1) << 31)) return fail(E3_ERR_SHAPE, "N = %lld", (long long)N);
  if (B < 1 || B >= (int64_t(1) << 31)) return fail(E3_ERR_SHAPE, "B = %lld", (long long)B);
  if (!one_ok && B != 1) return fail(E3_ERR_INVALID_ARG, "row_ptr is NULL but B is %lld", (long long)B);
  return E3_OK;
}

e3_status check_pointers(const void* const* required, const char* const* names, int n, const void* const* optional,
                         int m) {
  for (int i = 0; i < n; ++i) {
    if (required[i] == nullptr) return fail(E3_ERR_INVALID_ARG, "%s is NULL", names[i]);
    if (reinterpret_cast<uintptr_t>(required[i]) & 15u)
      return fail(E3_ERR_INVALID_ARG, "%s is not 16-byte aligned", names[i]);
  }
  for (int i = 0; i < m; ++i)
    if (reinterpret_cast<uintptr_t>(optional[i]) & 15u)
      return fail(E3_ERR_INVALID_ARG, "an optional pointer is not 16-byte aligned");
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
  if (N > 0) {
    if (ws == nullptr || (reinterpret_cast<uintptr_t>(ws) & 15u))
      return fail(E3_ERR_INVALID_ARG, "workspace is NULL or not 16-byte aligned");
    if (ws_bytes < c->total)
      return fail(E3_ERR_SHAPE, "workspace of %zu bytes, %zu needed", ws_bytes, c->total);
  }
  if ((st = ensure_device_tables()) != E3_OK) return st;
  if ((st = device_status_ptr(&a->status)) != E3_OK) return st;
  a->N = N;
  a->B = int32_t(B);
  a->row_ptr = row_ptr;
  a->act = act;
  a->lay = f->lay;
  char* base = static_cast<char*>(ws);
  a->part = reinterpret_cast<double*>(base + c->part);
  a->coef = reinterpret_cast<double*>(base + c->coef);
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
}  // namespace e3b

using namespace e3b;

extern "C" e3_status e3_group_norm_workspace_size(const e3_features* f, int64_t N, int64_t B, int64_t max_rows,
                                                  size_t* bytes) {
  clear_error();
  if (f == nullptr || bytes == nullptr) return fail(E3_ERR_INVALID_ARG, "features or bytes is NULL");
  if (N < 0 || N >= (int64_t(1) << 31) || B < 1 || B >= (int64_t(1) << 31))
    return fail(E3_ERR_SHAPE, "N = %lld, B = %lld", (long long)N, (long long)B);
  *bytes = 0;
  for (int op = GN_FWD; op <= GN_DBL; ++op) {
    NormArgs a{};
    *bytes = std::max(*bytes, configure(f, N, B, max_rows, op, &a).total);
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
  if (!(eps > 0.0) || !std::isfinite(eps)) return fail(E3_ERR_INVALID_ARG, "eps = %g must be positive", eps);
  NormArgs a{};
  GnConfig c;
  bool on = false;
  st = begin(f, N, B, row_ptr, max_rows, GN_FWD, act, drop, workspace, workspace_bytes, &a, &c, &on);
  if (st != E3_OK || N == 0) return st;
  const void* req[3] = {x, y, stats};
  const char* names[3] = {"x", "y", "stats"};
  const void* opt[2] = {weight, bias};
  if ((st = check_pointers(req, names, 3, opt, 2)) != E3_OK) return st;
  a.x = x;
  a.w = weight;
  a.b = bias;
  a.o0 = y;
  a.stats = stats;
  a.eps = eps;
  return gn_launch_fwd(a, c, f->dtype == E3_F64, on, static_cast<cudaStream_t>(stream));
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
  const void* opt[5] = {weight, bias, grad_x, grad_weight, grad_bias};
  if ((st = check_pointers(req, names, 3, opt, 5)) != E3_OK) return st;
  a.x = x;
  a.g = grad_y;
  a.w = weight;
  a.b = bias;
  a.o0 = grad_x;
  a.stats = const_cast<double*>(stats);
  if (grad_weight || grad_bias) a.colpart = reinterpret_cast<double*>(static_cast<char*>(workspace) + c.colpart);
  if (grad_x == nullptr && a.colpart == nullptr) return E3_OK;
  if ((st = gn_launch_bwd(a, c, f->dtype == E3_F64, on, s)) != E3_OK) return st;
  launch_colsum(f, c, a.colpart, grad_weight, grad_bias, s);
  const cudaError_t err = cudaGetLastError();
  if (err != cudaSuccess) return fail(E3_ERR_CUDA, "group norm backward launch failed: %s", cudaGetErrorString(err));
  return E3_OK;
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
  const void* opt[9] = {weight, bias, u_x, u_weight, u_bias, d_grad_y, d_x, d_weight, d_bias};
  if ((st = check_pointers(req, names, 3, opt, 9)) != E3_OK) return st;
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
  if (d_weight || d_bias) a.colpart = reinterpret_cast<double*>(static_cast<char*>(workspace) + c.colpart);
  if (d_x == nullptr && d_grad_y == nullptr && a.colpart == nullptr) return E3_OK;
  if ((st = gn_launch_dbl(a, c, f->dtype == E3_F64, on, s)) != E3_OK) return st;
  launch_colsum(f, c, a.colpart, d_weight, d_bias, s);
  const cudaError_t err = cudaGetLastError();
  if (err != cudaSuccess)
    return fail(E3_ERR_CUDA, "group norm double backward launch failed: %s", cudaGetErrorString(err));
  return E3_OK;
}
